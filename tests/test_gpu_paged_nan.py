"""A query row with a NaN comes out as NaN, output and log-sum alike, whatever kernel takes
it and however its history is cut: (0, -inf) is kept for rows that see nothing.  The rows
beside it are what they are without it, bit for bit."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import Pages
from test_gpu_paged_cross import Cross
from test_gpu_paged_decode import Decode

pytestmark = pytest.mark.gpu


def poison(c, rows, heads, call_rows):
    """Calls c clean and with a NaN in the given (row, head) queries, and compares."""
    H, G, D = c.pg.H, c.G, c.pg.D
    c.call()
    c.check()
    o, lse = c.o.clone(), c.lse.clone()
    mark = torch.zeros(call_rows, H * G, dtype=torch.bool)
    for i, r in enumerate(rows):
        for j, h in enumerate(heads):
            at = h * D + (7 * i + 13 * j) % D
            c.dq[r, at] = float("nan")
            mark[r, h] = True
    c.o.fill_(5.0)
    c.lse.fill_(5.0)
    c.ws.fill_(0xFF)
    c.call()
    torch.cuda.synchronize()
    mark = mark.cuda()
    live = ~torch.isnan(lse[:call_rows])
    got_o = c.o[:call_rows, :H * G * D].view(call_rows, H * G, D)
    assert torch.isnan(got_o[mark]).all() and torch.isnan(c.lse[:call_rows][mark]).all()
    same = live & ~mark
    assert torch.equal(got_o[same], o[:call_rows, :H * G * D].view(call_rows, H * G, D)[same])
    assert torch.equal(c.lse[:call_rows][same], lse[:call_rows][same])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,H,G,pages", [([100, 300, 40], 1, 4, None),          # whole, up to 8 rows a run
                                            ([(i * 37) % 300 + 1 for i in range(60)], 4, 16, 5),  # 16 rows
                                            ([(i * 137) % 700 + 1 for i in range(110)], 4, 3, None),
                                            ([5000, 70], 1, 8, None),               # cut
                                            ([(i * 379) % 1500 + 1 for i in range(12)], 4, 20, 40),
                                            ([(i * 37) % 400 + 1 for i in range(300)], 1, 2, 40)],
                         ids=lambda x: f"{len(x)}x{max(x)}" if isinstance(x, list) else str(x))
def test_decode(lens, H, G, pages, D):
    d = Decode(Pages(lens, H, D, "bf16", 3, max_pages=pages), G)
    poison(d, range(0, len(lens), 2), [0, H * G - 1], len(lens))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,lens,H,G", [([3, 2], [100, 300], 1, 4), ([4, 3], [5000, 64], 1, 2),  # split kernel
                                         ([200, 150], [300, 70], 64, 1),                     # row tiles
                                         ([300, 20], [2000, 700], 1, 2), ([40, 130], [900, 3000], 1, 3)],  # keys split
                         ids=lambda x: "-".join(map(str, x)) if isinstance(x, list) else str(x))
def test_cross(nq, lens, H, G, D):
    c = Cross(Pages(lens, H, D, "f16", 4), nq, G)
    poison(c, range(0, c.T, 3), [0, H * G - 1], c.T)


def test_cross_ranges_with_split_keys():
    """A row that sees nothing beside a NaN row: one is empty, the other is not."""
    r = [(0, 0) if i % 4 == 1 else (i * 3, i * 3 + 500) for i in range(300)]
    c = Cross(Pages([2000], 1, 128, "bf16", 5), [300], 2, ranges=r)
    poison(c, range(0, 300, 4), [1], 300)
    assert (c.lse[1::4] == float("-inf")).all() and (c.o[1::4] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [200, 5000])
def test_an_infinite_value_stays_in_its_channel(n, D):
    pg = Pages([n], 1, D, "bf16", 6)
    d = Decode(pg, 4)
    d.call()
    d.check()
    o, lse = d.o.clone(), d.lse.clone()
    d.v[pg.table[0, 1].item(), 0, 5, 7] = float("inf")
    d.call()
    torch.cuda.synchronize()
    got = d.o.view(4, D)
    assert not torch.isfinite(got[:, 7]).any() and torch.equal(d.lse, lse)
    keep = torch.arange(D) != 7
    assert torch.equal(got[:, keep], o.view(4, D)[:, keep])
