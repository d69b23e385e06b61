"""float16 weights far below a row's largest: many of them together count although each is
below float16's smallest step.

Bound: paged_util's, and what a weight held in 16 bits loses at the bottom of float16's
range.  Its step there is 2^-24; in the split kernel the weights are scaled by 2^15 and the
part that rounding left is held too, so a weight is off by at most 2^-40 of the largest; in
the row tiles they are scaled by 2^11 against the row's reference, so by at most 2^-36.
Every token of N may lose that: N 2^-40 (N 2^-36) max |v| in the output."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import PAGE, attention, attention_bounds
from test_gpu_paged_cross import Cross
from test_gpu_paged_decode import Decode
from paged_util import Pages

pytestmark = pytest.mark.gpu


def peaked(n, at, below, D, dtype="f16"):
    """One token at `at` whose value is 0, `below` above n - 1 others in the scores of q = e0."""
    pg = Pages([n], 1, D, dtype, 1)
    k, v = torch.zeros(n, D, dtype=torch.float64), torch.rand(n, D, generator=pg.gen, dtype=torch.float64) / 2 + 0.5
    k[at, 0], v[at] = below, 0
    k, v = k.to(pg.dtype), v.to(pg.dtype)
    pg.keys, pg.values = [k.double()[:, None]], [v.double()[:, None]]
    t = torch.arange(n)
    slot = pg.table[0, t // PAGE].long()
    pg.k[slot, 0, t % PAGE], pg.v[slot, 0, t % PAGE] = k, v
    return pg


def check(c, rows, D, out_dtype, step, one_plane):
    torch.cuda.synchronize()
    pg = c.pg
    n = pg.lens[0]
    o, lse, a, s = attention(c.q[:rows, :D].double(), pg.keys[0][:, 0], pg.values[0][:, 0],
                             torch.ones(rows, n, dtype=torch.bool), c.scale)
    o_tol, lse_tol = attention_bounds(o, lse, a, s, D, n, out_dtype, pg.dtype, one_plane)
    d = (c.o[:rows, :D].double().cpu() - o).abs()
    assert (d <= o_tol + n * step).all(), f"o off by {(d / (o_tol + n * step)).max():.2f} of its bound, {(d / o).max():.1e} of itself"
    d = (c.lse[:rows, 0].double().cpu() - lse).abs()
    assert (d <= lse_tol).all(), f"lse off by {(d / lse_tol).max():.2f} of its bound"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,at", [(500, 3), (500, 499), (3000, 5), (9000, 4000)])
@pytest.mark.parametrize("below", [12.0, 17.40625, 24.0])
def test_decode(n, at, below, D):
    pg = peaked(n, at, below, D)
    d = Decode(pg, 1, o_f32=True, scale=1.0)
    for x in (d.q, d.dq):
        x.zero_()
        x[:, 0] = 1
    d.call()
    check(d, 1, D, torch.float32, 2.0 ** -40, False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,n,at", [(1, 4000, 2), (200, 65537, 0), (200, 65537, 60000), (9000, 20000, 70), (9000, 300, 1)])
@pytest.mark.parametrize("below", [12.0, 17.40625])
def test_cross(rows, n, at, below, D):
    """One row, keys split into parts, keys not split."""
    pg = peaked(n, at, below, D)
    c = Cross(pg, [rows], 1, scale=1.0)
    for x in (c.q, c.dq):
        x.zero_()
        x[:, 0] = 1
    c.call()
    c.q = c.q[:1]
    same = c.o[:rows, :D]
    assert torch.equal(same, same[:1].expand_as(same))
    check(c, 1, D, torch.float16, 2.0 ** -36, True)
