"""Finite queries and keys whose scores are so large that a float32 holds them to whole
units or worse.  One token, of one new token per request or of few queries, takes the
weight and nothing overflows; rows of many queries may refuse with NaN in both outputs
from the documented size on, and only from there.  (The bounds of paged_util grow with the
scores, so what is tested is that outputs are finite and within the values' range; rows
whose largest score stands far enough out are its tokens' mean value.)"""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import Pages
from test_gpu_paged_cross import Cross
from test_gpu_paged_decode import Decode

pytestmark = pytest.mark.gpu


def far(pg, rows, top, neg):
    """Keys and queries along channel 0, up to `top` in size."""
    for b, n in enumerate(pg.lens):
        k = torch.zeros(n, pg.H, pg.D, dtype=torch.float64)
        k[..., 0] = top * (0.3 + 0.7 * torch.rand(n, pg.H, generator=pg.gen, dtype=torch.float64)) * (-1 if neg else 1)
        k = k.to(pg.dtype)
        pg.keys[b] = k.double()
        for i in range(-(-n // 64)):
            part = k[i * 64:(i + 1) * 64]
            pg.k[pg.table[b, i], :, :part.shape[0]] = part.transpose(0, 1)


def check(c, off, what, limit=float("inf")):
    torch.cuda.synchronize()
    pg, G, D = c.pg, c.G, c.pg.D
    o, lse = c.o.double().cpu(), c.lse.double().cpu()
    sure = 0
    for b, n in enumerate(pg.lens):
        for j in range(pg.H * G):
            rows = slice(off[b], off[b + 1])
            x = c.q[rows, j * D:(j + 1) * D].double() @ pg.keys[b][:, j // G].T * c.scale
            top = x.max(1).values
            got, v = o[rows, j * D:(j + 1) * D], pg.values[b][:, j // G]
            refused = torch.isnan(lse[rows, j]) & torch.isnan(got).all(1)
            assert (x.abs().max(1).values[refused] > limit).all(), what
            keep = ~refused
            got, top, x, line = got[keep], top[keep], x[keep], lse[rows, j][keep]
            assert torch.isfinite(got).all() and torch.isfinite(line).all(), what
            lo, hi = v.min(0).values, v.max(0).values
            slack = 2.0 ** -7 * v.abs().max()
            assert (got >= lo - slack).all() and (got <= hi + slack).all(), what
            # float32 holds the score to 2^-23 of itself after 2^-22 a matrix step
            err = (D // 16 + 2) * 2.0 ** -22 * top.abs()
            assert ((line - top).abs() <= err + 20).all(), what
            # tokens of the largest score (16-bit keys repeat) share the weight evenly
            ties = (x == top[:, None]).double()
            mean = ties @ v / ties.sum(1, keepdim=True)
            second = x.masked_fill(ties > 0, float("-inf")).max(1).values
            out = top - second > 2 * err + 40
            sure += int(out.sum())
            assert ((got[out] - mean[out]).abs() <= slack).all(), what
    assert sure > 0 or limit < float("inf")


@pytest.mark.parametrize("dtype,top", [("f16", 1.5e3), ("f16", 3e3), ("f16", 2e4), ("f16", 6e4), ("bf16", 1e4), ("bf16", 2e5), ("bf16", 1e8), ("bf16", 1e15)])
@pytest.mark.parametrize("D,nq,lens,G", [(64, [200, 150], [300, 700], 64), (128, [300], [2000], 2), (256, [300, 90], [900, 40], 2),
                                         (128, [3], [700], 2), (64, [700], [128], 16)])
@pytest.mark.parametrize("scale", [1.0, -0.5])
def test_cross(D, nq, lens, G, dtype, top, scale):
    pg = Pages(lens, 1, D, dtype, 5)
    far(pg, sum(nq), top, scale < 0)
    c = Cross(pg, nq, G, scale=scale)
    c.q.zero_()
    first = top * (0.3 + 0.7 * torch.rand(c.T, G, generator=pg.gen, dtype=torch.float64))
    c.q.view(c.T, G, D)[..., 0] = first.to(pg.dtype)
    c.dq.copy_(c.q)
    c.call()
    check(c, c.off, f"{dtype} {top:g}", 2.0 ** 22 if dtype == "f16" else 2.0 ** 28)
    assert tpk.get_device_status(reset=True) == (0, 0)


@pytest.mark.parametrize("dtype,top", [("f16", 6e4), ("bf16", 1e8)])
@pytest.mark.parametrize("D,n", [(64, 300), (128, 5000), (256, 900)])
def test_decode(D, n, dtype, top):
    pg = Pages([n], 1, D, dtype, 6)
    far(pg, 1, top, False)
    d = Decode(pg, 3, scale=1.0)
    d.q.zero_()
    d.q.view(1, 3, D)[..., 0] = torch.tensor([top, top / 2, top / 3], dtype=torch.float64).to(pg.dtype)
    d.dq.copy_(d.q)
    d.call()
    check(d, [0, 1], f"{dtype} {top:g}")


def test_a_far_first_tile_is_refused_or_overcome():
    """The first 128 keys' scores are far below zero, the others near it: they have no weight."""
    for dtype, size in (("f16", 6e4), ("bf16", 1e9)):
        pg = Pages([900], 1, 128, dtype, 7)
        k = pg.keys[0].clone()
        k[:128] = 0
        k[:128, :, 0] = -size
        k = k.to(pg.dtype)
        pg.keys[0] = k.double()
        for i in range(15):
            part = k[i * 64:(i + 1) * 64]
            pg.k[pg.table[0, i], :, :part.shape[0]] = part.transpose(0, 1)
        c = Cross(pg, [300], 2, scale=1.0)
        c.q.view(300, 2, 128)[..., 0] = size
        k0 = k.clone()
        k0[128:, :, 0] = 0  # the others do not see the large channel
        pg.keys[0] = k0.double()
        for i in range(2, 15):
            pg.k[pg.table[0, i], :, :min(64, 900 - 64 * i), 0] = 0
        c.k.copy_(pg.k)
        c.dq.copy_(c.q)
        c.call()
        torch.cuda.synchronize()
        o, lse = c.o.double().cpu(), c.lse.double().cpu()
        refused = torch.isnan(lse)
        assert torch.equal(refused, torch.isnan(o.view(300, 2, 128)).all(2))
        for j in range(2):
            x = c.q[:, j * 128:(j + 1) * 128].double() @ pg.keys[0][:, 0].T
            keep = ~refused[:, j]
            assert torch.isfinite(o[:, j * 128:(j + 1) * 128][keep]).all()
            assert ((lse[:, j] - torch.logsumexp(x, 1)).abs()[keep] <= 1e-3).all()
