"""Shared prefixes where scores are far out: tokens of one score share the weight evenly, whichever side of
the prefix's end they are on and whichever launch reads them.

Queries and keys are along one channel, so that a score is one product, exact in float32, and equal scores
are equal to the bit.  The tokens below the largest score have half of it, too little for any weight; the others
have the weight 1 (2^11 in float16's row tiles) to exp2's 2^-21, which rounds to 16 bits without a rest.  So
the output is their mean value, to its own rounding, twice that 2^-21 of A = mean |v| (their numerator and
their sum), as much again for the factors of the join, and a truncation of 2^-22 A a matrix step.  lse: the score's
way to base 2 and back, and the sum's logarithm on the way, are at most eight float32 roundings of it."""
import math

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import attention, attention_bounds
from test_gpu_paged_shared import FEW_AND_MANY, Shared

pytestmark = pytest.mark.gpu


def far(groups, H, G, D, dtype, exponent, sign=1.0, **kw):
    """A call whose largest score is 1.71875 * 2^exponent, at the tokens whose value is positive in channel 0."""
    c = Shared(groups, H, G, D, dtype, **kw)
    a, b = exponent // 2, exponent - exponent // 2
    up = c.v[..., 0] > 0
    key = torch.where(up, 1.25 * 2.0 ** a, 1.25 * 2.0 ** (a - 1)) * sign
    key = torch.where(torch.isnan(c.k[..., 0]), float("nan"), key)
    c.k.masked_fill_(~torch.isnan(c.k), 0)
    c.k[..., 0] = key.to(c.dtype)
    c.dq.zero_()
    c.dq[:, :H * G * D].view(c.n, H * G, D)[..., 0] = 1.375 * 2.0 ** b / abs(c.scale)
    c.top = 1.71875 * 2.0 ** exponent
    return c


def check_far(c, what):
    c.call()
    torch.cuda.synchronize()
    H, G, D = c.H, c.G, c.D
    o, lse = c.o.double().cpu(), c.lse.double().cpu()
    eps = torch.finfo(c.o.dtype)
    for b, n in enumerate(c.lens):
        for h in range(H):
            got, line = o[b, h * G * D:(h + 1) * G * D].view(G, D), lse[b, h * G:(h + 1) * G]
            v, top = c.values[b][:, h], c.top
            at = f"{what} request {b} of {n} head {h}"
            if n == 0:
                assert (got == 0).all() and (line == float("-inf")).all(), at
                continue
            up = v[:, 0] > 0
            if up.any():
                v = v[up]
            else:
                top = top / 2
            mean, size = v.mean(0), v.abs().mean(0)
            tol = eps.eps / 2 * mean.abs() + (2.0 ** -19 + (n // 16 + 2) * 2.0 ** -22) * (1 + eps.eps / 2) * size + eps.tiny * eps.eps
            d = (got - mean).abs() / tol
            assert (d <= 1).all(), f"{at}: o off by {d.max():.2f} of its bound"
            want = top + math.log(len(v))
            d = (line - want).abs() / (2.0 ** -21 * want + 2.0 ** -20)
            assert (d <= 1).all(), f"{at}: lse off by {d.max():.2f} of its bound"
    assert tpk.get_device_status(reset=True) == (0, 0)


GROUPS = [[(300, [400, 401, 301])], [(1, [1001, 1, 2])], [(1000, [1001, 1000, 1300, 500, 0])], [(130, [140, 300]), (64, [65, 9000])]]


@FEW_AND_MANY
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,exponents", [("f16", [6, 13, 17, 20, 21]), ("bf16", [6, 13, 17, 20, 23, 27])])
def test_equal_scores_share_evenly(dtype, exponents, D, G, wide):
    for e in exponents:
        for groups in GROUPS:
            check_far(far(groups, 1, G, D, dtype, e, f32=True, scale=1.0, max_pages=wide), f"2^{e}")


@FEW_AND_MANY
def test_negative_scale_and_rounded_outputs(G, wide):
    for e in (14, 19, 21):
        check_far(far(GROUPS[0], 2, G, 128, "f16", e, sign=-1.0, scale=-0.5, max_pages=wide), f"2^{e}")
        check_far(far(GROUPS[2], 2, G, 64, "bf16", e, sign=-1.0, scale=-0.5, max_pages=wide, alone=(30, 77)), f"2^{e}")


@pytest.mark.parametrize("dtype,exponent", [("f16", 20), ("bf16", 26)])
def test_many_rows_behind_a_long_prefix(dtype, exponent):
    """Several row tiles and parts, ranges of what requests have of their own."""
    for D in (64, 256):
        check_far(far([(3000, [3000 + (i * 77) % 900 for i in range(70)])], 1, 8, D, dtype, exponent, f32=True, scale=1.0), "")


@FEW_AND_MANY
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0, 1.0, 16.0])
def test_bounds_without_a_join_of_logarithms(scale, dtype, G, wide):
    """Ordinary inputs: the bounds of decode with one plane, and 2^-21 of each weight for the join's factors."""
    for D in (64, 128, 256):
        c = Shared([(300, [350, 420, 301]), (70, [90, 75])], 2, G, D, dtype, f32=True, scale=scale, max_pages=wide, alone=(40,))
        c.call()
        torch.cuda.synchronize()
        o, lse = c.o.cpu(), c.lse.cpu()
        for b, n in enumerate(c.lens):
            for h in range(2):
                q = c.q[b, h * G * D:(h + 1) * G * D].double().view(G, D)
                ro, rl, a, s = attention(q, c.keys[b][:, h], c.values[b][:, h], torch.ones(G, n, dtype=torch.bool), c.scale)
                go, gl = o[b, h * G * D:(h + 1) * G * D].view(G, D), lse[b, h * G:(h + 1) * G]
                o_tol, lse_tol = attention_bounds(ro, rl, a, s, D, n, go.dtype, c.dtype, one_plane=True)
                assert ((go.double() - ro).abs() <= o_tol + 2.0 ** -20 * a).all(), (D, b, h)
                assert ((gl.double() - rl).abs() <= lse_tol + 2.0 ** -21).all(), (D, b, h)
        assert tpk.get_device_status(reset=True) == (0, 0)
