"""Float32 outputs of decode over shared prefixes, as they are merged with other partials: weights in two 16-bit
planes whichever launch reads the prefix, so the bounds of decode hold (paged_util), with 2^-20 A for the
factors of the join (2^-21 for each weight, in the numerator and in the sum)."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import attention, attention_bounds
from test_gpu_paged_shared import Shared

pytestmark = pytest.mark.gpu


def run(*args, status=(0, 0), **kw):
    c = Shared(*args, f32=True, **kw)
    c.call()
    torch.cuda.synchronize()
    H, G, D = c.H, c.G, c.D
    o, lse = c.o.cpu(), c.lse.cpu()
    for b, n in enumerate(c.lens):
        for h in range(H):
            go, gl = o[b, h * G * D:(h + 1) * G * D].view(G, D), lse[b, h * G:(h + 1) * G]
            if n == 0:
                assert (go == 0).all() and (gl == float("-inf")).all()
                continue
            q = c.q[b, h * G * D:(h + 1) * G * D].double().view(G, D)
            ro, rl, a, s = attention(q, c.keys[b][:, h], c.values[b][:, h], torch.ones(G, n, dtype=torch.bool), c.scale)
            o_tol, lse_tol = attention_bounds(ro, rl, a, s, D, n, go.dtype, c.dtype)
            d = (go.double() - ro).abs() / (o_tol + 2.0 ** -20 * a)
            assert (d <= 1).all(), f"request {b} of {n} head {h}: o off by {d.max():.2f} of its bound"
            assert ((gl.double() - rl).abs() <= lse_tol + 2.0 ** -21).all(), f"request {b} of {n} head {h}"
    assert tpk.get_device_status(reset=True) == status


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [1, 31, 64, 97, 128, 700])
def test_one_row_tile(prefix, D, dtype):
    """Groups of few rows behind a wide table."""
    run([(prefix, [prefix + 3, prefix, prefix + 300, 0]), (300, [290, 310, 305])], 1, 20, D, dtype, max_pages=20000)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0])
def test_two_row_tiles(D, dtype, scale):
    """Many rows a group, several tiles; requests with less than the prefix."""
    run([(500, [400 + (i * 7) % 190 for i in range(70)]), (65, [66] * 3)], 2, 8, D, dtype, scale=scale, alone=(30,), o_gap=8)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prefixes(D):
    run([(6000, [6000 + (i * 77) % 500 for i in range(33)])], 1, 5, D, "bf16", max_pages=20000)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_few_rows(D, dtype):
    """One launch over prefixes and the rest."""
    run([(300, [350, 420, 301])], 2, 4, D, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("groups,H,G,wide", [([(300, [310] * 70)], 2, 8, None), ([(500, [600, 700, 520])], 1, 20, 20000)])
def test_waits_are_bounded(groups, H, G, wide, D):
    from test_gpu_paged_wait_limit import stalled
    stalled(Shared(groups, H, G, D, "bf16", max_pages=wide, f32=True))
