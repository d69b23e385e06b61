"""The rotary store against its formula in 64 bits.

Bound, with (a, b) a pair: finfo.eps / 2 of the result (its rounding) plus
2^-20 (|a| + |b|): the angle is off by at most 2^-32 turns and its float32 form by
2^-24 of half a turn (under 2^-22 rad together), sincospif by 2^-22, and three float32
roundings of products and sums, 2^-23 of |a| + |b|."""
import numpy as np
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import DTYPES

pytestmark = pytest.mark.gpu


def rotated(x, pos, axis, freq, pairs):
    """x [T, heads, D] double -> (rotated, |a| + |b| of each channel's pair)."""
    rot = 2 * len(axis)
    y, s = x.clone(), torch.zeros_like(x)
    if rot == 0:
        return y, s
    angle = pos.double()[torch.tensor(axis, dtype=torch.long)].T * freq.double()
    c, n = angle.cos()[:, None], angle.sin()[:, None]
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * n, b * c + a * n
    s[..., lo] = s[..., hi] = a.abs() + b.abs()
    return y, s


def close(got, want, s, dtype):
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -20 * s + torch.finfo(dtype).tiny
    d = (got.double() - want).abs()
    assert (d <= tol).all(), f"off by {(d / tol).max():.2f} of the bound"


def case(T, H, G, D, rot, axes, pairs, dtype, seed=0, pad=0, far=1000, gap=0, base=1e6, in_place=False, q_only=False,
         store_only=False, stream=None):
    gen = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    w = (H * G + 2 * H) * D + gap
    qkv = torch.randn(T, w, generator=gen).to(dt)
    slots = -(-T // 64) + 2
    pool = torch.randn(2, slots, H, 64, D, generator=gen).to(dt)
    perm = torch.randperm(slots * 64, generator=gen)[:T]
    live = torch.ones(T, dtype=torch.bool)
    live[torch.randperm(T, generator=gen)[:pad]] = False
    slot = torch.where(live, perm, torch.full_like(perm, -1))
    pos = torch.randint(-far, far + 1, (axes, T), generator=gen, dtype=torch.int32)
    freq = torch.tensor([base ** (-2 * j / max(rot, 1)) for j in range(rot // 2)], dtype=torch.float32)
    axis = np.array([j % axes for j in range(rot // 2)], np.uint8)
    out = torch.randn(T, H * G * D + gap, generator=gen).to(dt)
    d = qkv.cuda()
    dq, dk, dv = d[:, :H * G * D], d[:, H * G * D:(H * G + H) * D], d[:, (H * G + H) * D:]
    dp, do = pool.cuda(), dq if in_place else out.cuda()
    s = tpk.PagedShape(H, G, D, dtype=tpk.BF16 if dtype == "bf16" else tpk.F16, kv_slots=slots)
    tpk.kv_rope_append(s, T, None if store_only else dq, w, None if q_only else dk, w, None if q_only else dv, w,
                       pos.cuda() if rot else None, axes, axis if axes > 1 else None, freq.cuda() if rot else None, rot,
                       pairs, None if q_only else slot.cuda(), None if store_only else do, do.stride(0),
                       None if q_only else dp[0], None if q_only else dp[1], stream=stream)
    torch.cuda.synchronize()
    assert tpk.get_device_status(reset=True) == (0, 0)
    x = qkv.double()
    q, k, v = (x[:, :H * G * D].view(T, H * G, D), x[:, H * G * D:(H * G + H) * D].view(T, H, D),
               x[:, (H * G + H) * D:(H * G + 2 * H) * D].view(T, H, D))
    if q_only:
        live[:] = True
    if not store_only:
        before = (qkv if in_place else out)[:, :H * G * D].double().view(T, H * G, D)
        y, sq = rotated(q, pos, axis, freq, pairs)
        got = do[:, :H * G * D].cpu().view(T, H * G, D)
        close(got[live], y[live], sq[live], dt)
        assert torch.equal(got[~live].double(), before[~live])
        if gap and not in_place:
            assert torch.equal(do[:, H * G * D:].cpu(), out[:, H * G * D:])
    want_k, want_v, scale = pool[0].double(), pool[1].double(), torch.zeros(slots, H, 64, D, dtype=torch.float64)
    if not q_only:
        y, sk = rotated(k, pos, axis, freq, pairs)
        at, row = slot[live] // 64, slot[live] % 64
        want_k[at, :, row], want_v[at, :, row], scale[at, :, row] = y[live], v[live], sk[live]
    close(dp[0].cpu(), want_k, scale, dt)
    assert torch.equal(dp[1].cpu().double(), want_v)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 0)])
def test_heads_and_pairs(D, rot, pairs, dtype):
    case(37, 2, 3, D, rot, 3, pairs, dtype, seed=D + rot, pad=5, gap=8)


@pytest.mark.parametrize("T", [1, 2, 63, 305, 700, 2500])
def test_lengths(T):
    case(T, 4, 8 if T < 1000 else 1, 128, 128, 1, False, "bf16", seed=T, pad=T // 7)


@pytest.mark.parametrize("H,G", [(1, 1), (1, 71), (12, 1), (3, 5), (40, 2)])
def test_head_layouts(H, G):
    case(9, H, G, 64, 64, 4, False, "f16", seed=H, gap=24)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    """Positions where a float32 product of position and frequency says nothing."""
    case(64, 2, 2, 128, 128, 2, False, "f16", seed=5, far=far)


def test_in_place_query_only_store_only():
    case(50, 2, 4, 128, 64, 3, True, "bf16", in_place=True, pad=4)
    case(50, 2, 4, 128, 128, 1, False, "f16", q_only=True)
    case(50, 2, 4, 128, 128, 2, False, "bf16", store_only=True, pad=3)
    case(50, 1, 1, 256, 0, 1, False, "bf16", store_only=True)


def test_bad_slots_are_skipped():
    """Slots at and past the pool's end write nothing and set the status bit."""
    s = tpk.PagedShape(1, 1, 64, kv_slots=2)
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    pools = torch.zeros(2, 3, 1, 64, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([5, 128, -1, 1 << 40], dtype=torch.int64, device="cuda")
    tpk.kv_rope_append(s, 4, x, 64, x, 64, x, 64, None, 1, None, None, 0, False, slot, out, 64, pools[0], pools[1])
    torch.cuda.synchronize()
    assert tpk.get_device_status(reset=True) == (4, 1)
    assert pools.sum().item() == 2 * 64 and pools[:, 0, 0, 5].sum().item() == 2 * 64
    assert out.sum(1).tolist() == [64, 0, 0, 0]


def test_zero_tokens_and_other_stream():
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        case(20, 2, 2, 64, 64, 1, False, "bf16", stream=st)
    s = tpk.PagedShape(1, 1, 64, kv_slots=2)
    tpk.kv_rope_append(s, 0, 16, 64, 16, 64, 16, 64, None, 1, None, None, 0, False, 16, 16, 64, 16, 16)
