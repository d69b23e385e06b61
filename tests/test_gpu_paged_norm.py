"""The rotary store with norms of the heads against its formula in 64 bits.

Bound, with (a, b) a pair of normed channels: finfo.eps / 2 of the result (its rounding),
2^-20 (|a| + |b|) for the rotation (its own test has the count), and the norm's: the sum of
squares is 16 float32 steps in a thread and at most 4 between threads, all of one sign, so
20 * 2^-24, of which the root takes half; mean and eps 2 * 2^-25; rsqrtf 2^-22; three products
3 * 2^-24: 18 * 2^-24 < 2^-19 of |a| + |b|.  Together below 2^-18 (|a| + |b|); channels that are
not rotated have themselves in its place."""
import numpy as np
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import DTYPES
from test_gpu_paged_rope import rotated

pytestmark = pytest.mark.gpu


def normed(x, w, eps):
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return y if w is None else y * w.double()


def check(got, x, w, eps, pos, axis, freq, pairs, dtype):
    y = normed(x, w, eps)
    want, s = rotated(y, pos, axis, freq, pairs)
    s[..., 2 * len(axis):] = y[..., 2 * len(axis):].abs()
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -18 * s + torch.finfo(dtype).tiny
    d = (got - want).abs()[fine]
    assert (d <= tol[fine]).all(), f"off by {(d / tol[fine]).max():.2f} of the bound"


def case(T, H, G, D, rot, pairs, dtype, seed=0, pad=0, axes=1, far=1000, gap=0, weights=(True, True), eps=1e-6,
         in_place=False, q_only=False, store_only=False, change=None, runner=None):
    gen = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    w = (H * G + 2 * H) * D + gap
    x = torch.randn(T, w, generator=gen) * torch.exp(2 * torch.randn(T, 1, generator=gen))
    if change:
        change(x)
    qkv = x.to(dt)
    slots = -(-T // 64) + 2
    pool = torch.randn(2, slots, H, 64, D, generator=gen).to(dt)
    slot = torch.randperm(slots * 64, generator=gen)[:T]
    live = torch.ones(T, dtype=torch.bool)
    live[torch.randperm(T, generator=gen)[:pad]] = False
    slot = torch.where(live, slot, torch.full_like(slot, -1))
    pos = torch.randint(-far, far + 1, (axes, T), generator=gen, dtype=torch.int32)
    freq = torch.tensor([1e4 ** (-2 * j / max(rot, 1)) for j in range(rot // 2)], dtype=torch.float32)
    axis = np.array([j % axes for j in range(rot // 2)], np.uint8)
    wq, wk = ((torch.randn(D, generator=gen) + 1).to(dt) if on else None for on in weights)
    out = torch.randn(T, H * G * D + gap, generator=gen).to(dt)
    d = qkv.cuda()
    dq, dk, dv = d[:, :H * G * D], d[:, H * G * D:(H * G + H) * D], d[:, (H * G + H) * D:]
    dp, do = pool.cuda(), dq if in_place else out.cuda()
    s = tpk.PagedShape(H, G, D, dtype=tpk.BF16 if dtype == "bf16" else tpk.F16, kv_slots=slots)
    dev = [None if t is None else t.cuda() for t in (wq, wk, pos if rot else None, freq if rot else None, None if q_only else slot)]

    def call():
        tpk.kv_norm_rope_append(s, T, None if store_only else dq, w, None if q_only else dk, w, None if q_only else dv, w, dev[0],
                                dev[1], eps, dev[2], axes, axis if axes > 1 else None, dev[3], rot, pairs, dev[4],
                                None if store_only else do, do.stride(0), None if q_only else dp[0], None if q_only else dp[1],
                                stream=torch.cuda.current_stream())

    (runner or (lambda f: f()))(call)
    torch.cuda.synchronize()
    assert tpk.get_device_status(reset=True) == (0, 0)
    x = qkv.double()
    q, k, v = (x[:, :H * G * D].view(T, H * G, D), x[:, H * G * D:(H * G + H) * D].view(T, H, D),
               qkv[:, (H * G + H) * D:(H * G + 2 * H) * D].view(T, H, D))
    if q_only:
        live[:] = True
    if not store_only:
        got = do[:, :H * G * D].cpu().view(T, H * G, D)
        check(got[live], q[live], wq, eps, pos[:, live], axis, freq, pairs, dt)
        assert torch.equal(got[~live], (qkv if in_place else out)[:, :H * G * D].view(T, H * G, D)[~live])
        if gap and not in_place:
            assert torch.equal(do[:, H * G * D:].cpu(), out[:, H * G * D:])
    at, row = slot[live] // 64, slot[live] % 64
    gk, gv = dp.cpu()
    if not q_only:
        check(gk[at, :, row], k[live], wk, eps, pos[:, live], axis, freq, pairs, dt)
        assert torch.equal(gv[at, :, row].view(torch.int16), v[live].view(torch.int16))  # bit for bit, NaN too
        pool[0][at, :, row], pool[1][at, :, row] = gk[at, :, row], gv[at, :, row]
    assert torch.equal(gk.view(torch.int16), pool[0].view(torch.int16))  # what is not a token's row is as it was
    assert torch.equal(gv.view(torch.int16), pool[1].view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 0), (256, 144)])
def test_heads_and_pairs(D, rot, pairs, dtype):
    case(37, 2, 3, D, rot, pairs, dtype, seed=D + rot, pad=5, axes=3, gap=8)


@pytest.mark.parametrize("T", [1, 2, 63, 305, 700, 2500])
def test_lengths(T):
    case(T, 4, 8 if T < 1000 else 1, 128, 128, False, "bf16", seed=T, pad=T // 7)


@pytest.mark.parametrize("H,G", [(1, 1), (1, 71), (12, 1), (3, 5), (40, 2)])
def test_head_layouts(H, G):
    """Also where a block's last warp is not full."""
    case(9, H, G, 64, 64, False, "f16", seed=H, gap=24, axes=4)


@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
def test_without_factors(weights):
    case(30, 2, 4, 128, 64, True, "bf16", weights=weights)


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-5, 3.0, 1e30])
def test_eps(eps):
    case(30, 2, 4, 128, 128, False, "bf16", eps=eps)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size,eps", [(1e25, 1e-6), (1e36, 1e-6), (1e-25, 0.0), (1e-36, 0.0), (1e-30, 1e-6), (1e-15, 1e-32)])
def test_squares_out_of_range(D, size, eps):
    """bfloat16 heads whose squares float32 does not hold, beside ordinary ones."""
    def change(x):
        x[::3] *= size / x[::3].abs().amax(1, keepdim=True)
    case(20, 1, 3, D, D, False, "bf16", eps=eps, change=change)


def test_zero_infinite_and_nan_heads():
    """Each head for itself: the others' results are the formula's.  Rows whose pairs meet an
    infinity are left to the formula too (NaN)."""
    D = 64

    def change(x):
        x[1, :D] = 0                    # a head of zeros stays zero
        x[2, 3] = float("nan")          # one NaN: its head
        x[3, 2 * D + 5] = float("nan")
        x[4, D:2 * D] = 0
    case(8, 1, 2, D, D, False, "f16", change=change)
    case(8, 1, 2, D, 0, False, "bf16", change=change)

    def infinite(x):
        x[2, 3] = float("inf")
    case(8, 1, 2, D, 0, False, "bf16", change=infinite)  # 0 beside NaN


def test_in_place_query_only_store_only():
    case(50, 2, 4, 128, 64, True, "bf16", in_place=True, pad=4, axes=3)
    case(50, 2, 4, 128, 128, False, "f16", q_only=True)
    case(50, 2, 4, 128, 128, False, "bf16", store_only=True, pad=3, axes=2)
    case(50, 1, 1, 256, 0, False, "bf16", store_only=True)


def test_far_positions():
    case(64, 2, 2, 128, 128, False, "f16", far=(1 << 31) - 1, axes=2)


def test_other_stream_and_captured():
    def on_stream(call):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            call()

    def captured(call):
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        g.replay()
        g.replay()

    case(40, 2, 2, 64, 64, False, "bf16", runner=on_stream)
    case(40, 2, 2, 64, 64, False, "bf16", runner=captured)


def test_bad_slots_are_skipped():
    s = tpk.PagedShape(1, 1, 64, kv_slots=2)
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    pools = torch.zeros(2, 3, 1, 64, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([5, 128, -1, 1 << 40], dtype=torch.int64, device="cuda")
    tpk.kv_norm_rope_append(s, 4, x, 64, x, 64, x, 64, None, None, 0.0, None, 1, None, None, 0, False, slot, out, 64, pools[0],
                            pools[1])
    torch.cuda.synchronize()
    assert tpk.get_device_status(reset=True) == (4, 1)
    assert pools.sum().item() == 2 * 64 and pools[:, 0, 0, 5].sum().item() == 2 * 64
    assert out.sum(1).tolist() == [64, 0, 0, 0]
