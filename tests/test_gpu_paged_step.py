"""The calls together as a serving step uses them: tables from lengths, rotary store,
decode, and cross attention to an encoder's states, captured once and replayed while
requests grow, finish and start."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import PAGE, attention, check_attention
from test_gpu_paged_rope import rotated

pytestmark = pytest.mark.gpu


def test_replayed_steps_of_a_growing_batch():
    H, G, D, n, max_pages, slots, cap = 2, 4, 128, 4, 8, 24, 200
    dt, dev = torch.bfloat16, "cuda"
    gen = torch.Generator().manual_seed(1)
    shape = tpk.PagedShape(H, G, D, kv_slots=slots, max_pages=max_pages)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    kp = torch.full((slots, H, PAGE, D), float("nan"), dtype=dt, device=dev)
    vp = kp.clone()
    lens, new, table = i32(n), i32(n), i32(n, max_pages)
    free = torch.arange(slots, dtype=torch.int32, device=dev)
    n_free = torch.tensor([slots], dtype=torch.int32, device=dev)
    granted, off = i32(n), i32(n + 1)
    slot = torch.zeros(cap, dtype=torch.int64, device=dev)
    pos, req, causal = i32(cap), i32(cap), i32(cap, 2)
    w = (H * G + 2 * H) * D
    qkv = torch.zeros(cap, w, dtype=dt, device=dev)
    q_out = torch.zeros(cap, H * G, D, dtype=dt, device=dev)
    freq = torch.tensor([1e4 ** (-2 * j / D) for j in range(D // 2)], dtype=torch.float32, device=dev)
    o = torch.zeros(cap, H * G, D, dtype=dt, device=dev)
    lse = torch.zeros(cap, H * G, device=dev)
    nbytes = tpk.cross_paged_workspace_bytes(shape, n, cap)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)

    def step():
        st = torch.cuda.current_stream()
        tpk.kv_tables_update(n, max_pages, lens, new, table, free, slots, n_free, n_free, lens, granted, off, slot, pos,
                             req, cap, stream=st)
        tpk.kv_rope_append(shape, cap, qkv, w, qkv[:, H * G * D:], w, qkv[:, (H * G + H) * D:], w, pos, 1, None, freq, D,
                           False, slot, q_out, H * G * D, kp, vp, stream=st)
        causal[:, 1] = pos + 1  # a new token sees its request up to itself
        tpk.cross_attn_paged(shape, n, cap, q_out, H * G * D, off, kp, vp, table, lens, causal, o, H * G * D, lse, ws,
                             nbytes, stream=st)

    step()  # the device's first calls, nothing to do
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # host model: each request's rotated keys and values so far
    hist = [(torch.zeros(0, H, D, dtype=torch.float64), torch.zeros(0, H, D, dtype=torch.float64)) for _ in range(n)]
    plan = [[70, 3, 0, 64], [71, 4, 10, 65], [72, 0, 11, 66], [73, 130, 11, 0], [74, 131, 12, 5], [140, 132, 13, 6]]
    for want in plan:
        old = [k.shape[0] for k, _ in hist]
        grow = [max(0, b - a) for a, b in zip(old, want)]
        x = torch.randn(cap, w, generator=gen).to(dt)
        qkv.copy_(x)
        new.copy_(torch.tensor(want, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert granted.tolist() == [1] * n and lens.tolist() == want
        at = 0
        for b in range(n):
            rows = slice(at, at + grow[b])
            at += grow[b]
            p = torch.arange(old[b], old[b] + grow[b])[None]
            xq = x[rows, :H * G * D].double().view(grow[b], H * G, D)
            xk = x[rows, H * G * D:(H * G + H) * D].double().view(grow[b], H, D)
            xv = x[rows, (H * G + H) * D:].double().view(grow[b], H, D)
            zero = [0] * (D // 2)
            q = rotated(xq, p, zero, freq.cpu(), False)[0].to(dt).double()
            k = rotated(xk, p, zero, freq.cpu(), False)[0].to(dt).double()
            # a half step of rounding may go either way: take the device's own values,
            # each within one step of the formula's
            got_q = q_out[rows].cpu().double()
            assert ((got_q - q).abs() <= torch.finfo(dt).eps * q.abs() + 1e-6).all()
            got_k = torch.empty_like(k)
            for i in range(grow[b]):
                t = old[b] + i
                s = int(table[b, t // PAGE])
                got_k[i] = kp[s, :, t % PAGE].cpu().double()
                assert torch.equal(vp[s, :, t % PAGE].cpu().double(), xv[i])
            assert ((got_k - k).abs() <= torch.finfo(dt).eps * k.abs() + 1e-6).all()
            keys, values = hist[b][0][:want[b]], hist[b][1][:want[b]]
            hist[b] = (torch.cat([keys, got_k]), torch.cat([values, xv]))
            seen = torch.arange(want[b]) < (torch.arange(old[b], old[b] + grow[b]) + 1)[:, None]
            for j in range(H * G):
                ref = attention(got_q[:, j], hist[b][0][:, j // G], hist[b][1][:, j // G], seen, D ** -0.5)
                check_attention(o[rows, j].cpu(), lse[rows, j].cpu(), ref, D, max(want), dt, one_plane=True,
                                what=f"request {b} head {j} at {want[b]}")
        used = sum(-(-c // PAGE) for c in want)
        assert n_free.item() == slots - used
        assert sorted(set(free[:n_free.item()].tolist()) | {int(table[b, i]) for b in range(n)
                                                            for i in range(-(-want[b] // PAGE))}) == list(range(slots))
        # the last new token of each request again, by the single-token call
        if all(g > 0 for g in grow):
            q1 = torch.stack([q_out[sum(grow[:b + 1]) - 1] for b in range(n)]).contiguous()
            o1, l1 = torch.zeros(n, H * G, D, dtype=dt, device=dev), torch.zeros(n, H * G, device=dev)
            nb = tpk.decode_paged_workspace_bytes(shape, n)
            ws1 = torch.empty(nb, dtype=torch.uint8, device=dev)
            tpk.decode_attn_paged(shape, n, q1, H * G * D, kp, vp, table, lens, None, o1, H * G * D, False, l1, ws1, nb)
            torch.cuda.synchronize()
            for b in range(n):
                for j in range(H * G):
                    k, v = hist[b]
                    ref = attention(q1[b, j:j + 1].cpu().double(), k[:, j // G], v[:, j // G],
                                    torch.ones(1, k.shape[0], dtype=torch.bool), D ** -0.5)
                    check_attention(o1[b, j:j + 1].cpu(), l1[b, j:j + 1].cpu(), ref, D, k.shape[0], dt)
    assert tpk.get_device_status(reset=True) == (0, 0)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements, the history in its last slots: stored there by
    the rotary call, read back by both attention calls."""
    H, G, D, n = 4, 2, 256, 150
    slots = 2 ** 32 // (H * PAGE * D) + 8
    dt = torch.bfloat16
    kp, vp = (torch.empty(slots, H, PAGE, D, dtype=dt, device="cuda") for _ in range(2))
    shape = tpk.PagedShape(H, G, D, kv_slots=slots, max_pages=12)
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(2, n, H, D, generator=gen).to(dt)
    table = torch.full((1, 12), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor([slots - 1, slots - 3, slots - 2])
    t = torch.arange(n)
    slot = table[0, t // PAGE].long() * PAGE + t % PAGE
    d = x.cuda()
    tpk.kv_rope_append(shape, n, None, 0, d[0], H * D, d[1], H * D, None, 1, None, None, 0, False, slot.cuda(), None, 0, kp, vp)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ref = x.double()
    for nq in (1, 200):
        q = torch.randn(nq, H * G, D, generator=gen).to(dt)
        o, lse = torch.zeros(nq, H * G, D, dtype=dt, device="cuda"), torch.zeros(nq, H * G, device="cuda")
        w = H * G * D
        if nq == 1:
            nb = tpk.decode_paged_workspace_bytes(shape, 1)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            tpk.decode_attn_paged(shape, 1, q.cuda(), w, kp, vp, table.cuda(), lens, None, o, w, False, lse, ws, nb)
        else:
            nb = tpk.cross_paged_workspace_bytes(shape, 1, nq)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            off = torch.tensor([0, nq], dtype=torch.int32, device="cuda")
            tpk.cross_attn_paged(shape, 1, nq, q.cuda(), w, off, kp, vp, table.cuda(), lens, None, o, w, lse, ws, nb)
        torch.cuda.synchronize()
        for j in range(H * G):
            want = attention(q[:, j].double(), ref[0, :, j // G], ref[1, :, j // G], torch.ones(nq, n, dtype=torch.bool), D ** -0.5)
            check_attention(o[:, j].cpu(), lse[:, j].cpu(), want, D, n, dt, one_plane=True, what=f"{nq} queries head {j}")
    assert tpk.get_device_status(reset=True) == (0, 0)
