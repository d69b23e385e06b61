"""The documented loop captured as it stands: tables from lengths, the store, and both
attention calls on what those have just written, replayed without a pause while every
request grows, shrinks, finishes and starts.  The joins of cut histories and of split
keys follow the lengths of their own replay, never of one before."""
import random

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import PAGE, attention, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,H,G,D,most,grow,cap,steps", [(3, 2, 4, 128, 2300, 280, 900, 8), (2, 1, 12, 256, 2400, 300, 640, 6),
                                                         (140, 1, 2, 64, 260, 9, 800, 6), (1, 4, 8, 64, 2500, 400, 400, 7)])
def test_captured_loop(n, H, G, D, most, grow, cap, steps):
    dt, dev, max_pages = torch.bfloat16, "cuda", 40  # wide enough for every history to be cut
    rng, gen = random.Random(n), torch.Generator().manual_seed(n)
    slots = n * (-(-most // PAGE)) + 2
    w = H * G * D
    shape = tpk.PagedShape(H, G, D, kv_slots=slots, max_pages=max_pages)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    kp, vp = (torch.full((slots, H, PAGE, D), float("nan"), dtype=dt, device=dev) for _ in range(2))
    lens, new, table, granted, off = i32(n), i32(n), i32(n, max_pages), i32(n), i32(n + 1)
    free, n_free = torch.arange(slots, dtype=torch.int32, device=dev), i32(1) + slots
    slot, pos, req = torch.zeros(cap, dtype=torch.int64, device=dev), i32(cap), i32(cap)
    q1, q, k, v = (torch.zeros(r, c, dtype=dt, device=dev) for r, c in [(n, w), (cap, w), (cap, H * D), (cap, H * D)])
    o1, l1, o, lse = (torch.zeros(s, dtype=t, device=dev) for s, t in [((n, w), dt), ((n, H * G), torch.float32), ((cap, w), dt),
                                                                      ((cap, H * G), torch.float32)])
    sizes = tpk.decode_paged_workspace_bytes(shape, n), tpk.cross_paged_workspace_bytes(shape, n, cap)
    ws = [torch.full((b,), 0xFF, dtype=torch.uint8, device=dev) for b in sizes]

    def step():
        st = torch.cuda.current_stream()
        tpk.kv_tables_update(n, max_pages, lens, new, table, free, slots, n_free, n_free, lens, granted, off, slot, pos,
                             req, cap, stream=st)
        tpk.kv_rope_append(shape, cap, None, 0, k, H * D, v, H * D, None, 1, None, None, 0, False, slot, None, 0, kp, vp,
                           stream=st)
        tpk.decode_attn_paged(shape, n, q1, w, kp, vp, table, lens, None, o1, w, False, l1, ws[0], sizes[0], stream=st)
        tpk.cross_attn_paged(shape, n, cap, q, w, off, kp, vp, table, lens, None, o, w, lse, ws[1], sizes[1], stream=st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # the plan: every length changes at every step, the tokens fit
    plan, now = [], [0] * n
    for i in range(steps):
        want = []
        for b in range(n):
            x = now[b] + rng.randint(1, grow)
            if i and rng.random() < 0.3:
                x = rng.choice([0, rng.randint(0, now[b]), 1])
            want.append(x if 0 <= x <= most and x != now[b] else now[b] + 1)
        plan.append(want)
        now = want
    data = [[torch.randn(x.shape, generator=gen).to(dt) for x in (q1, q, k, v)] for _ in range(steps)]
    sent = [[x.to(dev) for x in d] for d in data]
    news = torch.tensor(plan, dtype=torch.int32).to(dev)
    outs = [[torch.zeros_like(x) for x in (o1, l1, o, lse, granted, lens)] for _ in range(steps)]
    torch.cuda.synchronize()
    for i in range(steps):
        for x, y in zip((q1, q, k, v, new), sent[i] + [news[i]]):
            x.copy_(y)
        graph.replay()
        for x, y in zip(outs[i], (o1, l1, o, lse, granted, lens)):
            x.copy_(y)
    torch.cuda.synchronize()
    assert tpk.get_device_status(reset=True) == (0, 0)
    hist = [(torch.zeros(0, H, D, dtype=torch.float64), torch.zeros(0, H, D, dtype=torch.float64)) for _ in range(n)]
    for i, want in enumerate(plan):
        g1, gl1, g, gl, gr, ln = (x.cpu() for x in outs[i])
        assert gr.tolist() == [1] * n and ln.tolist() == want
        xq1, xq, xk, xv = (x.double() for x in data[i])
        at = 0
        for b in range(n):
            add = max(0, want[b] - hist[b][0].shape[0])
            rows = slice(at, at + add)
            at += add
            hist[b] = tuple(torch.cat([h[:want[b]], x[rows].view(add, H, D)]) for h, x in zip(hist[b], (xk, xv)))
            for j in range(H * G):
                keys, values = (x[:, j // G] for x in hist[b])
                c = slice(j * D, (j + 1) * D)
                ones = torch.ones(1 + add, want[b], dtype=torch.bool)
                ref = attention(torch.cat([xq1[b:b + 1, c], xq[rows, c]]), keys, values, ones, D ** -0.5)
                what = f"step {i} request {b} ({want[b]} tokens, {add} new) head {j}"
                check_attention(g1[b:b + 1, c], gl1[b:b + 1, j], [x[:1] for x in ref], D, want[b], dt, what="decode " + what)
                if add:
                    check_attention(g[rows, c], gl[rows, j], [x[1:] for x in ref], D, want[b], dt, one_plane=True,
                                    what="cross " + what)
        assert at <= cap
