"""Cross attention of ragged queries to paged states, against the formula in 64 bits
(bounds in paged_util)."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import PAGE, Pages, attention, check_attention

pytestmark = pytest.mark.gpu


class Cross:
    def __init__(self, pg, nq, G, ranges=None, q_gap=0, o_gap=0, scale=0.0, lead=0, tail=0, mute=()):
        """lead, tail: query rows before the first and after the last request."""
        self.pg, self.nq, self.G, self.scale = pg, nq, G, scale or pg.D ** -0.5
        w = pg.H * G * pg.D
        self.off = [lead + sum(nq[:i]) for i in range(len(nq) + 1)]
        self.T = self.off[-1] + tail
        self.q = pg.randn(max(self.T, 1), w + q_gap)
        self.ranges = ranges
        self.mute = set(mute)
        table = pg.table.clone()
        for i, (b, p) in enumerate(mute):
            table[b, p] = [-1, pg.slots, 2 ** 31 - 1, -2 ** 31][i % 4]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.dq, self.table, self.lens, self.doff = self.q.cuda(), table.cuda(), i32(pg.lens), i32(self.off)
        self.k, self.v = pg.k.cuda(), pg.v.cuda()
        self.dr = None
        if ranges is not None:
            r = torch.full((max(self.T, 1), 2), 77, dtype=torch.int32)
            r[lead:self.off[-1]] = torch.tensor(ranges, dtype=torch.int32).view(-1, 2)
            self.dr = r.cuda()
        self.o = torch.full((max(self.T, 1), w + o_gap), float("nan"), dtype=pg.dtype, device="cuda")
        self.lse = torch.full((max(self.T, 1), pg.H * G), float("nan"), device="cuda")
        self.shape = tpk.PagedShape(pg.H, G, pg.D, dtype=tpk.BF16 if pg.dtype == torch.bfloat16 else tpk.F16,
                                    kv_slots=pg.slots, max_pages=pg.max_pages, sm_scale=scale)
        self.nbytes = tpk.cross_paged_workspace_bytes(self.shape, len(nq), self.T)
        self.ws = torch.full((self.nbytes,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        tpk.cross_attn_paged(self.shape, len(self.nq), self.T, self.dq, self.dq.stride(0), self.doff, self.k, self.v,
                             self.table, self.lens, self.dr, self.o, self.o.stride(0), self.lse, self.ws, self.nbytes,
                             stream=stream)

    def check(self, what=""):
        torch.cuda.synchronize()
        pg, G, D, H = self.pg, self.G, self.pg.D, self.pg.H
        w = H * G * D
        o, lse = self.o.cpu(), self.lse.cpu()
        for b, n in enumerate(pg.lens):
            i, e = self.off[b], self.off[b + 1]
            seen = torch.ones(e - i, n, dtype=torch.bool)
            if self.ranges is not None:
                at = torch.arange(n)
                r = torch.tensor(self.ranges).view(-1, 2)[i - self.off[0]:e - self.off[0]]
                seen = (at >= r[:, :1]) & (at < r[:, 1:])
            for bb, p in self.mute:
                if bb == b:
                    seen[:, p * PAGE:(p + 1) * PAGE] = False
            for j in range(H * G):
                h = j // G
                q = self.q[i:e, j * D:(j + 1) * D].double()
                want = attention(q, pg.keys[b][:, h], pg.values[b][:, h], seen, self.scale)
                check_attention(o[i:e, j * D:(j + 1) * D], lse[i:e, j], want, D, n, pg.dtype, one_plane=True,
                                what=f"{what} request {b} ({e - i} of {n}) head {j}")
        assert torch.isnan(o[:, w:]).all()
        for x in (o, lse):  # rows of no request are left as they were
            assert torch.isnan(x[:self.off[0]]).all() and torch.isnan(x[self.off[-1]:]).all()


def run(nq, lens, H, G, D, dtype, seed=0, status=(0, 0), max_pages=None, **kw):
    c = Cross(Pages(lens, H, D, dtype, seed, max_pages=max_pages), nq, G, **kw)
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == status
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8, 20])
def test_heads(G, D, dtype):
    run([5, 1, 0, 40], [100, 64, 30, 333], 2, G, D, dtype, seed=G)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,lens", [([1], [1]), ([1], [0]), ([0], [5]), ([300], [65]), ([127, 128, 129], [127, 128, 129]),
                                     ([700], [1000]), ([3, 260], [0, 2000]), ([513], [63])],
                         ids=lambda x: "-".join(map(str, x)))
def test_lengths(nq, lens, D):
    run(nq, lens, 1, 1, D, "bf16", seed=len(nq))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,nq", [(1, [150, 70]), (4, [90, 33]), (7, [40, 19])])
def test_ranges(D, G, nq):
    """Clips, a causal prompt, empty rows, ranges past the states' end."""
    lens = [700, 130]
    r = [(0, 0) if i < 5 else ((i * 4) // 64 * 64, (i * 4) // 64 * 64 + 64) for i in range(nq[0])]
    r += [(0, i + 1) if i % 7 else (200, 100) if i % 2 else (-50, 10 ** 6) for i in range(nq[1])]
    run(nq, lens, 1, G, D, "bf16", ranges=r)


@pytest.mark.parametrize("G", [1, 4])
def test_causal_prompt(G):
    run([333], [333], 2, G, 128, "bf16", ranges=[(0, i + 1) for i in range(333)])


def test_no_row_sees_anything():
    run([300], [500], 1, 2, 128, "bf16", ranges=[(9, 9)] * 300)


def test_strides_scale_and_untouched_rows():
    run([70, 200], [150, 600], 2, 2, 64, "f16", q_gap=16, o_gap=24, scale=0.4, lead=3, tail=9)
    run([70, 200], [150, 600], 2, 2, 256, "bf16", q_gap=8, o_gap=40, lead=1, tail=130, scale=-0.05)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores(D):
    run([200], [700], 1, 2, D, "bf16", scale=4.0)


def test_bad_pages_contribute_nothing():
    run([200, 4], [1000, 64], 2, 2, 128, "bf16", mute=[(0, 0), (0, 7), (0, 15), (1, 0)], status=(4, 1))


def test_bad_lengths_and_offsets_are_clamped():
    c = Cross(Pages([128, 100], 1, 64, "bf16", 3, max_pages=2), [150, 20], 1)
    c.lens.copy_(torch.tensor([10 ** 9, -4], dtype=torch.int32))
    c.doff.copy_(torch.tensor([-9, 150, 10 ** 9], dtype=torch.int32))
    c.pg.lens = [128, 0]
    c.pg.keys[1], c.pg.values[1] = c.pg.keys[1][:0], c.pg.values[1][:0]
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == (4, 1)


@pytest.mark.parametrize("n", [9, 300])
def test_extreme_ranges(n):
    """Range bounds at the ends of int32: cut to the states, empty where they cross."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    r = [[(lo, hi), (0, lo), (hi, hi), (lo, 5), (300, hi), (hi, lo), (lo, lo), (64, 65)][i % 8] for i in range(n)]
    run([n], [700], 1, 2, 128, "bf16", ranges=r)


def test_short_wait_limit_alone_changes_nothing():
    c = Cross(Pages([3000, 900], 2, 128, "bf16", 4), [400, 300], 2)
    tpk.set_test_wait(50_000_000, -1)
    try:
        c.call()
        c.check()
    finally:
        tpk.set_test_wait()
    assert tpk.get_device_status(reset=True) == (0, 0)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,lens,pages,G", [([1], [1], 5, 1), ([1], [0], 5, 3), ([0], [5], 5, 1), ([70], [250], 4, 8),
                                             ([4, 0, 1, 2], [300, 20, 0, 65], 8, 20), ([2], [3000], 47, 8),
                                             ([2, 3], [20000, 129], 313, 4), ([30], [20000], 313, 8)],
                         ids=lambda x: "-".join(map(str, x)) if isinstance(x, list) else str(x))
def test_few_rows(nq, lens, pages, G, D):
    """Tables wider than the lengths, on both sides of the choice of kernel."""
    run(nq, lens, 1, G, D, "f16", seed=G, max_pages=pages, lead=1, tail=2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,most,every,G", [(200, 700, 1, 1), (160, 130, 1, 8), (300, 90, 3, 3), (180, 400, 40, 1),
                                            (40, 2500, 1, 4)])
def test_rows_of_many_requests(n, most, every, G, D):
    """About a token a request, spread evenly or gathered in every third or fortieth."""
    run([every if i % every == 0 else 0 for i in range(n)], [(i * 37) % most for i in range(n)], 1, G, D, "bf16",
        seed=G, tail=3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,most,q,pages,G", [(128, 500, 3, 8, 1), (128, 60, 5, 1, 4), (7, 300, 30, 6, 3), (100, 2000, 2, 32, 4),
                                              (129, 400, 2, 7, 4), (3, 500, 70, 8, 2), (1, 64, 1, 1, 128)])
def test_runs_not_cut(n, most, q, pages, G, D):
    """A block per run: requests with no rows, no states, several runs."""
    run([(i * 5) % (q + 1) if n > 1 else q for i in range(n)], [(i * 37 + 64) % (most + 1) for i in range(n)], 1, G, D,
        "bf16", seed=q, lead=2, tail=5, max_pages=pages)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,H,G,q,pages", [(700, 1, 1, 33, None), (60, 4, 4, 9, 8)])
def test_sixteen_rows_of_many_requests(n, H, G, q, pages, D):
    run([(i * 7) % q for i in range(n)], [(i * 37) % 200 for i in range(n)], H, G, D, "f16", seed=2, max_pages=pages)


def test_rows_of_many_requests_see_ranges():
    r = [(0, 0) if i % 5 == 0 else (i % 200, i % 200 + 65) for i in range(170)]
    run([1] * 170, [(i * 37) % 300 for i in range(170)], 1, 2, 128, "bf16", ranges=r)


def test_few_rows_with_bad_pages():
    run([4, 3], [1000, 64], 1, 2, 128, "bf16", mute=[(0, 0), (0, 7), (0, 15), (1, 0)], status=(4, 1))


def test_no_queries():
    run([0, 0], [100, 5], 1, 1, 64, "bf16")


@pytest.mark.parametrize("n,most,queries", [(1000, 100, 5), (200, 250, 3), (100, 500, 2), (70, 600, 90), (65, 3000, 40)])
def test_many_requests(n, most, queries):
    """Row tiles and 16-row units, their requests sorted, numbered by a warp, by the block."""
    run([(i * 13) % queries for i in range(n)], [(i * 37) % most for i in range(n)], 1, 1, 64, "bf16", seed=9)


@pytest.mark.parametrize("nq", [[9, 5], [400, 300]])
def test_bit_identical_twice(nq):
    c = Cross(Pages([3000, 900], 2, 128, "bf16", 4), nq, 2)
    c.call()
    torch.cuda.synchronize()
    o, lse = c.o.clone(), c.lse.clone()
    c.ws.random_(0, 255)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), c.o.view(torch.int16)) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("nq", [[9, 5, 2], [300, 200, 100]])
def test_two_streams_and_capture(nq):
    a, b = Cross(Pages([900, 33, 64], 2, 128, "bf16", 5), nq, 2), Cross(Pages([64, 500, 0], 2, 128, "bf16", 6), nq, 2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.call(sa)
        b.call(sb)
    a.check("first stream")
    b.check("second stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=sa):
        a.call(torch.cuda.current_stream())
    lens = [100, 0, 64]
    a.pg.lens = lens
    a.pg.keys, a.pg.values = [k[:n] for k, n in zip(a.pg.keys, lens)], [v[:n] for v, n in zip(a.pg.values, lens)]
    a.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    a.o.fill_(float("nan"))
    g.replay()
    a.check("replayed with other lengths")


@pytest.mark.parametrize("nq,lens,pages,G", [([1], [100], 5, 2), ([300], [900], None, 2), ([4, 3], [1000, 64], None, 20),
                                             ([3, 2], [5000, 200], None, 4)],
                         ids=lambda x: "-".join(map(str, x)) if isinstance(x, list) else str(x))
def test_between_copies_forks_and_joins(nq, lens, pages, G):
    """A call waits for whatever is before it in its stream, and what follows waits for it: copies
    into its queries and over its results, calls of another stream, captured and not."""
    a, b, c = (Cross(Pages(lens, 1, 128, "bf16", i, max_pages=pages), nq, G) for i in (1, 2, 3))
    q, zero = c.dq.clone(), torch.zeros_like(c.dq)
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()

    def step(cur):
        a.call(cur)
        s2.wait_stream(cur)
        b.call(s2)
        a.call(cur)
        cur.wait_stream(s2)
        c.dq.copy_(q)
        c.call(cur)
        c.o.zero_()
        c.o[:, c.pg.H * G * 128:] = float("nan")
        c.call(cur)
        c.dq.copy_(zero)

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(10):
            step(s)
    for x in (a, b, c):
        x.check("eager")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(torch.cuda.current_stream())
    for x in (a, b, c):
        x.o.fill_(float("nan"))
        x.lse.fill_(float("nan"))
    for _ in range(3):
        g.replay()
    for x in (a, b, c):
        x.check("captured")
    assert tpk.get_device_status(reset=True) == (0, 0)
