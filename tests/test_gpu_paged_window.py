"""Attention through windows whose first tokens stay visible, against the formula in 64 bits
(bounds in paged_util).  Pages without a visible token hold NaN, and their table entries are
out of the pool: a stray read shows up in the result or in the device status."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import PAGE, Pages, attention, check_attention
from test_gpu_paged_wait_limit import stalled

pytestmark = pytest.mark.gpu


def seen_by(c, n, window, sinks):
    """[c, n]: what the last c of n tokens see."""
    t, x = torch.arange(n), (n - c + torch.arange(c))[:, None]
    near = (t <= x) & (t > x - window) if window else t <= x
    return near | ((t <= x) & (t < sinks))


class Window:
    """nq None: one query token per request, without offsets."""

    def __init__(self, pg, nq, G, window, sinks, q_gap=0, o_gap=0, scale=0.0, lead=0, tail=0, mute=()):
        self.pg, self.G, self.scale, self.window, self.sinks = pg, G, scale or pg.D ** -0.5, window, sinks
        self.decode = nq is None
        self.nq = nq = [1] * len(pg.lens) if nq is None else nq
        w = pg.H * G * pg.D
        self.off = [lead + sum(nq[:i]) for i in range(len(nq) + 1)]
        self.T = self.off[-1] + tail
        self.q = pg.randn(max(self.T, 1), w + q_gap)
        self.seen = [seen_by(c, n, window, sinks) for c, n in zip(nq, pg.lens)]
        table = pg.table.clone()
        self.k, self.v = pg.k.cuda(), pg.v.cuda()
        for b, n in enumerate(pg.lens):
            for i in range(-(-n // PAGE)):
                if not self.seen[b][:, i * PAGE:(i + 1) * PAGE].any():
                    self.k[table[b, i]] = self.v[table[b, i]] = float("nan")
                    table[b, i] = [-1, 2 ** 31 - 1, -2 ** 31][i % 3]
        for i, (b, p) in enumerate(mute):
            table[b, p] = [-1, pg.slots, 2 ** 31 - 1, -2 ** 31][i % 4]
            self.seen[b][:, p * PAGE:(p + 1) * PAGE] = False
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.dq, self.table, self.lens, self.doff = self.q.cuda(), table.cuda(), i32(pg.lens), i32(self.off)
        self.o = torch.full((max(self.T, 1), w + o_gap), float("nan"), dtype=pg.dtype, device="cuda")
        self.lse = torch.full((max(self.T, 1), pg.H * G), float("nan"), device="cuda")
        self.shape = tpk.PagedShape(pg.H, G, pg.D, dtype=tpk.BF16 if pg.dtype == torch.bfloat16 else tpk.F16,
                                    kv_slots=pg.slots, max_pages=pg.max_pages, sm_scale=scale)
        self.nbytes = tpk.window_paged_workspace_bytes(self.shape, len(nq), self.T)
        self.ws = torch.full((self.nbytes,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        tpk.window_attn_paged(self.shape, len(self.nq), self.T, self.window, self.sinks, self.dq, self.dq.stride(0),
                              None if self.decode else self.doff, self.k, self.v, self.table, self.lens, self.o,
                              self.o.stride(0), self.lse, self.ws, self.nbytes, stream=stream)

    def check(self, what=""):
        torch.cuda.synchronize()
        pg, G, D, H = self.pg, self.G, self.pg.D, self.pg.H
        w = H * G * D
        o, lse = self.o.cpu(), self.lse.cpu()
        for b, n in enumerate(pg.lens):
            i, e = self.off[b], self.off[b + 1]
            for j in range(H * G):
                q = self.q[i:e, j * D:(j + 1) * D].double()
                want = attention(q, pg.keys[b][:, j // G], pg.values[b][:, j // G], self.seen[b], self.scale)
                check_attention(o[i:e, j * D:(j + 1) * D], lse[i:e, j], want, D, n, pg.dtype, one_plane=not self.decode,
                                what=f"{what} request {b} ({e - i} of {n}) head {j}")
        assert torch.isnan(o[:, w:]).all()
        for x in (o, lse):  # rows of no request are left as they were
            assert torch.isnan(x[:self.off[0]]).all() and torch.isnan(x[self.off[-1]:]).all()


def run(nq, lens, H, G, D, dtype, window, sinks, seed=0, status=(0, 0), max_pages=None, **kw):
    c = Window(Pages(lens, H, D, dtype, seed, max_pages=max_pages), nq, G, window, sinks, **kw)
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == status
    return c


WINDOWS = [(1, 0), (1, 1), (63, 4), (64, 64), (65, 65), (100, 130), (200, 20), (0, 0), (0, 7), (1000, 4), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_token_each(D, window, sinks):
    run(None, [700, 0, 1, 64, 65, 129, 333, 20], 2, 4, D, "bf16", window, sinks, seed=window % 100)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts(D, window, sinks):
    """Whole prompts, later parts, a query or two; many rows and few."""
    run([300, 120, 1, 0, 40], [300, 700, 400, 50, 64], 2, 2, D, "f16", window, sinks, seed=sinks % 100)


@pytest.mark.parametrize("window,sinks", [(150, 4), (64, 70), (0, 0), (9, 300)])
@pytest.mark.parametrize("nq", [[3, 1, 2], [16, 9, 0]])
def test_few_query_tokens(nq, window, sinks):
    """Drafts to be verified: the split kernel's runs, in one piece and cut."""
    run(nq, [2000, 77, 640], 2, 2, 128, "bf16", window, sinks)
    run(nq, [200, 77, 130], 1, 1, 64, "f16", window, sinks)
    run(nq, [2000, 300, 640], 1, 3, 256, "bf16", window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G", [1, 3, 8, 20, 128])
def test_heads(G, dtype):
    run(None, [500, 130], 2, G, 64, dtype, 90, 5, seed=G)
    run([70, 30], [500, 130], 1, G, 128, dtype, 90, 5, seed=G)
    run([40, 3], [300, 130], 1, G, 256, dtype, 50, 66, seed=G)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_before_the_first_token(D):
    """More query tokens than tokens: those in front see nothing."""
    run([200, 3, 5], [150, 1, 0], 1, 2, D, "bf16", 40, 3)
    run([4, 3, 5], [2, 1, 0], 2, 2, D, "bf16", 1, 0)


@pytest.mark.parametrize("window,sinks", [(3000, 4), (500, 1000), (0, 0)])
def test_long_histories(window, sinks):
    """Cut into ranges and joined; keys split into parts, first tokens in several of them."""
    run(None, [20000, 9000], 1, 8, 128, "bf16", window, sinks)
    run([60, 5], [9000, 5000], 1, 2, 256, "bf16", window, sinks)
    run([200], [6000], 1, 2, 128, "f16", window, sinks)


def test_many_requests():
    lens = [(i * 37) % 400 for i in range(300)]
    run(None, lens, 1, 2, 64, "f16", 70, 10)
    run([i % 4 for i in range(300)], lens, 1, 2, 64, "f16", 70, 10)
    run([(i * 7) % 30 for i in range(150)], [500 + i for i in range(150)], 1, 8, 128, "bf16", 100, 70)


def test_strides_scale_and_untouched_rows():
    run([70, 200], [150, 600], 2, 2, 64, "f16", 90, 4, q_gap=16, o_gap=24, scale=0.4, lead=3, tail=9)
    run([70, 200], [150, 600], 2, 2, 256, "bf16", 90, 4, q_gap=8, o_gap=40, lead=1, tail=130, scale=-0.05)
    run(None, [70, 200], 2, 2, 128, "bf16", 90, 4, q_gap=8, o_gap=8, scale=-0.05)


def test_bad_pages_are_skipped():
    """Entries out of the pool among the first tokens' pages and the window's."""
    run(None, [1000, 640], 1, 4, 128, "bf16", 300, 130, status=(4, 1), mute=[(0, 0), (1, 8)])
    run([150, 20], [1000, 640], 1, 4, 128, "bf16", 300, 130, status=(4, 1), mute=[(0, 1), (0, 13), (1, 6)])
    run([150, 20], [1000, 640], 1, 2, 256, "f16", 300, 130, status=(4, 1), mute=[(0, 2), (0, 15), (1, 0)])


def test_lengths_out_of_range():
    """Past the table row, and below 0: cut, and told in the status."""
    c = Window(Pages([128, 100], 1, 64, "bf16", 0), None, 2, 50, 3)
    c.lens.copy_(torch.tensor([1000, -5], dtype=torch.int32))
    c.call()
    torch.cuda.synchronize()
    assert tpk.get_device_status(reset=True) == (4, 1)
    assert (c.lse[1] == float("-inf")).all() and (c.o[1] == 0).all() and torch.isfinite(c.lse[0]).all()


def test_other_stream_captured_and_grown():
    c = Window(Pages([300, 40], 2, 128, "bf16", 5), None, 4, 100, 4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.call(stream=st)
    c.check("stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(stream=torch.cuda.current_stream())
    # one token less: the lengths are read at every replay
    c.o.fill_(float("nan"))
    g.replay()
    c.check("replayed")
    assert tpk.get_device_status(reset=True) == (0, 0)


def test_no_queries():
    s = tpk.PagedShape(2, 2, 64, kv_slots=4, max_pages=2)
    tpk.window_attn_paged(s, 2, 0, 5, 1, None, 256, 16, 16, 16, 16, 16, None, 256, None, None, 0)


def test_a_window_of_everything_is_the_causal_prompt():
    """The same results, bit for bit, as cross attention with the causal ranges and decode."""
    from test_gpu_paged_cross import Cross
    pg = Pages([300, 90], 2, 128, "bf16", 3)
    a = Window(pg, [300, 90], 2, 0, 0)
    a.call()
    torch.cuda.synchronize()
    b = Cross(pg, [300, 90], 2, ranges=[(0, i + 1) for i in range(300)] + [(0, i + 1) for i in range(90)])
    b.dq.copy_(a.dq)
    b.call()
    torch.cuda.synchronize()
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("D", [64, 128, 256])
# 9,000 tokens through this window are 9 pages and 3 units more, 4 to a block: blocks 0 to 2 have work
@pytest.mark.parametrize("nq,lens,H,G,unit", [(None, [500, 40], 1, 4, 0), (None, [9000], 1, 8, 1), ([4, 3], [5000, 64], 1, 2, 0),
                                              ([300, 200], [1300, 700], 1, 2, 0), ([513, 700], [600, 1000], 16, 4, 0)])
def test_waits_are_bounded(nq, lens, H, G, unit, D):
    stalled(Window(Pages(lens, H, D, "bf16", 3), nq, G, 400, 70), unit)
