"""Attention of one new token over paged histories whose lengths live on the device,
against the formula in 64 bits (bounds in paged_util)."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import PAGE, Pages, attention, check_attention

pytestmark = pytest.mark.gpu


class Decode:
    def __init__(self, pg, G, begin=None, q_gap=0, o_gap=0, scale=0.0, o_f32=False, mute=()):
        """mute: pages (request, index) whose table entries are out of the pool."""
        self.pg, self.G, self.begin, self.scale = pg, G, begin, scale or pg.D ** -0.5
        n, w = len(pg.lens), pg.H * G * pg.D
        self.q = pg.randn(n, w + q_gap)
        self.mute = set(mute)
        table = pg.table.clone()
        for i, (b, p) in enumerate(mute):
            table[b, p] = [-1, pg.slots, 2 ** 31 - 1, -2 ** 31][i % 4]
        self.dq, self.table, self.lens = self.q.cuda(), table.cuda(), torch.tensor(pg.lens, dtype=torch.int32).cuda()
        self.k, self.v = pg.k.cuda(), pg.v.cuda()
        self.dbegin = None if begin is None else torch.tensor(begin, dtype=torch.int32).cuda()
        self.o = torch.full((n, w + o_gap), float("nan"), dtype=torch.float32 if o_f32 else pg.dtype, device="cuda")
        self.lse = torch.full((n, pg.H * G), float("nan"), device="cuda")
        self.o_f32 = o_f32
        self.shape = tpk.PagedShape(pg.H, G, pg.D, dtype=tpk.BF16 if pg.dtype == torch.bfloat16 else tpk.F16,
                                    kv_slots=pg.slots, max_pages=pg.max_pages, sm_scale=scale)
        self.nbytes = tpk.decode_paged_workspace_bytes(self.shape, n)
        self.ws = torch.full((self.nbytes,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, stream=None, ws=None):
        tpk.decode_attn_paged(self.shape, len(self.pg.lens), self.dq, self.dq.stride(0), self.k, self.v, self.table,
                              self.lens, self.dbegin, self.o, self.o.stride(0), self.o_f32, self.lse,
                              self.ws if ws is None else ws, self.nbytes, stream=stream)

    def check(self, what=""):
        torch.cuda.synchronize()
        pg, G, D = self.pg, self.G, self.pg.D
        w = pg.H * G * D
        o, lse = self.o.cpu(), self.lse.cpu()
        if self.o_f32:
            assert o.dtype == torch.float32
        for b, n in enumerate(pg.lens):
            seen = torch.ones(G, n, dtype=torch.bool)
            if self.begin is not None:
                seen[:, :max(0, self.begin[b])] = False
            for bb, p in self.mute:
                if bb == b:
                    seen[:, p * PAGE:(p + 1) * PAGE] = False
            for h in range(pg.H):
                rows = slice(h * G, (h + 1) * G)
                q = self.q[b, :w].double().view(pg.H * G, D)[rows]
                want = attention(q, pg.keys[b][:, h], pg.values[b][:, h], seen, self.scale)
                check_attention(o[b, :w].view(pg.H * G, D)[rows], lse[b, rows], want, D, n, pg.dtype,
                                what=f"{what} request {b} ({n} tokens) head {h}")
        assert torch.isnan(o[:, w:]).all()


def run(lens, H, G, D, dtype, seed=0, status=(0, 0), **kw):
    d = Decode(Pages(lens, H, D, dtype, seed, max_pages=kw.pop("max_pages", None)), G, **kw)
    d.call()
    d.check()
    assert tpk.get_device_status(reset=True) == status
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 5, 8, 9, 16, 33])
def test_heads(G, D, dtype):
    run([1, 63, 64, 65, 0, 300, 17], 2, G, D, dtype, seed=G + D)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [0], [64], [15, 16, 17], [0, 0, 0], [5000], [1, 9000, 2, 0, 700], [64] * 70,
                                  list(range(0, 130))], ids=lambda x: f"{len(x)}x{max(x)}")
def test_lengths(lens, D):
    run(lens, 1, 4, D, "bf16", seed=len(lens))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,most,H,G,pages", [(60, 300, 4, 16, 5), (12, 1500, 4, 20, 40), (130, 200, 2, 12, 40), (7, 900, 3, 33, 40)])
def test_many_rows(n, most, H, G, pages, D):
    """More than eight heads a group, histories whole and cut, numbered by a warp, by the block."""
    lens = [(i * 379 + i // 3) % (most + 1) for i in range(n)]
    run(lens, H, G, D, "bf16", seed=G, max_pages=pages)


@pytest.mark.parametrize("n,D", [(110, 128), (130, 64), (130, 128), (110, 64)])
def test_waves_of_whole_runs(n, D):
    """One block per SM more or not; windows, bad pages, empty requests among them."""
    lens = [(i * 137) % 700 for i in range(n)]
    begin = [max(0, x - 200) if i % 3 == 0 else 0 for i, x in enumerate(lens)]
    lens[7], begin[7] = 690, 0
    run(lens, 4, 3, D, "f16", begin=begin, o_f32=True, mute=[(7, 1), (7, 10)], status=(4, 1), o_gap=8)


@pytest.mark.parametrize("pages", [24, 40])
def test_many_rows_windows_and_bad_pages(pages):
    n = 24
    lens = [(i * 379) % 1500 for i in range(n)]
    begin = [max(0, x - 130 * (i % 5)) for i, x in enumerate(lens)]
    lens[3], begin[3], begin[5] = 1000, 0, 0
    run(lens, 4, 16, 128, "f16", begin=begin, o_f32=True, max_pages=pages, mute=[(3, 2), (3, 15), (5, 0)], status=(4, 1))


@pytest.mark.parametrize("D", [64, 256])
def test_windows(D):
    lens = [1, 64, 65, 200, 1000, 1000, 1000, 500, 0]
    begin = [0, 63, 64, 100, 999, 1000, 2000, -5, 0]
    run(lens, 2, 8, D, "bf16", begin=begin, max_pages=40, status=(4, 1))  # -5 is clamped and reported


def test_strides_scale_and_f32_output():
    run([100, 700], 2, 3, 128, "bf16", q_gap=40, o_gap=16, scale=0.3)
    run([100, 700, 0], 2, 8, 256, "f16", o_f32=True, scale=-0.1)
    run([100, 700], 1, 12, 64, "bf16", o_f32=True, o_gap=8)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_scores(dtype):
    """Scores in the hundreds: one token takes nearly all the weight."""
    run([300, 64, 5000], 1, 8, 128, dtype, scale=8.0)


def test_bad_pages_contribute_nothing():
    run([1000, 64, 130], 2, 8, 128, "bf16", mute=[(0, 0), (0, 7), (1, 0), (2, 2)], status=(4, 1))


def test_bad_lengths_are_clamped():
    d = Decode(Pages([128, 100], 1, 64, "bf16", 3, max_pages=2), 4)
    d.lens.copy_(torch.tensor([10 ** 9, -4], dtype=torch.int32))
    d.pg.lens = [128, 0]
    d.pg.keys[1] = d.pg.keys[1][:0]
    d.pg.values[1] = d.pg.values[1][:0]
    d.call()
    d.check()
    assert tpk.get_device_status(reset=True) == (4, 1)


@pytest.mark.parametrize("n,most,max_pages", [(4096, 150, None), (129, 2000, None), (300, 130, 40), (600, 60, 33),
                                              (130, 1500, 32), (128, 900, 33)])
def test_many_requests(n, most, max_pages):
    """Whole and split histories, numbered by a warp and by the block."""
    lens = [(i * 37 + i // 7) % most for i in range(n)]
    pg = Pages(lens, 1, 64, "bf16", 9, max_pages=max_pages)
    d = Decode(pg, 2)
    d.call()
    torch.cuda.synchronize()
    o, lse = d.o.cpu(), d.lse.cpu()
    for b in list(range(0, n, 97 if n > 1000 else 11)) + [0, n - 1]:
        want = attention(d.q[b].double().view(2, 64), pg.keys[b][:, 0], pg.values[b][:, 0],
                         torch.ones(2, lens[b], dtype=torch.bool), d.scale)
        check_attention(o[b].view(2, 64), lse[b], want, 64, lens[b], pg.dtype, what=f"request {b}")


def test_bit_identical_whatever_the_workspace_holds():
    d = Decode(Pages([3000, 10, 900], 2, 128, "bf16", 4), 8)
    d.call()
    torch.cuda.synchronize()
    o, lse = d.o.clone(), d.lse.clone()
    d.ws.random_(0, 255)
    d.o.zero_()
    d.call()
    torch.cuda.synchronize()
    assert torch.equal(o, d.o) and torch.equal(lse, d.lse)


def test_two_streams_with_their_own_workspaces():
    a, b = Decode(Pages([4000, 33], 2, 128, "bf16", 5), 8), Decode(Pages([64, 2500], 2, 128, "bf16", 6), 8)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.call(sa)
        b.call(sb)
    a.check("first stream")
    b.check("second stream")


def test_captured_once_lengths_change():
    """A captured call follows lengths, tables and windows changed between replays."""
    pg = Pages([700, 300, 64], 2, 128, "bf16", 7)
    d = Decode(pg, 8, begin=[0, 0, 0])
    d.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        d.call(torch.cuda.current_stream())
    keys, values = pg.keys, pg.values
    for lens, begin in [([700, 300, 64], [0, 0, 0]), ([1, 299, 0], [0, 100, 0]), ([650, 0, 33], [649, 0, 5])]:
        pg.lens = lens
        pg.keys, pg.values = [k[:n] for k, n in zip(keys, lens)], [v[:n] for v, n in zip(values, lens)]
        d.begin = begin
        d.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        d.dbegin.copy_(torch.tensor(begin, dtype=torch.int32))
        # rows past a shorter length hold what they held: finite here, NaN elsewhere
        g.replay()
        d.check(str(lens))


def test_partials_fold_with_other_tiers():
    """A float32 result is a partial that tpk_merge_lse folds: two halves of a history
    (the second by its window) give the whole."""
    pg = Pages([1500], 2, 256, "bf16", 8)
    whole, first = Decode(pg, 8, o_f32=True), Decode(pg, 8, o_f32=True)
    second = Decode(pg, 8, begin=[777], o_f32=True)
    for d in (first, second):
        d.q, d.dq = whole.q, whole.dq
    first.lens = torch.tensor([777], dtype=torch.int32, device="cuda")
    acc, lse = torch.zeros_like(whole.o), torch.full_like(whole.lse, float("-inf"))
    for d in (whole, first, second):
        d.call()
    parts, lses = torch.stack([first.o, second.o]), torch.stack([first.lse, second.lse])
    tpk.merge_lse(2, 16, 256, parts, lses, acc, lse)
    whole.check()
    whole.o, whole.lse = acc, lse
    whole.check("folded")
