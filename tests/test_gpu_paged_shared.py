"""Decode attention of groups that share a prefix, against the formula in 64 bits for each request
by itself.

Bounds as in paged_util with one plane (a prefix's weights are rounded once), and the join's: what a
request does not share comes as a log-sum, whose rounding and way back into base 2 are four float32
roundings of it, so the two sides' weights are off by 2^-22 |lse| relative to each other, |lse| being
at most S + ln n + 1: lse moves by that, o by twice that times A."""
import math

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import DTYPES, PAGE, attention, attention_bounds
from test_gpu_paged_wait_limit import stalled

pytestmark = pytest.mark.gpu


class Shared:
    """groups: (prefix tokens, [each request's tokens, the prefix counted in]).  Rows of pages that hold no
    token are NaN, table entries without a page out of the pool."""

    def __init__(self, groups, H, G, D, dtype, seed=0, alone=(), f32=False, q_gap=0, o_gap=0, scale=0.0, max_pages=None, leaders=True):
        gen = torch.Generator().manual_seed(seed)
        dt = self.dtype = DTYPES[dtype]
        self.H, self.G, self.D, self.scale, self.f32 = H, G, D, scale or D ** -0.5, f32
        rnd = lambda *s: torch.randn(*s, generator=gen).to(dt)  # noqa: E731
        front, back = alone[:len(alone) // 2], alone[len(alone) // 2:]  # requests in no group
        off, shared, self.lens, self.keys, self.values, rows = [len(front)], [], [], [], [], []
        pages = []  # (keys, values) [tokens, H, D] of each page

        def own(k, v):
            out = []
            for i in range(0, k.shape[0], PAGE):
                pages.append((k[i:i + PAGE], v[i:i + PAGE]))
                out.append(len(pages) - 1)
            return out

        def add(pk, pv, whole, n):
            p = pk.shape[0]
            k, v = torch.cat([pk, rnd(max(0, n - p), H, D)])[:n], torch.cat([pv, rnd(max(0, n - p), H, D)])[:n]
            self.lens.append(n)
            self.keys.append(k.double())
            self.values.append(v.double())
            # its whole pages of the prefix are the group's, a part of one is its own copy
            mine = whole[:n // PAGE]
            rows.append(mine + own(k[len(mine) * PAGE:], v[len(mine) * PAGE:]))

        none = rnd(0, H, D)
        for n in front:
            add(none, none, [], n)
        for p, lens in groups:
            pk, pv = rnd(p, H, D), rnd(p, H, D)
            whole = own(pk[:p // PAGE * PAGE], pv[:p // PAGE * PAGE])
            for n in lens:
                add(pk, pv, whole, n)
            off.append(len(self.lens))
            shared.append(p)
        for n in back:
            add(none, none, [], n)
        n = len(self.lens)
        self.slots = len(pages) + 2
        self.max_pages = max_pages or max(1, max(len(r) for r in rows), max(-(-p // PAGE) for p, _ in groups))
        perm = torch.randperm(self.slots, generator=gen)
        kp = torch.full((self.slots, H, PAGE, D), float("nan"), dtype=dt)
        vp = torch.full((self.slots, H, PAGE, D), float("inf"), dtype=dt)
        for i, (k, v) in enumerate(pages):
            kp[perm[i], :, :k.shape[0]], vp[perm[i], :, :v.shape[0]] = k.transpose(0, 1), v.transpose(0, 1)
        table = torch.full((n, self.max_pages), -7, dtype=torch.int32)
        for b, r in enumerate(rows):
            table[b, :len(r)] = perm[r].int()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        w = H * G * D
        self.n, self.n_grp = n, len(groups)
        self.q = rnd(n, w + q_gap)
        self.dq, self.k, self.v, self.table = self.q.cuda(), kp.cuda(), vp.cuda(), table.cuda()
        self.dlens, self.off, self.shared = i32(self.lens), i32(off), i32(shared)
        self.o = torch.full((n, w + o_gap), float("nan"), dtype=torch.float32 if f32 else dt, device="cuda")
        self.lse = torch.full((n, H * G), float("nan"), device="cuda")
        self.shape = tpk.PagedShape(H, G, D, dtype=tpk.BF16 if dtype == "bf16" else tpk.F16, kv_slots=self.slots,
                                    max_pages=self.max_pages, sm_scale=scale)
        self.nbytes = tpk.decode_shared_workspace_bytes(self.shape, n, self.n_grp)
        self.ws = torch.full((self.nbytes,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        tpk.decode_attn_shared(self.shape, self.n, self.n_grp, self.dq, self.dq.stride(0), self.k, self.v, self.table, self.dlens,
                               self.off, self.shared, self.o, self.o.stride(0), self.f32, self.lse, self.ws, self.nbytes,
                               stream=stream)

    def check(self, what=""):
        torch.cuda.synchronize()
        H, G, D = self.H, self.G, self.D
        o, lse = self.o.cpu(), self.lse.cpu()
        for b, n in enumerate(self.lens):
            for h in range(H):
                q = self.q[b, h * G * D:(h + 1) * G * D].double().view(G, D)
                want = attention(q, self.keys[b][:, h], self.values[b][:, h], torch.ones(G, n, dtype=torch.bool), self.scale)
                go, gl = o[b, h * G * D:(h + 1) * G * D].view(G, D), lse[b, h * G:(h + 1) * G]
                at = f"{what} request {b} of {n} head {h}"
                if n == 0:
                    assert (go == 0).all() and (gl == float("-inf")).all(), at
                    continue
                ro, rl, a, s = want
                o_tol, lse_tol = attention_bounds(ro, rl, a, s, D, n, go.dtype, self.dtype, one_plane=True)
                join = 2.0 ** -22 * (s + math.log(n) + 1)
                d = (go.double() - ro).abs() / (o_tol + 2 * join[:, None] * a)
                assert (d <= 1).all(), f"{at}: o off by {d.max():.2f} of its bound"
                d = (gl.double() - rl).abs() / (lse_tol + join)
                assert (d <= 1).all(), f"{at}: lse off by {d.max():.2f} of its bound"
        assert torch.isnan(o[:, H * G * D:]).all()


def run(groups, H, G, D, dtype, status=(0, 0), **kw):
    c = Shared(groups, H, G, D, dtype, **kw)
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == status
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8, 20, 128])
def test_heads(G, D, dtype):
    run([(200, [230, 260, 201])], 2 if G < 100 else 1, G, D, dtype, seed=G)


# Few rows a group go through one launch in runs of 8 or 16, many (or some behind a wide table) as row
# tiles: all of these
FEW_AND_MANY = pytest.mark.parametrize("G,wide", [(2, None), (20, None), (20, 20000)])


@FEW_AND_MANY
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 128, 1000])
def test_prefix_lengths(prefix, D, G, wide):
    """Also one that ends inside a page, requests with nothing of their own, and with less than it."""
    run([(prefix, [prefix + 3, prefix, prefix + 64, prefix + 200])], 1, G, D, "bf16", max_pages=wide)
    run([(prefix, [prefix + 3, prefix // 2, 0, prefix])], 1, G, D, "bf16", max_pages=wide)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 65, 700])
def test_wide_tables(prefix, D, dtype):
    """Tables much wider than what they hold: groups of up to 16 rows in runs of 16."""
    run([(prefix, [prefix + 3, prefix // 2, 0, prefix + 300]), (40, [300, 41])], 2, 4, D, dtype, max_pages=20000, alone=(30, 500))


@FEW_AND_MANY
@pytest.mark.parametrize("D", [64, 128, 256])
def test_groups_of_all_sizes(D, G, wide):
    run([(300, [320] * 2 + [0]), (40, [41]), (700, []), (130, [130 + i for i in range(70)]), (64, [0, 0])], 2, G, D, "f16",
        alone=(70, 0, 333, 1), max_pages=wide)
    run([(300, [320] * 2 + [0]), (40, [41]), (700, []), (130, [130 + i for i in range(7)]), (64, [0, 0])], 1, G, D, "bf16",
        alone=(70, 0, 333, 1), max_pages=wide)


@pytest.mark.parametrize("G,n", [(8, 40), (1, 300), (5, 60)])
def test_more_rows_than_a_tile(G, n):
    run([(500, [500 + (i * 7) % 90 for i in range(n)])], 2, G, 64, "bf16")
    run([(500, [500 + (i * 7) % 90 for i in range(n)])], 1, G, 256, "f16")


@FEW_AND_MANY
def test_long_prefixes(G, wide):
    """Cut into many parts; own parts cut into ranges."""
    run([(9000, [9100, 9003, 9000, 12000])], 1, G, 128, "bf16", max_pages=wide)
    run([(6000, [6100, 6003]), (3000, [3000, 8000, 3500])], 1, G, 256, "bf16", max_pages=wide)


@FEW_AND_MANY
def test_nobody_has_the_whole_prefix(G, wide):
    """The row with the most of it is read, whichever that is."""
    run([(500, [0, 130, 300, 300, 20]), (200, [0, 199])], 1, G, 128, "bf16", max_pages=wide)


@FEW_AND_MANY
def test_strides_scale_and_output_type(G, wide):
    run([(100, [150, 120])], 2, G, 64, "f16", f32=True, q_gap=16, o_gap=24, scale=0.4, max_pages=wide)
    run([(100, [150, 120])], 2, G, 256, "bf16", q_gap=8, o_gap=8, scale=-0.05, alone=(30,), max_pages=wide)
    run([(100, [150, 120])], 2, G, 128, "bf16", f32=True, max_pages=wide)


@FEW_AND_MANY
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores(D, G, wide):
    run([(300, [350, 420])], 1, G, D, "bf16", scale=4.0, max_pages=wide)


def test_many_requests_and_groups():
    run([(64 * (i % 4), [64 * (i % 4) + j * 9 for j in range(1 + i % 7)]) for i in range(90)], 1, 2, 64, "bf16")


@FEW_AND_MANY
def test_nan_queries_stay_in_their_row(G, wide):
    c = Shared([(200, [230, 260, 201])], 2, G, 128, "bf16", max_pages=wide)
    c.dq[1, 128:256] = float("nan")
    c.call()
    torch.cuda.synchronize()
    assert torch.isnan(c.o[1, 128:256]).all() and torch.isnan(c.lse[1, 1])
    c.o[1, 128:256], c.lse[1, 1] = 0, 0
    assert torch.isfinite(c.o).all() and torch.isfinite(c.lse).all()


@FEW_AND_MANY
def test_bad_entries_and_counts(G, wide):
    """A page of the prefix that is not there is left out for everybody; values out of range are cut."""
    c = Shared([(300, [320, 330])], 1, G, 64, "bf16", max_pages=wide)
    c.table[0, 1] = c.slots  # the row that is read for the group
    c.keys = [torch.cat([k[:64], k[128:]]) for k in c.keys]
    c.values = [torch.cat([v[:64], v[128:]]) for v in c.values]
    c.lens = [n - 64 for n in c.lens]
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == (4, 1)
    c = Shared([(128, [128, 128])], 1, G, 64, "bf16", max_pages=wide)
    c.shared.fill_(64 * c.max_pages + 1)  # past the table row
    c.off.copy_(torch.tensor([-3, 9], dtype=torch.int32))
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == (4, 1)


@FEW_AND_MANY
def test_other_stream_captured_and_grown(G, wide):
    c = Shared([(300, [320, 330]), (64, [100, 70])], 2, G, 128, "bf16", alone=(40, 50), max_pages=wide)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.call(stream=st)
    c.check("stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(stream=torch.cuda.current_stream())
    # a request goes, another prefix: lengths are read at every replay
    c.lens[1] = 0
    c.keys[1], c.values[1] = c.keys[1][:0], c.values[1][:0]
    c.dlens[1] = 0
    c.shared[0] = 128
    c.o.fill_(float("nan"))
    g.replay()
    c.check("replayed")
    a, b = c.o.clone(), c.lse.clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c.o) and torch.equal(b, c.lse)  # bit for bit
    assert tpk.get_device_status(reset=True) == (0, 0)


def test_one_workspace_for_fewer_requests():
    big = Shared([(600, [620] * 30)], 2, 4, 64, "bf16")
    for groups in ([(600, [620] * 2)], [(600, [620] * 3)] * 8, [(50, [70])] * 30):
        c = Shared(groups, 2, 4, 64, "bf16")
        assert c.nbytes <= big.nbytes
        c.ws = big.ws
        c.call()
        c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("groups,H,G", [([(3000, [3100, 3300])], 1, 4), ([(300, [310] * 70)], 2, 8),
                                        ([(500, [600, 700]), (80, [90] * 5)], 1, 2),
                                        ([(500, [600, 700]), (80, [90] * 5)], 1, 20)])
def test_waits_are_bounded(groups, H, G, D):
    stalled(Shared(groups, H, G, D, "bf16"))


def test_waits_are_bounded_in_wide_tables():
    for D in (64, 128, 256):
        stalled(Shared([(500, [600, 700, 520])], 1, 4, D, "bf16", max_pages=20000))


def test_forked_requests_decode_together():
    """A run of the calls as sampling uses them: a prompt is stored, forked, its open page copied; each
    sample's next token is normed, rotated and stored; the group decodes; the batch is compacted and
    decodes the same."""
    H, G, D, n, max_pages, slots = 2, 4, 128, 4, 8, 24
    dt, dev = torch.bfloat16, "cuda"
    gen = torch.Generator().manual_seed(3)
    prompt = 200
    shape = tpk.PagedShape(H, G, D, kv_slots=slots, max_pages=max_pages)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    zeros = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    kp = torch.full((slots, H, PAGE, D), float("nan"), dtype=dt, device=dev)
    vp = kp.clone()
    w = (H * G + 2 * H) * D
    free, n_free = torch.arange(slots, dtype=torch.int32, device=dev), i32([slots])
    lens, table, shares = zeros(n), zeros(n, max_pages) - 1, zeros(slots)
    granted, off = zeros(n), zeros(n + 1)
    wq, wk = ((torch.randn(D, generator=gen) * 0.2 + 1).to(dt).to(dev) for _ in range(2))
    freq = torch.tensor([1e4 ** (-2 * j / D) for j in range(D // 2)], device=dev)

    def grow(new, cap):
        slot, pos, req = torch.zeros(cap, dtype=torch.int64, device=dev), zeros(cap), zeros(cap)
        tpk.kv_tables_update(n, max_pages, lens, i32(new), table, free, slots, n_free, n_free, lens, granted, off, slot, pos, req, cap)
        qkv = torch.randn(cap, w, generator=gen).to(dt).to(dev)
        q = torch.zeros(cap, H * G * D, dtype=dt, device=dev)
        tpk.kv_norm_rope_append(shape, cap, qkv, w, qkv[:, H * G * D:], w, qkv[:, (H * G + H) * D:], w, wq, wk, 1e-6, pos, 1, None,
                                freq, D, False, slot, q, H * G * D, kp, vp)
        return q

    def history(b):
        m = int(lens[b])
        page = table[b, :-(-m // PAGE)].long()
        return [x[page].transpose(1, 2).reshape(-1, H, D)[:m].double().cpu() for x in (kp, vp)]

    def decode(q):
        o, lse = torch.zeros(n, H * G * D, dtype=dt, device=dev), torch.zeros(n, H * G, device=dev)
        size = tpk.decode_shared_workspace_bytes(shape, n, 1)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        tpk.decode_attn_shared(shape, n, 1, q, H * G * D, kp, vp, table, lens, i32([0, n]), i32([prompt]), o, H * G * D, False, lse,
                               ws, size)
        torch.cuda.synchronize()
        return o, lse

    grow([prompt, 0, 0, 0], prompt)
    size = tpk.kv_pages_workspace_bytes(slots, n)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    out, src, dst = zeros(n, max_pages) - 1, zeros(n), zeros(n)
    tpk.kv_pages_fork(n, max_pages, slots, zeros(n), lens, None, table, out, shares, shares, free, slots, n_free, n_free, lens, granted,
                      src, dst, ws, size)
    tpk.kv_pages_copy(shape, [kp], [vp], n, src, dst)
    table = out
    torch.cuda.synchronize()
    assert lens.tolist() == [prompt] * n and granted.tolist() == [1] * n
    assert n_free.item() == slots - 4 - 3 and src.tolist()[0] == -1 and shares.sum().item() == 3 * 3
    q = grow([prompt + 1] * n, n)
    first = decode(q)
    for b in range(n):
        k, v = history(b)
        for j in range(H * G):
            x = q[b, j * D:(j + 1) * D].double().cpu()[None]
            ro, rl, a, s = attention(x, k[:, j // G], v[:, j // G], torch.ones(1, prompt + 1, dtype=torch.bool), D ** -0.5)
            o_tol, lse_tol = attention_bounds(ro, rl, a, s, D, prompt + 1, dt, dt, one_plane=True)
            join = 2.0 ** -22 * (s + math.log(prompt + 1) + 1)
            assert ((first[0][b, j * D:(j + 1) * D].double().cpu() - ro).abs() <= o_tol + 2 * join[:, None] * a).all()
            assert ((first[1][b, j].double().cpu() - rl).abs() <= lse_tol + join).all()
    # one sample ends, the others' pages move together
    out = table.clone()
    tpk.kv_pages_fork(n, max_pages, slots, i32([0, -1, 2, 3]), lens, None, table, out, shares, shares, free, slots, n_free, n_free, lens,
                      granted, src, dst, ws, size)
    table = out
    new, cs, cd, nc = zeros(slots), zeros(slots), zeros(slots), zeros(1)
    tpk.kv_pages_compact(n, max_pages, slots, lens, table, table, shares, shares, free, free, slots, n_free, n_free, new, slots, cs, cd,
                         nc, ws, size)
    tpk.kv_pages_copy(shape, [kp], [vp], slots, cs, cd)
    again = decode(q)
    torch.cuda.synchronize()
    live = [0, 2, 3]
    assert torch.equal(again[0][live], first[0][live]) and torch.equal(again[1][live], first[1][live])
    assert (again[1][1] == float("-inf")).all()
    held = sorted({int(x) for b in live for x in table[b, :4]})
    assert held == list(range(len(held))) and n_free.item() == slots - len(held)
    assert tpk.get_device_status(reset=True) == (0, 0)
