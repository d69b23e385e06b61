"""Forks, compaction and page copies against plain models: every output exactly, entries that
are to be left alone as well."""
import random

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from pages_util import compact_model, fork_model, pages_of

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def workspace(kv_slots, n):
    size = tpk.kv_pages_workspace_bytes(kv_slots, n)
    return torch.randint(0, 255, (size,), dtype=torch.uint8, device="cuda"), size


# A small pool and table go to one block; the same rows in a wide table, or a pool with more slots, to a cluster
WIDE = 40000


def check_rows(got, before, rows):
    for b, row in enumerate(rows):
        assert got[b].tolist() == row + before[b][len(row):].tolist(), f"row {b}"


def fork(source, lens, keep, table, shares, free, n_free, in_place=False, stream=None, graph=False, wide=None):
    if wide is None and len(shares) < 100:  # both forms
        fork(source, lens, keep, table, shares, free, n_free, in_place, stream, graph, wide=True)
    n, max_pages, slots = len(lens), len(table[0]), len(shares)
    if wide:  # slots past those of the case: held by nobody here
        shares, slots = shares + [0] * (9000 - slots), 9000
    want = fork_model(source, lens, keep, table, shares, free, n_free, slots)
    d = {k: i32(v) for k, v in dict(source=source, lens=lens, table=table, shares=shares, free=free, n_free=[n_free]).items()}
    dk = None if keep is None else i32(keep)
    out = torch.full((n, max_pages), -9, dtype=torch.int32, device="cuda")
    so = d["shares"] if in_place else torch.full((slots,), -9, dtype=torch.int32, device="cuda")
    nf = d["n_free"] if in_place else i32([-9])
    lo = d["lens"] if in_place else torch.full((n,), -9, dtype=torch.int32, device="cuda")
    granted, cs, cd = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(3))
    ws, size = workspace(slots, n)

    def call():
        tpk.kv_pages_fork(n, max_pages, slots, d["source"], d["lens"], dk, d["table"], out, d["shares"], so, d["free"],
                          len(free), d["n_free"], nf, lo, granted, cs, cd, ws, size,
                          stream=stream or torch.cuda.current_stream())

    if graph:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        g.replay()
    else:
        call()
    torch.cuda.synchronize()
    rows, shares_out, free_out, left, length, ok, copy_src, copy_dst, bad = want
    assert tpk.get_device_status(reset=True)[1] == (1 if bad else 0)
    assert granted.tolist() == ok and lo.tolist() == length
    assert cs.tolist() == copy_src and cd.tolist() == copy_dst
    assert nf.tolist() == [left] and d["free"].tolist() == free_out and so.tolist() == shares_out
    check_rows(out.cpu(), torch.full((n, max_pages), -9, dtype=torch.int32), rows)
    assert d["table"].tolist() == table
    return want


def random_family(rng, n, max_pages, spare, most, share=0.6, pins=0.1):
    """A batch whose rows share beginnings, and the stack of what is left."""
    lens = [rng.randint(0, most) for _ in range(n)]
    need = sum(pages_of(x) for x in lens)
    slots = need + spare + 1
    order = list(range(slots))
    rng.shuffle(order)
    table, shares, at = [], [0] * slots, 0
    for b in range(n):
        row = []
        if b and rng.random() < share:
            p = rng.randrange(b)
            row = table[p][:rng.randint(0, min(lens[p] // 64, lens[b] // 64))]
            for x in row:
                shares[x] += 1
        while len(row) < pages_of(lens[b]):
            row.append(order[at])
            at += 1
        table.append(row + [-1 - b % 3] * (max_pages - len(row)))
    for x in order[:at]:
        shares[x] += rng.random() < pins  # holders outside the batch
    free = order[at:]
    return lens, table, shares, free[:spare] + [-5] * (slots - min(spare, len(free))), min(spare, len(free))


@pytest.mark.parametrize("seed", range(12))
def test_random_forks(seed):
    rng = random.Random(seed)
    n = rng.choice([1, 2, 3, 17, 60, 300])
    max_pages = rng.choice([1, 3, 12])
    lens, table, shares, free, n_free = random_family(rng, n, max_pages, rng.choice([0, 3, 40]), 64 * max_pages)
    source = [rng.choice([b, b, rng.randrange(n), rng.randrange(n), -1]) for b in range(n)]
    keep = [lens[s] if rng.random() < 0.5 else rng.randint(0, lens[s]) if s >= 0 else 0 for s in source]
    fork(source, lens, keep if seed % 3 else None, table, shares, free, n_free, in_place=seed % 2 == 1)


@pytest.mark.parametrize("n,max_pages,most", [(4096, 3, 192), (1, 5000, 320000), (5, 1100, 70000), (1025, 20, 1000), (256, 4, 256)])
def test_large_forks(n, max_pages, most):
    """All places of the launch: more requests than threads, rows longer than a team's step."""
    rng = random.Random(n)
    lens, table, shares, free, n_free = random_family(rng, n, max_pages, n // 2, most)
    source = [rng.randrange(n) if rng.random() < 0.6 else b for b in range(n)]
    keep = [lens[s] if rng.random() < 0.6 else rng.randint(0, lens[s]) for s in source]
    fork(source, lens, keep, table, shares, free, n_free)


def test_samples_beams_ends_and_cuts():
    # one prompt of 130 tokens sampled four times: three copies of its last page
    w = fork([0, 0, 0, 0], [130, 0, 0, 0], None, [[3, 4, 5], [-1] * 3, [-1] * 3, [-1] * 3], [0] * 9, [0, 1, 2, 6, 7, 8], 6)
    assert w[0] == [[3, 4, 5], [3, 4, 8], [3, 4, 7], [3, 4, 6]] and w[6] == [-1, 5, 5, 5] and w[1][3] == 3
    # beams change places: one stays and is copied from, into the page that nobody holds any more
    w = fork([1, 1, 0], [65, 66, 128], None, [[0, 1], [0, 2], [0, 3]], [2, 0, 0, 0], [-1] * 4, 0)
    assert w[0] == [[0, 3], [0, 2], [0, 1]] and w[6] == [2, -1, -1] and w[3] == 0
    # the prompt's own row ends: the first sample keeps the last page
    w = fork([-1, 0, 0], [100, 0, 0], None, [[1, 0], [-1, -1], [-1, -1]], [0] * 4, [2, 3, -1, -1], 2)
    assert w[0] == [[], [1, 0], [1, 3]] and w[6] == [-1, -1, 0]
    # cut inside a page that another holds whole, cut inside one's own, cut to a page's end, to nothing
    w = fork([0, 1, 2, 3], [128, 128, 128, 70], [100, 100, 64, 0], [[0, 1], [0, 2], [0, 3], [4, 5]], [2] + [0] * 7,
             [6, 7] + [-1] * 6, 2)
    assert w[0] == [[0, 1], [0, 2], [0], []] and w[3] == 5
    # a page held outside the batch as well is never written on
    w = fork([-1, 0], [30, 0], None, [[0], [-1]], [1, 0], [1], 1)
    assert w[0] == [[], [1]] and w[1] == [0, 0] and w[7] == [-1, 1]


def test_a_row_of_its_own_source_after_others():
    """Sources that are forks themselves: all read the rows of before."""
    fork([1, 2, 3, 0], [10, 74, 138, 64], None, [[0, -1, -1], [1, 2, -1], [3, 4, 5], [6, -1, -1]], [0] * 10, [7, 8, 9], 3)
    fork([2, 2, 0, 0], [10, 74, 138, 64], [138, 65, 10, 9], [[0, -1, -1], [1, 2, -1], [3, 4, 5], [6, -1, -1]], [0] * 10,
         [7, 8, 9], 3, in_place=True)


def test_too_few_slots():
    w = fork([0, 0, 0, 0], [70, 0, 0, 0], None, [[0, 1], [-1, -1], [-1, -1], [-1, -1]], [0] * 4, [3, 2, -1], 1)
    assert w[5] == [1, 1, 0, 0] and w[4] == [70, 70, 64, 64] and w[0][2] == [0]
    fork([0, 0], [5, 0], None, [[0], [-1]], [0], [], 0)  # no stack at all


def test_refusals_and_bad_entries():
    # sources and lengths out of range: the request stays as it was
    fork([5, -2, 0, 1, 3], [64, 64, 64, 64, 64], [0, 0, 65, -1, 64], [[0], [1], [2], [3], [4]], [0] * 6, [5], 1)
    # a length past the row, and one below 0, are cut
    fork([1, 1, 0], [200, -3, 10], None, [[0, 1], [2, 3], [4, 5]], [0] * 6, [-1] * 4, 0)
    # entries outside the pool: whole pages are carried along, an open page is not there to copy
    fork([0, 0], [128, 0], None, [[9, -4], [-1, -1]], [0] * 3, [0, 1, 2], 3)
    fork([0, 0], [100, 0], None, [[1, 77], [-1, -1]], [0] * 3, [0, 2], 2)
    # more releases than holders
    fork([-1, -1], [64, 64], None, [[0], [0]], [0, 0], [1, -1, -1], 1)
    # a stack without room, and counts out of range
    fork([-1, -1], [128, 64], None, [[0, 1], [2, -1]], [0] * 4, [3, -1], 1)
    fork([-1], [64], None, [[0]], [0, 0, 0], [1, 2], 7)
    fork([-1], [64], None, [[0]], [0, 0, 0], [1, 2, -1], -3)


def test_other_stream_and_captured():
    st = torch.cuda.Stream()
    args = ([0, 0, 0, 0], [130, 0, 0, 0], None, [[3, 4, 5], [-1] * 3, [-1] * 3, [-1] * 3], [0] * 9, [0, 1, 2, 6, 7, 8], 6)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        fork(*args, stream=st)
    fork(*args, graph=True)


def compact(lens, table, shares, free, n_free, max_copies, in_place=False, wide=None):
    if wide is None and len(shares) < 100 and all(0 <= n <= 64 * len(table[0]) for n in lens):  # both forms
        compact(lens, [r + [-1] * (-(-WIDE // len(lens)) - len(r)) for r in table], shares, free, n_free, max_copies, in_place, wide=True)
    n, max_pages, slots = len(lens), len(table[0]), len(shares)
    want = compact_model(lens, table, shares, free, n_free, slots, max_copies)
    d = {k: i32(v) for k, v in dict(lens=lens, table=table, shares=shares, n_free=[n_free]).items()}
    d["free"] = i32(free) if free else torch.zeros(1, dtype=torch.int32, device="cuda")
    empty = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out, so, fo, nf = ((d[k] for k in ("table", "shares", "free", "n_free")) if in_place
                       else (empty(n, max_pages), empty(slots), d["free"].clone(), empty(1)))
    cs, cd, nc, new = empty(max_copies + 1), empty(max_copies + 1), empty(1), empty(slots)
    ws, size = workspace(slots, n)
    tpk.kv_pages_compact(n, max_pages, slots, d["lens"], d["table"], out, d["shares"], so, d["free"], fo, len(free), d["n_free"],
                         nf, new, max_copies, cs, cd, nc, ws, size, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    rows, shares_out, free_out, left, new_slot, copy_src, copy_dst, n_copies, bad = want
    assert tpk.get_device_status(reset=True)[1] == (1 if bad else 0)
    assert nc.tolist() == [n_copies] and cs.tolist() == copy_src + [-9] and cd.tolist() == copy_dst + [-9]
    assert new.tolist() == new_slot and so.tolist() == shares_out and nf.tolist() == [left]
    assert fo.tolist()[:len(free)] == free_out
    before = torch.tensor(table, dtype=torch.int32) if in_place else torch.full((n, max_pages), -9, dtype=torch.int32)
    check_rows(out.cpu(), before, rows)
    return want


@pytest.mark.parametrize("seed", range(10))
def test_random_compaction(seed):
    rng = random.Random(100 + seed)
    n, max_pages = rng.choice([1, 4, 50, 700]), rng.choice([1, 9, 60])
    lens, table, shares, free, n_free = random_family(rng, n, max_pages, rng.choice([0, 5, 200, 3000]), 64 * max_pages)
    used = {x for b in range(n) for x in table[b][:pages_of(lens[b])]}
    stack = [x for x in range(len(shares)) if x not in used or rng.random() < 0]
    rng.shuffle(stack)
    shares = [0 if x not in used else s for x, s in enumerate(shares)]
    free = stack + [-5] * rng.choice([0, 7])
    compact(lens, table, shares, free, len(stack), rng.choice([0, 1, 6, len(shares), len(shares) // 3]), in_place=seed % 2 == 1)


@pytest.mark.parametrize("slots,held", [(100000, 0.5), (8192, 0.02), (8193, 0.98), (70000, 0.999)])
def test_large_pools(slots, held):
    rng = random.Random(slots)
    order = list(range(slots))
    rng.shuffle(order)
    k = int(slots * held)
    n, max_pages = 16, -(-k // 16) + 1
    table = [order[b * max_pages:min(k, (b + 1) * max_pages)] for b in range(n)]
    lens = [64 * len(r) for r in table]
    table = [r + [-1] * (max_pages - len(r)) for r in table]
    shares = [0] * slots
    for x in order[:k]:
        shares[x] = rng.randrange(4)
    compact(lens, table, shares, order[k:], slots - k, slots)


def test_lists_longer_than_the_pool():
    compact([64, 64], [[3], [0]], [0, 0, 0, 5], [1, 2], 2, 50)
    compact([64, 64], [[3], [0]], [0, 0, 0, 5], [1, 2], 2, 50, in_place=True)
    compact([64], [[0]], [0], [], 0, 9)
    compact([64], [[9000]], [0] * 9001, list(range(9000)), 9000, 20000)


def test_compaction_of_odd_inputs():
    compact([64], [[0]], [0], [], 0, 1)                                  # full
    compact([0], [[0]], [0, 0, 0], [2, 0, 1], 3, 3)                      # empty
    compact([64, 64], [[3], [0]], [0, 0, 0, 5], [1, 2], 2, 4)            # one move
    compact([64, 64], [[3], [0]], [0, 0, 0, 5], [1, 2], 2, 4, in_place=True)
    compact([64], [[1]], [0, 0, 0], [0, 9, -1, 0], 4, 3)                 # twice on the stack, out of the pool
    compact([200, -1], [[1, 7], [2, 2]], [0, 0, 0], [0], 1, 3)           # lengths and entries out of range
    compact([64], [[0]], [0, 0, 0], [0, 2], 2, 3)                        # a page that is on the stack


@pytest.mark.parametrize("H,D,dtype", [(1, 64, tpk.F16), (3, 128, tpk.BF16), (8, 256, tpk.BF16)])
@pytest.mark.parametrize("layers", [1, 3, 70])
def test_copies(H, D, dtype, layers):
    """Also more pools than a launch takes, and pairs that are none."""
    slots = 24
    dt = torch.bfloat16 if dtype == tpk.BF16 else torch.float16
    gen = torch.Generator(device="cuda").manual_seed(layers)
    pools = torch.randint(-30000, 30000, (layers, 2, slots, H, 64, D), device="cuda", generator=gen, dtype=torch.int16)
    src = [3, -1, 7, 3, 5, 0, 23, -1]
    dst = [4, 6, -1, 9, 5, 22, 1, -1]
    want = pools.clone()
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            want[:, :, d] = pools[:, :, s]
    data = pools.view(dt)
    s = tpk.PagedShape(H, 1, D, dtype=dtype, kv_slots=slots)
    tpk.kv_pages_copy(s, [data[i, 0] for i in range(layers)], [data[i, 1] for i in range(layers)], len(src), i32(src), i32(dst),
                      stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(pools, want)
    assert tpk.get_device_status(reset=True) == (0, 0)
    tpk.kv_pages_copy(s, tuple(data[i, 0] for i in range(layers)), [data[i, 1] for i in range(layers)], 3, i32([24, 2, 8]),
                      i32([2, 24, 10]))
    torch.cuda.synchronize()
    want[:, :, 10] = want[:, :, 8]
    assert torch.equal(pools, want) and tpk.get_device_status(reset=True) == (4, 1)
    tpk.kv_pages_copy(s, [data[0, 0]], [data[0, 1]], 0, None, None)


def test_copy_lists_longer_than_a_block_holds():
    H, D, slots, n = 1, 64, 9000, 4500
    gen = torch.Generator(device="cuda").manual_seed(1)
    pools = torch.randint(-30000, 30000, (2, slots, H, 64, D), device="cuda", generator=gen, dtype=torch.int16)
    perm = torch.randperm(slots, device="cuda", generator=gen).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    src[torch.rand(n, device="cuda", generator=gen) < 0.3] = -1
    src[:2500] = -1  # a whole stretch of the list without copies
    src[2490] = perm[2490]
    want, live = pools.clone(), src >= 0
    want[:, dst[live].long()] = pools[:, src[live].long()]
    s = tpk.PagedShape(H, 1, D, kv_slots=slots)
    tpk.kv_pages_copy(s, [pools[0]], [pools[1]], n, src, dst)
    torch.cuda.synchronize()
    assert torch.equal(pools, want)


def test_copies_past_32_bits():
    """Pages more than 2^32 bytes apart."""
    H, D = 4, 256
    slots = 2 ** 33 // (H * 64 * D * 2) + 4
    pool = torch.empty(slots, H, 64, D, dtype=torch.bfloat16, device="cuda")
    page = torch.randn(H, 64, D, device="cuda").to(torch.bfloat16)
    pool[slots - 1] = page
    pool[0] = -page
    s = tpk.PagedShape(H, 1, D, kv_slots=slots)
    tpk.kv_pages_copy(s, [pool], [pool], 2, i32([slots - 1, 0]), i32([1, slots - 2]))
    torch.cuda.synchronize()
    assert torch.equal(pool[1], page) and torch.equal(pool[slots - 2], -page) and torch.equal(pool[0], -page)
