"""Page tables and slot maps built on the GPU against a stack-and-loop model: exact,
whatever grows, shrinks, finishes or is refused."""
import random

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import tables_model

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(old, new, table, free, n_free, max_tokens, in_place=False, stream=None):
    n, mp = len(old), len(table[0])
    d = {"old": i32(old), "new": i32(new), "table": i32(table), "free": i32(free + [0]), "fin": i32([n_free]),
         "fout": i32([-9]), "out": i32([-9] * n), "granted": i32([-9] * n), "off": i32([-9] * (n + 1)),
         "slot": torch.full((max_tokens + 1,), -9, dtype=torch.int64, device="cuda"), "pos": i32([-9] * (max_tokens + 1)),
         "req": i32([-9] * (max_tokens + 1))}
    if in_place:
        d["fout"], d["out"] = d["fin"], d["old"] if in_place == "old" else d["new"]
    tpk.kv_tables_update(n, mp, d["old"], d["new"], d["table"], d["free"], len(free), d["fin"], d["fout"], d["out"],
                         d["granted"], d["off"], d["slot"], d["pos"], d["req"], max_tokens, stream=stream)
    torch.cuda.synchronize()
    return d


def check(old, new, table, free, n_free, max_tokens, in_place=False):
    d = run(old, new, table, free, n_free, max_tokens, in_place)
    t, f = [list(r) for r in table], list(free)
    n_out, length, granted, off, slot, pos, req = tables_model(old, new, t, f, n_free, max_tokens)
    assert d["granted"].tolist() == granted
    assert d["out"].tolist() == length
    assert d["off"].tolist() == off
    assert d["fout"].item() == n_out
    assert d["table"].tolist() == t
    assert d["free"].tolist() == f + [0]
    assert d["slot"].tolist() == slot + [-9] and d["pos"].tolist() == pos + [-9] and d["req"].tolist() == req + [-9]


def random_case(seed, n, hi, max_pages, free_share=1.0, chunk=200, bad=False):
    rng = random.Random(seed)
    old = [rng.choice([0, 1, 63, 64, 65, rng.randint(0, hi)]) for _ in range(n)]
    new = []
    for a in old:
        r = rng.random()
        new.append(a if r < 0.1 else 0 if r < 0.2 else rng.randint(0, a) if r < 0.3 else a + 1 if r < 0.7
                   else a + rng.randint(1, chunk))
    if bad:
        for i in range(0, n, 5):
            old[i], new[i] = rng.choice([(-1, 5), (5, -1), (-3, -3), (max_pages * 64 + 1, 2), (3, max_pages * 64 + 1),
                                         (2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 1)])
    pages = lambda x: max(0, (x + 63) // 64)  # noqa: E731
    used = sum(min(max_pages, pages(a)) for a in old)
    want = sum(max(0, min(max_pages, pages(b)) - min(max_pages, pages(a))) for a, b in zip(old, new))
    n_free = int(want * free_share) + 1
    perm = list(range(used + n_free))
    rng.shuffle(perm)
    table = [[-1] * max_pages for _ in range(n)]
    for i, a in enumerate(old):
        for j in range(min(max_pages, pages(a))):
            table[i][j] = perm.pop()
    return old, new, table, perm + [-5] * used, len(perm)


@pytest.mark.parametrize("in_place", [False, "old", "new"])
@pytest.mark.parametrize("n,hi,max_pages", [(1, 10, 1), (2, 200, 9), (33, 900, 20), (257, 2000, 40), (1025, 700, 16),
                                            (4096, 300, 9)])
def test_random_batches(n, hi, max_pages, in_place):
    old, new, table, free, n_free = random_case(n, n, hi, max_pages)
    tokens = sum(max(0, b - a) for a, b in zip(old, new))
    check(old, new, table, free, n_free, tokens + 5, in_place)


@pytest.mark.parametrize("seed", range(4))
def test_refusals(seed):
    """Bad lengths, too few free slots, too small a token map."""
    old, new, table, free, n_free = random_case(seed, 70, 1500, 24, free_share=0.5, bad=seed % 2 == 1)
    tokens = sum(max(0, b - a) for a, b in zip(old, new) if 0 <= a and 0 <= b < 1 << 20)
    check(old, new, table, free, n_free, tokens // 2 if seed >= 2 else tokens + 1)


def test_edges():
    check([0], [0], [[-1]], [], 0, 0)              # nothing at all
    check([0], [1], [[-1]], [4], 1, 1)             # the first token of a request
    check([0], [64], [[-1, -1]], [4, 5], 2, 64)    # exactly a page
    check([64], [65], [[3, -1]], [4], 0, 1)        # no free slot
    check([64, 64], [0, 65], [[3, -1], [2, -1]], [7], 0, 1)          # a page given back is taken again
    check([64, 64, 64], [0, 0, 0], [[3], [2], [1]], [9, -1], 1, 0)   # more given back than the list holds
    st, flags = tpk.get_device_status(reset=True)
    assert st == 4 and flags == 1
    check([1, 5], [70000, 6], [[0] + [-1] * 1200, [1] + [-1] * 1200], list(range(2, 1200)), 1198, 70010)  # a long prompt


def test_free_count_is_clamped():
    d = run([0], [1], [[-1]], [4, 5], 99, 1)
    assert d["fout"].item() == 1 and d["table"].tolist() == [[5]]
    d = run([0], [1], [[-1]], [4, 5], -3, 1)
    assert d["fout"].item() == 0 and d["granted"].item() == 0


def test_graph_replay_advances_in_place():
    """One captured call, its lengths and free count in place, replayed: requests grow a
    token a step."""
    n, mp, free0 = 3, 4, list(range(20))
    length, grown = i32([0, 60, 127]), i32([0, 0, 0])
    table0 = [[-1] * mp, [20, -1, -1, -1], [21, 22, -1, -1]]
    table, free, nf = i32(table0), i32(free0), i32([20])
    granted, off = i32([0] * n), i32([0] * (n + 1))
    slot = torch.zeros(8, dtype=torch.int64, device="cuda")
    pos, req = i32([0] * 8), i32([0] * 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run([0], [1], [[-1]], [4], 1, 1)  # the device's first call, outside the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        torch.add(length, 1, out=grown)
        tpk.kv_tables_update(n, mp, length, grown, table, free, 20, nf, nf, length, granted, off, slot, pos, req, 8,
                             stream=torch.cuda.current_stream())
    lens, t, f, k = [0, 60, 127], [list(r) for r in table0], list(free0), 20
    for _ in range(70):
        g.replay()
        k, lens, gr, o, sl, ps, rq = tables_model(lens, [x + 1 for x in lens], t, f, k, 8)
        assert gr == [1, 1, 1]
        torch.cuda.synchronize()
        assert slot.tolist() == sl and pos.tolist() == ps and req.tolist() == rq
        assert length.tolist() == lens and table.tolist() == t and nf.item() == k and off.tolist() == o
