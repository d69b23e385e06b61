"""The calls on shared pages refuse bad arguments on the host, before any launch (no GPU needed),
and their plain models agree with themselves."""
import ctypes
import random

import pytest

import tiered_paged_kv_gb300 as tpk
from pages_util import compact_model, fork_model
from tiered_paged_kv_gb300 import build
from test_paged_args import BAD_SHAPES, INVALID, NOMEM, err, shape

BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return tpk.lib()


def fork(L, n=2, mp=4, slots=9, source=16, len_in=16, keep=16, tin=16, tout=48, sin=16, sout=16, free=16, cap=8, nin=16, nout=16,
         out=16, granted=16, cs=16, cd=16, ws=16, nbytes=BIG):
    return L.tpk_kv_pages_fork(n, mp, slots, source, len_in, keep, tin, tout, sin, sout, free, cap, nin, nout, out, granted, cs, cd,
                               ws, nbytes, None)


def compact(L, n=2, mp=4, slots=9, lens=16, tin=16, tout=16, sin=16, sout=16, fin=16, fout=16, cap=8, nin=16, nout=16, new=16, mc=3,
            cs=16, cd=16, nc=16, ws=16, nbytes=BIG):
    return L.tpk_kv_pages_compact(n, mp, slots, lens, tin, tout, sin, sout, fin, fout, cap, nin, nout, new, mc, cs, cd, nc, ws,
                                  nbytes, None)


def pools(*p):
    return (ctypes.c_void_p * len(p))(*p)


def copy(L, s, layers=2, k=(16, 16), v=(16, 16), n=3, src=16, dst=16):
    return L.tpk_kv_pages_copy(ctypes.byref(s) if s else None, layers, pools(*k) if k else None, pools(*v) if v else None, n, src,
                               dst, None)


COMMON = [{"n": 0}, {"n": 4097}, {"mp": 0}, {"mp": 1 << 25}, {"n": 4096, "mp": 1 << 20}, {"slots": 0}, {"slots": -1},
          {"slots": 1 << 31}, {"slots": (1 << 31) - 9}, {"cap": -1}, {"ws": None}, {"ws": 8}, {"nin": None}, {"nout": None},
          {"tin": None}, {"tout": None}, {"sin": None}, {"sout": None}, {"cs": None}, {"cd": None}, {"tin": 18}, {"sout": 17}]


def test_fork_arguments_are_refused(L):
    for kw in COMMON + [{"source": None}, {"len_in": None}, {"free": None}, {"out": None}, {"granted": None}, {"tout": 16},
                        {"keep": 2}, {"free": 6}]:
        assert fork(L, **kw) == INVALID, (kw, err(L))
    assert fork(L, nbytes=100) == NOMEM and "required" in err(L)
    # tables of 32 bytes, holders of 36: a part in common
    for kw in [{"tin": 48, "tout": 48}, {"tin": 48, "tout": 20}, {"tin": 48, "tout": 76}, {"sout": 20}, {"sin": 48}]:
        assert fork(L, **kw) == INVALID and "overlaps" in err(L), kw


def test_compact_arguments_are_refused(L):
    for kw in COMMON + [{"lens": None}, {"fin": None}, {"fout": None}, {"new": None}, {"nc": None}, {"mc": -1}, {"mc": 0x7fffffff}, {"new": 6}]:
        assert compact(L, **kw) == INVALID, (kw, err(L))
    assert compact(L, nbytes=100) == NOMEM
    for kw in [{"tout": 20}, {"tin": 44}, {"sout": 48}, {"fout": 44}, {"fin": 44}]:
        assert compact(L, **kw) == INVALID and "overlaps" in err(L), kw


@pytest.mark.parametrize("kw,code", BAD_SHAPES, ids=lambda x: str(x))
def test_copy_shapes_are_refused(L, kw, code):
    assert copy(L, shape(**kw)) == code, err(L)
    assert copy(L, None) == INVALID


def test_copy_arguments_are_refused(L):
    s = shape()
    for kw in [{"layers": 0}, {"layers": 4097}, {"n": -1}, {"k": None}, {"v": None}, {"k": (16, None)}, {"v": (None, 16)},
               {"k": (16, 8)}, {"v": (4, 16)}, {"src": None}, {"dst": None}, {"src": 2}, {"dst": 3}]:
        assert copy(L, s, **kw) == INVALID, (kw, err(L))
    assert copy(L, s, n=0) == 0 and copy(L, s, n=0, src=None, dst=None) == 0


def test_python_calls_marshal():
    s = shape()
    tpk.kv_pages_copy(s, [16, 16], (32, 32), 0, None, None)
    for args, exc in [(([16], [16, 16], 0, None, None), ValueError), ((16, [16], 0, None, None), TypeError),
                      (([1.5], [16], 0, None, None), TypeError), (([None], [16], 0, None, None), tpk.TpkError),
                      (([], [], 0, None, None), tpk.TpkError)]:
        with pytest.raises(exc):
            tpk.kv_pages_copy(s, *args)
    x = 16
    with pytest.raises(tpk.TpkError, match="n_req"):
        tpk.kv_pages_fork(0, 4, 9, x, x, None, x, 48, x, x, x, 8, x, x, x, x, x, x, x, BIG)
    with pytest.raises(tpk.TpkError, match="max_copies"):
        tpk.kv_pages_compact(1, 4, 9, x, x, x, x, x, x, x, 8, x, x, x, -1, x, x, x, x, BIG)
    with pytest.raises(tpk.TpkError, match="workspace"):
        tpk.kv_pages_fork(1, 4, 9, x, x, None, x, 48, x, x, x, 8, x, x, x, x, x, x, x, -1)


def test_workspace_sizes(L):
    assert tpk.kv_pages_workspace_bytes(100, 1) >= 800 and tpk.kv_pages_workspace_bytes(0, 1) == 0
    assert tpk.kv_pages_workspace_bytes(100, 0) == 0 and tpk.kv_pages_workspace_bytes(100, 4097) == 0
    assert tpk.kv_pages_workspace_bytes(1 << 31, 1) == 0


def test_models_keep_every_page_held_once():
    """Forks, growth and compaction in turn: what is held and what is free make up the pool, and holders are counted right."""
    rng = random.Random(1)
    n, max_pages, slots = 9, 6, 60
    table, lens, shares, free, n_free = [[-1] * max_pages for _ in range(n)], [0] * n, [0] * slots, list(range(slots)), slots
    for step in range(60):
        source = [rng.choice([b, b, rng.randrange(n), -1]) for b in range(n)]
        keep = [0 if s < 0 else rng.choice([lens[s], lens[s], rng.randint(0, lens[s])]) for s in source]
        rows, shares, free, n_free, lens, *_ = fork_model(source, lens, keep, table, shares, free, n_free, slots)
        if step % 4 == 3:
            table = [r + [-1] * (max_pages - len(r)) for r in rows]
            rows, shares, free, n_free, *_ = compact_model(lens, table, shares, free, n_free, slots, rng.choice([2, slots]))
        for b in range(n):  # every request grows a little
            for _ in range(rng.randrange(40)):
                if lens[b] < 64 * max_pages and (lens[b] % 64 or n_free):
                    if lens[b] % 64 == 0:
                        n_free -= 1
                        rows[b].append(free[n_free])
                    lens[b] += 1
        table = [r + [-1] * (max_pages - len(r)) for r in rows]
        held = [x for r in rows for x in r]
        assert sorted(set(held) | set(free[:n_free])) == list(range(slots)) and not set(held) & set(free[:n_free])
        assert all(shares[x] == held.count(x) - 1 for x in set(held)) and all(shares[x] == 0 for x in free[:n_free])
        for b in range(n):  # nobody else holds a page that will be written on
            assert lens[b] % 64 == 0 or held.count(rows[b][-1]) == 1
