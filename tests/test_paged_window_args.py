"""Windowed attention refuses bad arguments on the host, before any launch (no GPU needed)."""
import ctypes

import pytest

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build
from test_paged_args import BAD_SHAPES, BIG, INVALID, NOMEM, err, shape


@pytest.fixture(scope="module")
def L():
    build.build()
    return tpk.lib()


def window(L, s, n_req=2, n_q=5, w=100, sinks=4, q=16, qs=4096, off=16, k=16, v=16, table=16, n=16, o=16, os=4096, lse=16, ws=16,
           nbytes=BIG):
    return L.tpk_window_attn_paged(ctypes.byref(s) if s else None, n_req, n_q, w, sinks, q, qs, off, k, v, table, n, o, os, lse, ws,
                                   nbytes, None)


@pytest.mark.parametrize("kw,code", BAD_SHAPES, ids=lambda x: str(x))
def test_shapes_are_refused(L, kw, code):
    assert window(L, shape(**kw)) == code, err(L)
    assert window(L, None) == INVALID


def test_arguments_are_refused(L):
    s = shape()
    for kw in [{"n_req": 0}, {"n_req": 4097}, {"n_req": -1}, {"q": None}, {"k": None}, {"v": None}, {"table": None}, {"n": None},
               {"o": None}, {"lse": None}, {"ws": None}, {"q": 24}, {"k": 8}, {"v": 8}, {"o": 8}, {"ws": 8}, {"qs": 4088},
               {"qs": 4100}, {"os": 4088}, {"os": 4097}, {"w": -1}, {"sinks": -1}, {"off": None}, {"off": 18}, {"n_q": -1},
               {"n_q": 1 << 27}, {"off": None, "n_q": 3}, {"table": 18}, {"lse": 2}]:
        assert window(L, s, **kw) == INVALID, (kw, err(L))
    assert window(L, shape(max_pages=0)) == INVALID and window(L, shape(max_pages=1 << 25)) == INVALID
    assert window(L, s, nbytes=1000) == NOMEM and "required" in err(L)
    assert window(L, s, off=None, n_q=2, nbytes=1000) == NOMEM
    assert window(L, s, n_q=0, q=None, o=None, lse=None, ws=None) == 0
    assert window(L, s, n_q=0, off=None) == INVALID


def test_workspace_is_enough_for_every_window(L):
    """Whatever kernel a call takes: the refusal's threshold never passes the stated size."""
    for kw in [{}, {"head_dim": 64, "group": 1}, {"head_dim": 256, "kv_heads": 2}, {"max_pages": 3000, "group": 20}]:
        s = shape(**{"kv_slots": 10000, "max_pages": 400, **kw})
        w = 16 * s.kv_heads * s.group * s.head_dim
        for n_req, n_q in [(1, 1), (3, 3), (1, 40), (8, 300), (60, 2000), (4096, 9000), (2, 100000)]:
            size = tpk.window_paged_workspace_bytes(s, n_req, n_q)
            assert size > 0
            for win in (0, 1, 64, 1000, 50000):
                # the workspace's alignment is checked before its size, its size before anything is launched
                st = window(L, s, n_req=n_req, n_q=n_q, w=win, qs=w, os=w, nbytes=0)
                assert st == NOMEM
                need = int(err(L).split("<")[1].split()[0])
                assert need <= size, (kw, n_req, n_q, win)
    assert tpk.window_paged_workspace_bytes(shape(), 0, 5) == 0 and tpk.window_paged_workspace_bytes(shape(), 1, -1) == 0


def test_python_call_marshals():
    s = shape()
    tpk.window_attn_paged(s, 2, 0, 5, 1, None, 4096, 16, 16, 16, 16, 16, None, 4096, None, None, 0)
    with pytest.raises(tpk.TpkError, match="window"):
        tpk.window_attn_paged(s, 2, 1, -5, 1, 16, 4096, 16, 16, 16, 16, 16, 16, 4096, 16, 16, BIG)
    with pytest.raises(OverflowError):
        tpk.window_attn_paged(s, 2, 1, 1 << 40, 1, 16, 4096, 16, 16, 16, 16, 16, 16, 4096, 16, 16, BIG)
