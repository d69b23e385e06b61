"""Decode over shared prefixes refuses bad arguments on the host, before any launch (no GPU needed)."""
import ctypes

import pytest

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build
from test_paged_args import BAD_SHAPES, BIG, INVALID, NOMEM, err, shape


@pytest.fixture(scope="module")
def L():
    build.build()
    return tpk.lib()


def shared(L, s, n_req=2, n_grp=1, q=16, qs=4096, k=16, v=16, table=16, n=16, off=16, sh=16, o=16, os=4096, f32=0, lse=16, ws=16,
           nbytes=BIG):
    return L.tpk_decode_attn_shared(ctypes.byref(s) if s else None, n_req, n_grp, q, qs, k, v, table, n, off, sh, o, os, f32, lse, ws,
                                    nbytes, None)


@pytest.mark.parametrize("kw,code", BAD_SHAPES, ids=lambda x: str(x))
def test_shapes_are_refused(L, kw, code):
    assert shared(L, shape(**kw)) == code, err(L)
    assert shared(L, None) == INVALID


def test_arguments_are_refused(L):
    s = shape()
    for kw in [{"n_req": 0}, {"n_req": 4097}, {"n_grp": 0}, {"n_grp": 4097}, {"q": None}, {"k": None}, {"v": None}, {"table": None},
               {"n": None}, {"off": None}, {"sh": None}, {"o": None}, {"lse": None}, {"ws": None}, {"q": 24}, {"k": 8}, {"v": 8},
               {"o": 8}, {"ws": 8}, {"qs": 4088}, {"qs": 4100}, {"os": 4088}, {"os": 4097}, {"f32": 2}, {"off": 18}, {"sh": 2},
               {"table": 18}, {"n": 1}, {"lse": 2}]:
        assert shared(L, s, **kw) == INVALID, (kw, err(L))
    assert shared(L, shape(max_pages=0)) == INVALID and shared(L, shape(max_pages=1 << 25)) == INVALID
    assert shared(L, s, nbytes=1000) == NOMEM and "required" in err(L)


def test_workspace_grows_with_requests_only(L):
    for kw in [{}, {"head_dim": 64, "group": 1}, {"head_dim": 256, "kv_heads": 1, "group": 128}]:
        s = shape(**kw)
        sizes = [tpk.decode_shared_workspace_bytes(s, n, g) for n in (1, 2, 7, 64, 4096) for g in (1, 5, 4096)]
        assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[0] == sizes[2]
    assert tpk.decode_shared_workspace_bytes(shape(), 0, 1) == 0 and tpk.decode_shared_workspace_bytes(shape(), 1, 0) == 0
    assert tpk.decode_shared_workspace_bytes(shape(), 4097, 1) == 0 and L.tpk_decode_shared_workspace_bytes(None, 1, 1) == 0


def test_python_call_marshals():
    s = shape()
    with pytest.raises(tpk.TpkError, match="n_grp"):
        tpk.decode_attn_shared(s, 2, 0, 16, 4096, 16, 16, 16, 16, 16, 16, 16, 4096, False, 16, 16, BIG)
    with pytest.raises(tpk.TpkError, match="workspace"):
        tpk.decode_attn_shared(s, 2, 1, 16, 4096, 16, 16, 16, 16, 16, 16, 16, 4096, False, 16, 16, -1)
