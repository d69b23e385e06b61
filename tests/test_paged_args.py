"""The calls over device-side lengths refuse bad arguments on the host, before any
launch (no GPU needed), and their plain model agrees with itself."""
import ctypes

import numpy as np
import pytest

import tiered_paged_kv_gb300 as tpk
from paged_util import tables_model
from tiered_paged_kv_gb300 import build

INVALID, UNSUPPORTED, NOMEM = 1, 2, 5
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return tpk.lib()


def shape(**kw):
    d = dict(kv_heads=4, group=8, head_dim=128, kv_slots=100, max_pages=10)
    d.update(kw)
    return tpk.PagedShape(**d)


def err(L):
    return L.tpk_last_error_string().decode()


def decode(L, s, n_req=2, q=16, qs=4096, k=16, v=16, table=16, n=16, begin=None, o=16, os=4096, f32=0, lse=16, ws=16,
           nbytes=BIG):
    return L.tpk_decode_attn_paged(ctypes.byref(s) if s else None, n_req, q, qs, k, v, table, n, begin, o, os, f32, lse,
                                   ws, nbytes, None)


def cross(L, s, n_req=2, n_q=5, q=16, qs=4096, off=16, k=16, v=16, table=16, n=16, rng=None, o=16, os=4096, lse=16,
          ws=16, nbytes=BIG):
    return L.tpk_cross_attn_paged(ctypes.byref(s) if s else None, n_req, n_q, q, qs, off, k, v, table, n, rng, o, os,
                                  lse, ws, nbytes, None)


def rope(L, s, n=5, q=16, qs=4096, k=16, ks=512, v=16, vs=512, pos=16, axes=1, axis=None, freq=16, rot=128, pairs=0,
         slot=16, qo=16, qos=4096, kp=16, vp=16):
    return L.tpk_kv_rope_append(ctypes.byref(s) if s else None, n, q, qs, k, ks, v, vs, pos, axes, axis, freq, rot, pairs,
                                slot, qo, qos, kp, vp, None)


def tables(L, n_req=2, max_pages=4, old=16, new=16, table=16, free=16, cap=8, fin=16, fout=16, out=16, granted=16,
           off=16, slot=16, pos=16, req=16, mt=10):
    return L.tpk_kv_tables_update(n_req, max_pages, old, new, table, free, cap, fin, fout, out, granted, off, slot, pos,
                                  req, mt, None)


BAD_SHAPES = [({"kv_heads": 0}, INVALID), ({"kv_heads": 1025}, INVALID), ({"group": 0}, INVALID),
              ({"group": 129}, INVALID), ({"head_dim": 96}, UNSUPPORTED), ({"head_dim": 0}, UNSUPPORTED),
              ({"page_tokens": 32}, UNSUPPORTED), ({"dtype": 2}, INVALID), ({"sm_scale": float("nan")}, INVALID),
              ({"sm_scale": float("inf")}, INVALID), ({"kv_slots": 0}, INVALID),
              ({"kv_slots": 2 ** 31 // (4 * 64)}, UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_SHAPES, ids=lambda x: str(x))
@pytest.mark.parametrize("call", [decode, cross, rope], ids=lambda f: f.__name__)
def test_shapes_are_refused(L, call, kw, code):
    assert call(L, shape(**kw)) == code, err(L)
    assert call(L, None) == INVALID


@pytest.mark.parametrize("call", [decode, cross], ids=lambda f: f.__name__)
def test_attention_arguments_are_refused(L, call):
    s = shape()
    for kw in [{"n_req": 0}, {"n_req": 4097}, {"q": None}, {"k": None}, {"v": None}, {"table": None}, {"n": None},
               {"o": None}, {"lse": None}, {"ws": None}, {"q": 24}, {"k": 8}, {"v": 8}, {"o": 8}, {"ws": 8},
               {"qs": 4088}, {"qs": 4100}, {"os": 4088}, {"os": 4097}]:
        assert call(L, s, **kw) == INVALID, (kw, err(L))
    assert call(L, shape(max_pages=0)) == INVALID
    assert call(L, shape(max_pages=1 << 25)) == INVALID
    assert call(L, s, nbytes=1000) == NOMEM and "required" in err(L)
    assert decode(L, s, f32=2) == INVALID
    assert cross(L, s, off=None) == INVALID
    assert cross(L, s, n_q=-1) == INVALID
    assert cross(L, s, n_q=1 << 27) == INVALID


def test_workspace_sizes(L):
    s = shape()
    assert tpk.decode_paged_workspace_bytes(s, 1) > 0
    assert tpk.decode_paged_workspace_bytes(s, 0) == 0 and tpk.decode_paged_workspace_bytes(s, 4097) == 0
    assert tpk.cross_paged_workspace_bytes(s, 1, 0) > 0 and tpk.cross_paged_workspace_bytes(s, 1, -1) == 0
    assert tpk.decode_paged_workspace_bytes(shape(head_dim=80), 1) == 0
    assert L.tpk_decode_paged_workspace_bytes(None, 1) == 0


def test_rope_arguments_are_refused(L):
    s = shape()
    for kw in [{"n": -1}, {"rot": 130}, {"rot": 144}, {"rot": -16}, {"rot": 8}, {"pairs": 2}, {"q": None}, {"qo": None},
               {"k": None}, {"v": None}, {"kp": None}, {"vp": None}, {"slot": None}, {"pos": None}, {"freq": None},
               {"axes": 0}, {"axes": 5}, {"qs": 4088}, {"qos": 4090}, {"ks": 504}, {"vs": 511}, {"q": 8}, {"k": 24},
               {"v": 4}, {"qo": 8}, {"kp": 8}, {"vp": 8}, {"qs": 8192},  # in place with another stride
               {"q": None, "qo": None, "k": None, "v": None, "kp": None, "vp": None}]:
        assert rope(L, s, **kw) == INVALID, (kw, err(L))
    axis = np.zeros(64, np.uint8)
    axis[63] = 1
    assert rope(L, s, axis=axis.ctypes.data) == INVALID and "axis_of" in err(L)
    assert rope(L, s, n=0) == 0  # nothing to do
    with pytest.raises(ValueError):
        tpk.kv_rope_append(s, 1, 16, 4096, 16, 512, 16, 512, 16, 1, np.zeros(63, np.uint8), 16, 128, False, 16, 16,
                           4096, 16, 16)


def test_tables_arguments_are_refused(L):
    for kw in [{"n_req": 0}, {"n_req": 4097}, {"max_pages": 0}, {"max_pages": 1 << 25}, {"cap": -1}, {"mt": -1},
               {"n_req": 4096, "max_pages": 1 << 20}, {"cap": 0x7fffffff}, {"mt": 0x7fffffff}, {"old": None},
               {"new": None}, {"table": None}, {"free": None}, {"fin": None}, {"fout": None}, {"out": None},
               {"granted": None}, {"off": None}, {"slot": None}, {"pos": None}, {"req": None}]:
        assert tables(L, **kw) == INVALID, (kw, err(L))


def test_tables_model():
    # 3 free slots (top: 12); request 0 finishes (gives 5, 6), 1 grows two pages, 2 one
    table, free = [[5, 6, -1], [7, -1, -1], [8, -1, -1], [9, -1, -1]], [10, 11, 12, -1, -1, -1]
    out = tables_model([100, 60, 64, 3], [0, 130, 66, 3], table, free, 3, 80)
    n_free, length, granted, off, slot, pos, req = out
    assert n_free == 2 and free[:2] == [10, 11] and granted == [1, 1, 1, 1] and length == [0, 130, 66, 3]
    assert table[1] == [7, 6, 5] and table[2] == [8, 12, -1] and off == [0, 0, 70, 72, 72]
    assert slot[:5] == [7 * 64 + 60, 7 * 64 + 61, 7 * 64 + 62, 7 * 64 + 63, 6 * 64] and slot[70] == 12 * 64
    assert pos[70:73] == [64, 65, 0] and req[69:73] == [1, 2, 2, -1] and slot[72] == -1
    # too few slots: the second of two growing requests is refused and keeps its length
    table, free = [[0, -1], [1, -1]], [2, -1]
    n_free, length, granted, off, slot, pos, req = tables_model([64, 64], [65, 65], table, free, 1, 4)
    assert granted == [1, 0] and length == [65, 64] and slot == [128, -1, -1, -1] and n_free == 0


def test_python_calls_marshal_and_refuse():
    """The C module's conversions: pointers from ints, None and data_ptr(), errors as
    exceptions, statuses as TpkError."""
    class Ptr:
        def data_ptr(self):
            return 16

    class Stream:
        cuda_stream = 0

    s = shape(head_dim=64, group=1, kv_heads=1)
    x = Ptr()
    axis = np.zeros(32, np.uint8)
    good = dict(shape=s, n_tokens=0, q=x, q_stride=64, k=x, k_stride=64, v=x, v_stride=64, positions=x, n_axes=1,
                axis_of=axis, inv_freq=x, rot_dim=64, interleaved=False, slot_map=x, q_out=x, q_out_stride=64, k_pool=x,
                v_pool=16, stream=Stream())
    tpk.kv_rope_append(**good)
    tpk.kv_rope_append(**{**good, "axis_of": None, "stream": None})
    tpk.kv_rope_append(**{**good, "axis_of": axis.tobytes(), "stream": 0})
    for kw, exc in [({"q": "text"}, TypeError), ({"q": 1.5}, TypeError), ({"n_tokens": 1 << 40}, OverflowError),
                    ({"q_stride": "64"}, TypeError), ({"shape": None}, tpk.TpkError), ({"shape": b"short"}, ValueError),
                    ({"axis_of": axis[:31]}, ValueError), ({"axis_of": np.zeros(32, np.int32)}, ValueError),
                    ({"stream": "s"}, AttributeError), ({"rot_dim": 8}, ValueError), ({"k": None}, tpk.TpkError),
                    ({"q": -1}, Exception)]:
        with pytest.raises(exc):
            tpk.kv_rope_append(**{**good, **kw})
    with pytest.raises(tpk.TpkError, match="n_req"):
        tpk.decode_attn_paged(shape(), 0, x, 4096, x, x, x, x, None, x, 4096, False, x, x, BIG)
    with pytest.raises(tpk.TpkError, match="workspace"):
        tpk.cross_attn_paged(shape(), 1, 1, x, 4096, x, x, x, x, x, None, x, 4096, x, x, -1)
    with pytest.raises(tpk.TpkError, match="n_req"):
        tpk.kv_tables_update(0, 4, x, x, x, x, 8, x, x, x, x, x, x, x, x, 10)
