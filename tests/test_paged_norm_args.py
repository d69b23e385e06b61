"""The rotary store with norms refuses bad arguments on the host (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build
from test_paged_args import BAD_SHAPES, INVALID, err, shape


@pytest.fixture(scope="module")
def L():
    build.build()
    return tpk.lib()


def norm(L, s, n=5, q=16, qs=4096, k=16, ks=512, v=16, vs=512, wq=16, wk=16, eps=1e-6, pos=16, axes=1, axis=None, freq=16,
         rot=128, pairs=0, slot=16, qo=16, qos=4096, kp=16, vp=16):
    return L.tpk_kv_norm_rope_append(ctypes.byref(s) if s else None, n, q, qs, k, ks, v, vs, wq, wk, eps, pos, axes, axis, freq,
                                     rot, pairs, slot, qo, qos, kp, vp, None)


@pytest.mark.parametrize("kw,code", BAD_SHAPES, ids=lambda x: str(x))
def test_shapes_are_refused(L, kw, code):
    assert norm(L, shape(**kw)) == code, err(L)
    assert norm(L, None) == INVALID


def test_arguments_are_refused(L):
    s = shape()
    for kw in [{"n": -1}, {"rot": 130}, {"rot": 144}, {"rot": -16}, {"rot": 8}, {"pairs": 2}, {"q": None}, {"qo": None},
               {"k": None}, {"v": None}, {"kp": None}, {"vp": None}, {"slot": None}, {"pos": None}, {"freq": None},
               {"axes": 0}, {"axes": 5}, {"qs": 4088}, {"qos": 4090}, {"ks": 504}, {"vs": 511}, {"q": 8}, {"k": 24},
               {"v": 4}, {"qo": 8}, {"kp": 8}, {"vp": 8}, {"qs": 8192}, {"wq": 8}, {"wk": 2}, {"eps": -1e-6},
               {"eps": float("nan")}, {"eps": float("inf")}, {"slot": 4}, {"pos": 2}, {"freq": 2},
               {"q": None, "qo": None, "k": None, "v": None, "kp": None, "vp": None}]:
        assert norm(L, s, **kw) == INVALID, (kw, err(L))
    axis = np.zeros(64, np.uint8)
    axis[63] = 1
    assert norm(L, s, axis=axis.ctypes.data) == INVALID and "axis_of" in err(L)
    assert norm(L, s, n=0) == 0 and norm(L, s, n=0, wq=None, wk=None, eps=0.0) == 0


def test_python_call_marshals():
    s = shape(head_dim=64, group=1, kv_heads=1)
    good = dict(shape=s, n_tokens=0, q=16, q_stride=64, k=16, k_stride=64, v=16, v_stride=64, q_weight=16, k_weight=None, eps=1e-5,
                positions=16, n_axes=1, axis_of=None, inv_freq=16, rot_dim=64, interleaved=False, slot_map=16, q_out=16,
                q_out_stride=64, k_pool=16, v_pool=16)
    tpk.kv_norm_rope_append(**good)
    tpk.kv_norm_rope_append(**{**good, "eps": 0})
    for kw, exc in [({"eps": "x"}, TypeError), ({"eps": -1.0}, tpk.TpkError), ({"q_weight": 1.5}, TypeError),
                    ({"axis_of": np.zeros(31, np.uint8)}, ValueError), ({"shape": None}, tpk.TpkError)]:
        with pytest.raises(exc):
            tpk.kv_norm_rope_append(**{**good, **kw})
