"""What the C module takes for a shape, and how it is built and found (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


class Sub(tpk.PagedShape):
    pass


GOOD = dict(kv_heads=1, group=1, head_dim=64, kv_slots=4, max_pages=2)
SIZE = ctypes.sizeof(tpk.PagedShape)


def calls(shape):
    return [lambda: tpk.kv_rope_append(shape, 0, None, 64, None, 64, None, 64, None, 1, None, None, 0, False, None, None, 64,
                                       None, None),
            lambda: tpk.cross_attn_paged(shape, 1, 0, None, 64, 16, None, None, None, None, None, None, 64, None, None, 0)]


def refused(shape):
    return calls(shape) + [lambda: tpk.decode_attn_paged(shape, 0, 16, 64, 16, 16, 16, 16, None, 16, 64, False, 16, 16, 0)]


@pytest.mark.parametrize("cls", [tpk.PagedShape, Sub])
def test_a_shape(cls):
    for f in calls(cls(**GOOD)):
        f()


@pytest.mark.parametrize("other", [bytes(SIZE), bytes(tpk.PagedShape(**GOOD)), np.ones(SIZE, np.uint8), (ctypes.c_int64 * 16)(),
                                   (tpk.PagedShape * 2)(), tpk.Shape(4, kv_slots=4, rec_slots=4), "shape", 16, object()],
                         ids=lambda x: type(x).__name__)
def test_anything_else_is_refused(other):
    for f in refused(other):
        with pytest.raises((TypeError, ValueError)):
            f()


def test_a_module_per_python_version():
    import importlib.machinery
    assert build.CALL.endswith(importlib.machinery.EXTENSION_SUFFIXES[0]) and "cpython-3" in build.CALL


def test_without_the_headers_the_other_calls_are_built(tmp_path, monkeypatch):
    """No Python.h: the library is built all the same, and the calls that need the module say so."""
    monkeypatch.setattr(build.sysconfig, "get_path", lambda *a, **k: str(tmp_path))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "_tpk_call.so"))
    monkeypatch.setattr(tpk, "_call", None)
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build() == build.LIB
    assert tpk.lib().tpk_version()
    assert tpk.decode_paged_workspace_bytes(tpk.PagedShape(**GOOD), 1) > 0
    with pytest.raises(RuntimeError, match="Python.h"):
        tpk.decode_attn_paged(tpk.PagedShape(**GOOD), 0, 16, 64, 16, 16, 16, 16, None, 16, 64, False, 16, 16, 0)
