"""Lists of page copies that the launch could not number in 32 bits are refused on the host (no GPU needed)."""
import ctypes

import pytest

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build
from test_paged_args import INVALID, err, shape

MOST = 0x7fffffff - 16384


@pytest.fixture(scope="module")
def L():
    build.build()
    return tpk.lib()


@pytest.mark.parametrize("n", [MOST + 1, 0x7fffffff - 2047, 0x7fffffff])
def test_lists_next_to_32_bits_are_refused(L, n):
    pool = (ctypes.c_void_p * 1)(16)
    s = shape()
    assert L.tpk_kv_pages_copy(ctypes.byref(s), 1, pool, pool, n, 16, 16, None) == INVALID
    assert "n_pages" in err(L)
