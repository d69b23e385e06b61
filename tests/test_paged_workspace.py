"""A workspace sized for the largest call of a shape serves every smaller one (no GPU
needed: a call without a workspace is refused and names what it needs)."""
import ctypes
import random
import re

import pytest

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return tpk.lib()


def needed(L, s, n_req, n_q):
    w = s.kv_heads * s.group * s.head_dim
    if n_q is None:
        st = L.tpk_decode_attn_paged(ctypes.byref(s), n_req, 16, w, 16, 16, 16, 16, None, 16, w, 0, 16, 16, 0, None)
    else:
        st = L.tpk_cross_attn_paged(ctypes.byref(s), n_req, n_q, 16, w, 16, 16, 16, 16, 16, None, 16, w, 16, 16, 0, None)
    assert st == 5
    return int(re.search(r"(\d+) required", L.tpk_last_error_string().decode()).group(1))


COUNTS = [1, 2, 3, 4, 5, 8, 9, 13, 16, 17, 31, 32, 33, 50, 64, 65, 100, 127, 128, 129, 200, 255, 300, 512, 700, 1000, 2000, 4095, 4096]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,pages", [(8, 4, 94), (1, 8, 1000), (1, 1, 1), (4, 16, 9), (2, 128, 40), (64, 1, 8), (1, 3, 5000)])
def test_cross(L, D, H, G, pages):
    s = tpk.PagedShape(H, G, D, kv_slots=100, max_pages=pages)
    need = {(r, q): needed(L, s, r, q) for r in COUNTS for q in COUNTS}
    most = {}
    for i, r in enumerate(COUNTS):
        for j, q in enumerate(COUNTS):
            most[r, q] = max(need[r, q], most.get((COUNTS[i - 1], q), 0) if i else 0, most.get((r, COUNTS[j - 1]), 0) if j else 0)
    last = {}
    for i, r in enumerate(COUNTS):
        for j, q in enumerate(COUNTS):
            size = tpk.cross_paged_workspace_bytes(s, r, q)
            assert size >= most[r, q], (r, q)
            assert size >= last.get((r, COUNTS[j - 1]), 0) and size >= last.get((COUNTS[i - 1], q), 0), (r, q)
            last[r, q] = size


def test_random_shapes(L):
    rng = random.Random(5)
    for _ in range(300):
        s = tpk.PagedShape(rng.choice([1, 2, 5, 8, 40]), rng.choice([1, 2, 3, 7, 8, 33, 128]), rng.choice([64, 128, 256]),
                           kv_slots=10, max_pages=rng.choice([1, 3, 8, 9, 32, 33, 313, 100000]))
        r, q = rng.randint(1, 4096), int(2 ** rng.uniform(0, 12))
        size = tpk.cross_paged_workspace_bytes(s, r, q)
        for _ in range(20):
            assert needed(L, s, rng.randint(1, r), rng.randint(1, q)) <= size
        assert needed(L, s, r, None) <= tpk.decode_paged_workspace_bytes(s, r)
        assert tpk.decode_paged_workspace_bytes(s, r) >= tpk.decode_paged_workspace_bytes(s, rng.randint(1, r))


def test_documented_sizes(L):
    """8 requests of 8 x 4 heads of 128 and 94 pages: one size from 16 to 4096 tokens up."""
    s = tpk.PagedShape(8, 4, 128, kv_slots=100, max_pages=94)
    sizes = [tpk.cross_paged_workspace_bytes(s, 8, q) for q in (0, 1, 16, 64, 4096)]
    assert sizes == sorted(sizes) and sizes[-1] < 32 << 20
