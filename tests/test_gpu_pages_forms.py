"""Forks and compaction on both sides of the sizes at which one block hands over to a cluster, and the largest
calls of each form, against the plain models."""
import random

import pytest
import torch  # noqa: F401

from test_gpu_pages import compact, fork, random_family

pytestmark = pytest.mark.gpu

# one block up to kv_slots + 40 requests = 9,200 (forks), kv_slots + 14 requests = 8,000 (compaction), 8,192 slots,
# and 32,768 places of the table


@pytest.mark.parametrize("n,slots,max_pages", [(200, 1200, 5), (200, 1201, 5), (25, 8192, 60), (26, 8192, 60), (225, 200, 1),
                                               (229, 60, 1), (8, 8193, 900), (16, 4000, 2048), (16, 4000, 2049), (1, 8192, 8000)])
def test_forks(n, slots, max_pages):
    rng = random.Random(n + slots)
    pages = min(max_pages, slots // (2 * n)) if n > 1 else 6000
    lens, table, shares, free, n_free = random_family(rng, n, max_pages, n // 4, 64 * pages)
    lens = lens if n > 1 else [64 * 5000 + 9]
    if n == 1:
        table, shares, free, n_free = [list(range(5001)) + [-1] * (max_pages - 5001)], [0] * slots, list(range(5001, slots)) + [-5] * 9, slots - 5001
    assert len(shares) <= slots
    shares = shares + [0] * (slots - len(shares))
    source = [rng.choice([b, rng.randrange(n), rng.randrange(n), -1]) for b in range(n)]
    keep = [lens[s] if rng.random() < 0.5 else rng.randint(0, lens[s]) if s >= 0 else 0 for s in source]
    fork(source, lens, keep, table, shares, free, n_free, wide=False, in_place=n % 2 == 0)


@pytest.mark.parametrize("n,slots,max_pages", [(100, 6600, 30), (100, 6601, 30), (500, 1000, 1), (500, 1001, 1), (2, 7972, 3000),
                                               (2, 7973, 3000), (16, 3000, 2048), (16, 3000, 2049)])
def test_compactions(n, slots, max_pages):
    rng = random.Random(n + slots)
    lens, table, shares, free, n_free = random_family(rng, n, max_pages, n // 4, 64 * min(max_pages, max(1, slots // (2 * n))))
    used = {x for b in range(n) for x in table[b][:-(-lens[b] // 64)]}
    assert len(shares) <= slots
    stack = [x for x in range(slots) if x not in used]
    rng.shuffle(stack)
    shares = [s if x in used else 0 for x, s in enumerate(shares)] + [0] * (slots - len(shares))
    compact(lens, table, shares, stack, len(stack), rng.choice([slots, 7]), wide=False, in_place=slots % 2 == 0)
