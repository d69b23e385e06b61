"""Frequencies of every size at far positions against angles reduced in exact integers
(1 / 2 pi to 400 bits), and frequencies that are refused.

Bound: that of test_gpu_paged_rope.  The documented angle error, 2^-26 + 2^-31 turns, is
under 2^-23 rad; with sincospif's and the products' it stays below 2^-20 of |a| + |b|."""
import math
from fractions import Fraction

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from test_gpu_paged_rope import close

pytestmark = pytest.mark.gpu
BITS = 400


def inverse_two_pi():
    """floor(2^BITS / (2 pi)) by Machin's formula."""
    one = 1 << (BITS + 40)

    def arctan(n):
        total = term = one // n
        k = 1
        while term:
            term //= n * n
            k += 2
            total += -term // k if k % 4 == 3 else term // k
        return total

    pi = 4 * (4 * arctan(5) - arctan(239))
    return (one << BITS) // (2 * pi)


INV = inverse_two_pi()


def turns(freq, pos):
    """Fraction of a turn of freq * pos in [-1/2, 1/2), a float."""
    f = Fraction(freq) * pos
    t = (f.numerator * INV // f.denominator) % (1 << BITS)
    return float(Fraction(t, 1 << BITS) - (t >> (BITS - 1)))


def test_the_digits():
    assert abs(turns(1.0, 1) - 1 / (2 * math.pi)) < 1e-16 and abs(turns(2.0 ** 20, 1) - (2 ** 20 / (2 * math.pi)) % 1) < 1e-9


FREQ = [1.0, 0.1, 1e-4, 1e-30, 1e-40, 0.0, -0.0, -0.7, 1e3, 123456.7, -1e8, 2.0 ** 31, 3.1e9, 4294967040.0, -4294967040.0, 6.2831855]
POS = [0, 1, -1, 7, 64, 131072, 10 ** 6 + 1, 2 ** 24 + 1, -2 ** 30 - 5, 2 ** 31 - 1, -2 ** 31]


def call(freq, pos, pairs):
    n, rot = len(pos), 2 * len(freq)
    gen = torch.Generator().manual_seed(3)
    q = torch.randn(n, 64, generator=gen).half()
    out = torch.zeros(n, 64, dtype=torch.float16, device="cuda")
    s = tpk.PagedShape(1, 1, 64, dtype=tpk.F16, kv_slots=1)
    tpk.kv_rope_append(s, n, q.cuda(), 64, None, 64, None, 64, torch.tensor(pos, dtype=torch.int32, device="cuda"), 1, None,
                       torch.tensor(freq, dtype=torch.float32, device="cuda"), rot, pairs, None, out, 64, None, None)
    torch.cuda.synchronize()
    x = q.double()
    a, b = (x[:, 0:rot:2], x[:, 1:rot:2]) if pairs else (x[:, :rot // 2], x[:, rot // 2:rot])
    return x, a, b, out.cpu()


@pytest.mark.parametrize("pairs", [False, True])
def test_frequencies(pairs):
    x, a, b, got = call(FREQ, POS, pairs)
    f32 = torch.tensor(FREQ, dtype=torch.float32).tolist()
    t = torch.tensor([[turns(f, p) for f in f32] for p in POS], dtype=torch.float64) * (2 * math.pi)
    y, s = x.clone(), torch.zeros_like(x)
    lo, hi = (slice(0, 32, 2), slice(1, 32, 2)) if pairs else (slice(0, 16), slice(16, 32))
    y[:, lo], y[:, hi] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    s[:, lo] = s[:, hi] = a.abs() + b.abs()
    close(got, y, s, torch.float16)


def test_others_are_refused():
    bad = [2.0 ** 32, -2.0 ** 32, 1e10, 3e38, float("inf"), float("-inf"), float("nan"), 1.5]
    x, a, b, got = call(bad, POS, True)
    pair = got.view(len(POS), 32, 2)
    assert torch.isnan(pair[:, :7]).all() and not torch.isnan(pair[:, 7:]).any()
    assert tpk.get_device_status(reset=True) == (0, 0)
