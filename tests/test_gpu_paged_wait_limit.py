"""Bounded device waits of the paged attention kernels.  With a short limit and one block
whose first page (or key tile) is neither copied nor signalled, every role of the block gives
up, what it did copy lands, the call returns and the status word says so; the next call is
right."""
import time

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import Pages
from test_gpu_paged_cross import Cross
from test_gpu_paged_decode import Decode

pytestmark = pytest.mark.gpu

TPK_ERR_TIMEOUT = 6
LIMIT_NS = 1_000_000  # 1 ms


def stalled(c, unit=0):
    c.call()
    c.check("before")
    assert tpk.get_device_status(reset=True)[0] in (0, 4)
    tpk.set_test_wait(LIMIT_NS, unit)
    try:
        t0 = time.perf_counter()
        c.call()
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        tpk.set_test_wait()
    st, flags = tpk.get_device_status(reset=True)
    assert st == TPK_ERR_TIMEOUT and flags & 2, (st, flags)
    # some waits of 1 ms ran out one after the other; the default limit would take far longer
    assert dt < 1.0, dt
    for x in (c.o, c.lse):
        x.fill_(float("nan"))
    c.call()
    c.check("after")
    assert tpk.get_device_status(reset=True)[0] in (0, 4)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,H,G,pages,unit", [([500, 40], 1, 4, None, 0), ([30], 2, 4, None, 1), ([9000], 1, 8, None, 3),
                                                 ([3000, 10, 900], 2, 20, None, 0),
                                                 ([(i * 37) % 400 + 1 for i in range(300)], 1, 2, 40, 5)],
                         ids=lambda x: f"{len(x)}x{max(x)}" if isinstance(x, list) else str(x))
def test_decode(lens, H, G, pages, unit, D):
    stalled(Decode(Pages(lens, H, D, "bf16", 3, max_pages=pages), G), unit)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,lens,H,G,mute", [([4, 3], [5000, 64], 1, 2, []), ([200, 150], [1300, 70], 64, 1, []),
                                              ([300, 20], [2000, 700], 1, 2, [(0, 3)]), ([100], [30], 4, 1, []),
                                              ([513, 700], [400, 1000], 16, 4, [(1, 0), (1, 15)])],
                         ids=lambda x: "-".join(map(str, x)) if isinstance(x, list) and x and isinstance(x[0], int) else None)
def test_cross(nq, lens, H, G, mute, D):
    stalled(Cross(Pages(lens, H, D, "bf16", 4), nq, G, mute=mute))
