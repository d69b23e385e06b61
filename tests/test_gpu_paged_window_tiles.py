"""Row tiles through windows, with pages between the first tokens and the window that nobody sees: one and two
128-row tiles that share the keys.  Which kernel takes a call goes by sizes, so that each case says which it
means: the workspace that the call asks for tells row tiles whose keys are not split from the rest (256
bytes), and two tiles are taken where one would need more than 1.5 times the waves of 152 items."""
import re

import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import Pages
from test_gpu_paged_cross import Cross
from test_gpu_paged_wait_limit import stalled
from test_gpu_paged_window import Window

pytestmark = pytest.mark.gpu

SPLIT = "split"  # the other kernel's


def asked(c):
    """Bytes of workspace that the call asks for: a call without any is refused before its launch."""
    n, c.nbytes = c.nbytes, 0
    try:
        c.call()
    except tpk.TpkError as e:
        return int(re.search(r"< (\d+) required", str(e)).group(1))
    finally:
        c.nbytes = n
    raise AssertionError("taken without a workspace")


def tiles_of(c):
    """Row tiles of a block, by the rule on waves; only for calls that row tiles take."""
    each, H = -(-c.T // len(c.nq)), c.pg.H
    waves = lambda t: -(-len(c.nq) * -(-each // (t * (128 // c.G))) * H // 152)  # noqa: E731
    return 1 if c.pg.D == 256 or 2 * waves(1) <= 3 * waves(2) else 2


def window(nq, lens, H, G, D, dtype, win, sinks, tiles, unsplit=True, **kw):
    c = Window(Pages(lens, H, D, dtype, win % 100), nq, G, win, sinks, **kw)
    assert tiles_of(c) == tiles
    assert (asked(c) == 256) == unsplit
    return c


def gap(c):
    """Some page between the first tokens and a window is not seen by anybody."""
    return any(not s[:, i:i + 64].any() for s in c.seen for i in range(64, s.shape[1] - 128, 64))


TWO = [([200, 150], [700, 600], 90, 70), ([200, 150], [700, 600], 90, 0), ([130, 260], [1000, 900], 300, 4), ([1, 400], [900, 1200], 64, 130),
       ([300, 20], [1500, 64], 1, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq,lens,win,sinks", TWO)
def test_two_tiles_across_the_gap(nq, lens, win, sinks, D, dtype):
    c = window(nq, lens, 64, 1, D, dtype, win, sinks, 2)
    assert gap(c)
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == (0, 0)


@pytest.mark.parametrize("D", [64, 128])
def test_two_tiles_bad_pages_and_strides(D):
    c = window([200, 150], [700, 600], 64, 1, D, "bf16", 150, 70, 2, mute=[(0, 1), (0, 8), (1, 0), (1, 7)], q_gap=8, o_gap=24, lead=2,
               tail=3)
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == (4, 1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq,lens,win,sinks", TWO[::2])
def test_two_tiles_waits_are_bounded(nq, lens, win, sinks, D):
    stalled(window(nq, lens, 64, 1, D, "bf16", win, sinks, 2))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("win,sinks", [(60, 4), (64, 70), (1, 0), (100, 130)])
def test_one_tile_narrow_windows(win, sinks, D):
    """Keys in parts, the first tokens in one of them."""
    c = window([300, 200], [900, 640], 2, 8, D, "bf16", win, sinks, 1, unsplit=False)
    assert gap(c) and asked(c) != asked_by_one_row(D)
    c.call()
    c.check()
    assert tpk.get_device_status(reset=True) == (0, 0)


def asked_by_one_row(D):
    """What the split kernel asks for."""
    return asked(Window(Pages([30], 2, D, "bf16", 0), None, 8, 5, 0))


def causal(pg, nq, G):
    a = Window(pg, nq, G, 0, 0)
    b = Cross(pg, nq, G, ranges=[(0, n - c + i + 1) for n, c in zip(pg.lens, nq) for i in range(c)])
    b.dq.copy_(a.dq)
    a.call()
    b.call()
    torch.cuda.synchronize()
    return a, b


@pytest.mark.parametrize("D", [64, 128])
def test_a_window_of_everything_in_two_tiles_is_the_causal_prompt(D):
    """Two threads a row in both: the same sums in the same order, bit for bit."""
    a, b = causal(Pages([400, 150], 64, D, "bf16", 3), [200, 150], 1)
    assert tiles_of(a) == 2 and asked(a) == 256
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("D", [128, 256])
def test_a_window_of_everything_in_one_tile_is_the_causal_prompt_to_rounding(D):
    """Four threads a row against two, in another order: both within the bounds of the formula."""
    a, b = causal(Pages([700, 200], 2, D, "bf16", 3), [300, 200], 8)
    assert tiles_of(a) == 1 and asked(a) != asked_by_one_row(D)
    a.check()
    a.o, a.lse = b.o, b.lse
    a.check()
