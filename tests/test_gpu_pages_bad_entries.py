"""Forks of batches whose stack of free slots, or whose lengths, hold what they should not: no slot from
outside the pool is handed out, and the device status tells."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fork(source, lens, table, free, slots, keep=None, wide=False):
    """Returns what the call left as lists; `wide`: a pool that goes to a cluster, not to one block."""
    n, max_pages = len(lens), len(table[0])
    slots = 9000 if wide else slots
    d = {k: i32(v) for k, v in dict(source=source, lens=lens, table=table, free=free, n_free=[len(free)]).items()}
    shares = torch.zeros(slots, dtype=torch.int32, device="cuda")
    out = torch.full((n, max_pages), -9, dtype=torch.int32, device="cuda")
    lo, granted, cs, cd = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(4))
    size = tpk.kv_pages_workspace_bytes(slots, n)
    ws = torch.randint(0, 255, (size,), dtype=torch.uint8, device="cuda")
    tpk.kv_pages_fork(n, max_pages, slots, d["source"], d["lens"], None if keep is None else i32(keep), d["table"], out, shares, shares,
                      d["free"], len(free), d["n_free"], d["n_free"], lo, granted, cs, cd, ws, size,
                      stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return dict(rows=out.tolist(), len=lo.tolist(), granted=granted.tolist(), src=cs.tolist(), dst=cd.tolist(),
                n_free=d["n_free"].item(), shares=shares.tolist()[:6], status=tpk.get_device_status(reset=True))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("entry", [-1, -7, -2 ** 31, 9000, 2 ** 31 - 1])
def test_stack_entries_outside_the_pool_are_no_slots(entry, wide):
    # three copies of page 1 wanted: the second request takes slot 5, the third the bad entry, the fourth slot 4
    got = fork([0, 0, 0, 0], [70, 0, 0, 0], [[0, 1]] + [[-1, -1]] * 3, [3, 4, entry, 5], 6, wide=wide)
    assert got["status"] == (4, 1)
    assert got["granted"] == [1, 1, 0, 1] and got["len"] == [70, 70, 64, 70]
    assert got["src"] == [-1, 1, -1, 1] and got["dst"] == [-1, 5, -1, 4]
    assert got["rows"] == [[0, 1], [0, 5], [0, -9], [0, 4]]  # the refused one does not name the others' open page
    assert got["n_free"] == 1 and got["shares"] == [3, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("wide", [False, True])
def test_bad_entries_that_nobody_takes(wide):
    got = fork([0, 0], [70, 0], [[0, 1], [-1, -1]], [-1, 7000000, 2], 6, wide=wide)
    assert got["granted"] == [1, 1] and got["dst"] == [-1, 2] and got["n_free"] == 2 and got["status"] == (0, 0)


@pytest.mark.parametrize("wide", [False, True])
def test_lengths_out_of_range_are_cut(wide):
    """A length past the row counts as the whole row, one below 0 as none; the status tells.  What a request
    asks for of such a history goes by the length that it was cut to."""
    got = fork([1, 1, 0], [200, -3, 10], [[0, 1], [2, 3], [4, 5]], [], 6, wide=wide)
    assert got["status"] == (4, 1)
    assert got["len"] == [0, 0, 128] and got["granted"] == [1, 1, 1]
    assert got["rows"][2] == [0, 1] and got["shares"] == [0] * 6
    got = fork([0, 0], [200, 64], [[0, 1], [2, 3]], [], 6, keep=[129, 128], wide=wide)
    assert got["status"] == (4, 1) and got["granted"] == [0, 1] and got["len"] == [128, 128]
