"""Requests as long as a table row can make them: 64 (2^25 - 1) tokens, of which the last
are attended, and positions next to 2^31."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import attention, check_attention

pytestmark = pytest.mark.gpu
PAGES = (1 << 25) - 1


@pytest.mark.parametrize("back", [0, 1, 17, 63])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention(D, back):
    n = 64 * PAGES - back
    gen = torch.Generator().manual_seed(D + back)
    dt = torch.bfloat16
    k, v = (torch.randn(3 * 64, D, generator=gen).to(dt) for _ in range(2))
    k[3 * 64 - back:], v[3 * 64 - back:] = float("nan"), float("inf")
    pools = [x.view(3, 1, 64, D).cuda() for x in (k, v)]
    table = torch.full((1, PAGES), -1, dtype=torch.int32, device="cuda")
    table[0, -3:] = torch.arange(3, dtype=torch.int32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = i32([n])
    s = tpk.PagedShape(1, 2, D, kv_slots=3, max_pages=PAGES)
    last = 3 * 64 - back
    for rows, reach in [(1, 50 - min(back, 40)), (1, 120), (200, 50 - min(back, 40)), (200, 120)]:
        q = torch.randn(rows, 2, D, generator=gen).to(dt)
        o, lse = torch.zeros(rows, 2, D, dtype=dt, device="cuda"), torch.zeros(rows, 2, device="cuda")
        if rows == 1:
            nb = tpk.decode_paged_workspace_bytes(s, 1)
            ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
            tpk.decode_attn_paged(s, 1, q.cuda(), 2 * D, *pools, table, lens, i32([n - reach]), o, 2 * D, False, lse, ws, nb)
        else:
            nb = tpk.cross_paged_workspace_bytes(s, 1, rows)
            ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
            tpk.cross_attn_paged(s, 1, rows, q.cuda(), 2 * D, i32([0, rows]), *pools, table, lens,
                                 i32([[n - reach, n]] * rows), o, 2 * D, lse, ws, nb)
        torch.cuda.synchronize()
        seen = torch.ones(rows, reach, dtype=torch.bool)
        for j in range(2):
            want = attention(q[:, j].double(), k[last - reach:last].double(), v[last - reach:last].double(), seen, D ** -0.5)
            check_attention(o[:, j].cpu(), lse[:, j].cpu(), want, D, reach, dt, one_plane=rows > 1, what=f"{rows} rows, {reach} back")
    assert tpk.get_device_status(reset=True) == (0, 0)


def test_tables():
    old, new = 64 * PAGES - 70, 64 * PAGES
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((1, PAGES), -1, dtype=torch.int32, device="cuda")
    table[0, -2] = 5
    free, nf, lens, off, granted = i32([7, 9]), i32([2]), i32([old]), i32([0, 0]), i32([0])
    slot, pos, req = torch.zeros(72, dtype=torch.int64, device="cuda"), i32([0] * 72), i32([0] * 72)
    tpk.kv_tables_update(1, PAGES, lens, i32([new]), table, free, 2, nf, nf, lens, granted, off, slot, pos, req, 72)
    torch.cuda.synchronize()
    assert granted.item() == 1 and lens.item() == new and off.tolist() == [0, 70] and nf.item() == 1
    assert table[0, -2:].tolist() == [5, 9]
    want = list(range(old, new))
    assert pos.tolist() == want + [0, 0] and req.tolist() == [0] * 70 + [-1, -1]
    assert slot.tolist() == [(5 if p // 64 == PAGES - 2 else 9) * 64 + p % 64 for p in want] + [-1, -1]
