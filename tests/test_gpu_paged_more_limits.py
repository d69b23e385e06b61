"""Windows, shared prefixes, normed heads and shared pages at their limits: captured first, the
longest requests, the largest head counts, steps of several calls replayed."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import PAGE, Pages, attention, check_attention
from test_gpu_paged_capture import child
from test_gpu_paged_last_tokens import PAGES
from test_gpu_paged_norm import case as norm_case
from test_gpu_paged_shared import Shared
from test_gpu_paged_shared import run as run_shared
from test_gpu_paged_window import Window
from test_gpu_paged_window import run as run_window

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


ATTENTION = """
from test_gpu_paged_shared import Shared
from test_gpu_paged_window import Window
D, first = {D}, {first!r}
forms = [Window(Pages([5000, 70], 1, D, "bf16", 1), None, 8, 900, 4), Window(Pages([300, 64], 2, D, "bf16", 2), None, 3, 50, 0),
         Window(Pages([5000, 70], 1, D, "bf16", 1), None, 20, 900, 4), Window(Pages([3000, 64], 1, D, "bf16", 6), [4, 3], 2, 900, 70),
         Window(Pages([300, 170], 64, D, "bf16", 7), [200, 150], 1, 90, 4), Window(Pages([2000, 700], 1, D, "bf16", 8), [300, 20], 2, 0, 0),
         Window(Pages([(i * 37) % 300 for i in range(60)], 4, D, "bf16", 3, max_pages=5), None, 2, 100, 3),
         Shared([(200, [230, 260])], 2, 2, D, "bf16"), Shared([(200, [230, 260])], 2, 4, D, "bf16", max_pages=20000),
         Shared([(200, [230] * 9)], 2, 20, D, "bf16"), Shared([(2000, [2030] * 40), (60, [70, 80])], 2, 8, D, "bf16")]
warm = dict(decode=lambda: Decode(Pages([10], 1, D, "bf16", 0), 1), cross=lambda: Cross(Pages([10], 1, D, "bf16", 0), [1], 1),
            window=lambda: Window(Pages([10], 1, D, "bf16", 0), None, 1, 5, 0), shared=lambda: Shared([(9, [10])], 1, 1, D, "bf16"))[first]()
warm.call()
captured([f.call for f in forms])
for i, f in enumerate(forms):
    f.check(str(i))
assert tpk.get_device_status(reset=True) == (0, 0)
"""

PAGES_CALLS = """
import test_gpu_pages as pages
import test_gpu_paged_norm as norm
norm.case(5, 1, 1, 64, 64, False, "bf16")
pages.fork([0, 0], [10, 0], None, [[0], [-1]], [0, 0], [1, -1], 1, wide=False)
pages.compact([10], [[1]], [0, 0], [0], 1, 1, wide=False)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kp = torch.arange(9000, dtype=torch.int16, device="cuda").view(-1, 1, 1, 1).expand(9000, 1, 64, 64).contiguous()
vp = kp.clone()
s = tpk.PagedShape(1, 1, 64, kv_slots=9000)
tpk.kv_pages_copy(s, [kp], [vp], 1, i32([3]), i32([4]))
n, slots = 3, 9000  # more slots than one block takes
source = i32([0, 0, 0])
z = lambda *k: torch.full(k, -1, dtype=torch.int32, device="cuda")
size = tpk.kv_pages_workspace_bytes(slots, n)
ws = torch.empty(size, dtype=torch.uint8, device="cuda")
table, out, shares, free = i32([[8000], [-1], [-1]]), z(n, 1), i32([0] * slots), i32([5, 6])
nf, lens, granted, src, dst = i32([2]), i32([10, 0, 0]), z(n), z(n), z(n)
captured([lambda st: tpk.kv_pages_fork(n, 1, slots, source, lens, None, table, out, shares, shares, free, 2, nf, nf, lens, granted, src,
                                       dst, ws, size, stream=st),
          lambda st: tpk.kv_pages_copy(s, [kp], [vp], n, src, dst, stream=st)])
assert out[:, 0].tolist() == [8000, 6, 5] and (kp[[5, 6], 0, 0, 0] == 8000).all() and (vp[[5, 6], 0, 63, 63] == 8000).all()
assert nf.item() == 0 and granted.tolist() == [1, 1, 1]
assert tpk.get_device_status(reset=True) == (0, 0)
"""


@pytest.mark.parametrize("first", ["decode", "cross", "window", "shared"])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_captured_first(D, first):
    child(ATTENTION, D=D, first=first)


def test_pages_and_norms_captured_first():
    child(PAGES_CALLS)


def last_pages(D, back, seed):
    """The last three pages of the longest request a table row can have, and its first one."""
    n = PAGE * PAGES - back
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16
    k, v = (torch.randn(4 * PAGE, D, generator=gen).to(dt) for _ in range(2))
    k[4 * PAGE - back:], v[4 * PAGE - back:] = float("nan"), float("inf")
    pools = [x.view(4, 1, PAGE, D).cuda() for x in (k, v)]
    table = torch.full((1, PAGES), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    table[0, -3:] = torch.arange(1, 4, dtype=torch.int32)
    return n, gen, k[:4 * PAGE - back].double(), v[:4 * PAGE - back].double(), pools, table


@pytest.mark.parametrize("back", [0, 17, 63])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_windows_at_the_last_tokens(D, back):
    n, gen, k, v, pools, table = last_pages(D, back, D + back)
    s = tpk.PagedShape(1, 2, D, kv_slots=4, max_pages=PAGES)
    t = torch.cat([torch.arange(PAGE), torch.arange(n - (3 * PAGE - back), n)])  # the tokens that there are
    for rows, window, sinks, offsets in [(1, 60, 5, False), (1, 128, 64, True), (60, 65, 0, True), (70, 55, 40, True)]:
        q = torch.randn(rows, 2, D, generator=gen).to(torch.bfloat16)
        o, lse = torch.zeros(rows, 2, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, 2, device="cuda")
        nb = tpk.window_paged_workspace_bytes(s, 1, rows)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
        tpk.window_attn_paged(s, 1, rows, window, sinks, q.cuda(), 2 * D, i32([0, rows]) if offsets else None, *pools, table, i32([n]), o,
                              2 * D, lse, ws, nb)
        torch.cuda.synchronize()
        x = torch.arange(n - rows, n)[:, None]
        seen = (t <= x) & ((t > x - window) | (t < sinks))
        assert seen.sum(1).tolist() == [window + sinks] * rows  # the test's own: every visible token is there
        for j in range(2):
            want = attention(q[:, j].double(), k, v, seen, D ** -0.5)
            check_attention(o[:, j].cpu(), lse[:, j].cpu(), want, D, 4 * PAGE, torch.bfloat16, one_plane=offsets, what=f"{rows} rows")
    assert tpk.get_device_status(reset=True) == (0, 0)


@pytest.mark.parametrize("H,G,D", [(1024, 1, 64), (512, 2, 128), (1, 128, 256), (3, 127, 64)])
def test_the_largest_head_counts(H, G, D):
    run_window(None, [70, 0, 130], H, G, D, "bf16", 50, 3)
    run_window([3, 1, 60], [70, 5, 130], H, G, D, "f16", 20, 3)
    run_shared([(64, [70, 130])], H, G, D, "bf16")


def test_norms_of_the_largest_head_counts():
    norm_case(2, 1024, 64, 64, 64, False, "bf16", seed=1, axes=2)
    norm_case(3, 1, 128, 256, 256, True, "f16", seed=2, gap=8, axes=4)
    norm_case(9, 1024, 1, 64, 32, False, "f16", seed=3)


def test_requests_without_a_group_and_groups_without_requests():
    run_shared([(64, []), (70, []), (50, [60, 70]), (9, [])] + [(5, [])] * 60, 1, 2, 64, "bf16", alone=(3, 0, 100))
    run_shared([(64, [])] * 300 + [(50, [60, 70] * 20)], 1, 20, 64, "bf16", alone=(3, 0, 100))


def test_two_graphs_with_workspaces_of_their_own_on_two_streams():
    """Replayed at once: nothing is shared but the inputs."""
    a = Window(Pages([3000, 64, 700], 2, 128, "bf16", 1), None, 4, 500, 9)
    b = Shared([(900, [950, 1000, 901])], 2, 4, 128, "bf16")
    graphs = []
    for c in (a, b):
        c.call()
        torch.cuda.synchronize()
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            for _ in range(20):
                c.call(stream=torch.cuda.current_stream())
        graphs.append((g, st))
    for _ in range(10):
        for g, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    a.check()
    b.check()
    assert tpk.get_device_status(reset=True) == (0, 0)
