"""What may be captured first: after one uncaptured call of a head size and type, a capture
may launch any other form of the attention calls, and after one call of the tables and of
the rotary store any other of theirs.  Each in a process of its own, which has launched
nothing else."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

HEAD = """
import sys
sys.path[:0] = [{here!r}, {root!r}]
import torch
import tiered_paged_kv_gb300 as tpk
from paged_util import Pages
from test_gpu_paged_cross import Cross
from test_gpu_paged_decode import Decode

def captured(calls):
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        for c in calls:
            c(torch.cuda.current_stream())
    g.replay()
    torch.cuda.synchronize()
"""

ATTENTION = """
D, first = {D}, {first!r}
forms = [Decode(Pages([5000, 70], 1, D, "bf16", 1), 8), Decode(Pages([300, 64], 2, D, "bf16", 2), 3),
         Decode(Pages([(i * 37) % 300 for i in range(60)], 4, D, "bf16", 3, max_pages=5), 16),
         Decode(Pages([(i * 137) % 700 for i in range(110)], 4, D, "bf16", 4), 3),
         Decode(Pages([(i * 379) % 1500 for i in range(12)], 4, D, "bf16", 5), 20),
         Cross(Pages([3000, 64], 1, D, "bf16", 6), [4, 3], 2), Cross(Pages([300, 70], 64, D, "bf16", 7), [200, 150], 1),
         Cross(Pages([2000, 700], 1, D, "bf16", 8), [300, 20], 2), Cross(Pages([1500] * 9, 8, D, "bf16", 9), [900] * 9, 1)]
warm = Decode(Pages([10], 1, D, "bf16", 0), 1) if first == "decode" else Cross(Pages([10], 1, D, "bf16", 0), [1], 1)
warm.call()
captured([f.call for f in forms])
for i, f in enumerate(forms):
    f.check(str(i))
assert tpk.get_device_status(reset=True) == (0, 0)
"""

STORE = """
import test_gpu_paged_rope as rope
import test_gpu_paged_tables as tables
rope.case(5, 1, 1, 64, 64, 1, False, "bf16")
tables.check([1], [2], [[0, -1]], [4, 5], 2, 5)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
n = 40
T = 100 * n
old, new, table, free, nf = i32([0] * n), i32([100] * n), i32([[-1, -1]] * n), i32(list(range(2 * n))), i32([2 * n])
granted, off = i32([9] * n), i32([9] * (n + 1))
slot, pos, req = torch.zeros(T, dtype=torch.int64, device="cuda"), i32([9] * T), i32([9] * T)
x = torch.randn(T, 128, device="cuda").half()
kp, vp = (torch.zeros(2 * n, 1, 64, 128, dtype=torch.float16, device="cuda") for _ in range(2))
out = torch.zeros_like(x)
freq = torch.zeros(64, device="cuda")
s = tpk.PagedShape(1, 1, 128, dtype=tpk.F16, kv_slots=2 * n)
captured([lambda st: tpk.kv_tables_update(n, 2, old, new, table, free, 2 * n, nf, nf, old, granted, off, slot, pos, req, T,
                                          stream=st),
          lambda st: tpk.kv_rope_append(s, T, x, 128, x, 128, x, 128, pos, 1, None, freq, 128, True, slot, out, 128, kp, vp,
                                        stream=st)])
assert granted.tolist() == [1] * n and off.tolist() == [100 * i for i in range(n + 1)] and nf.item() == 0
assert torch.equal(out, x) and torch.equal(vp.view(-1, 128)[slot], x) and torch.equal(kp.view(-1, 128)[slot], x)
assert tpk.get_device_status(reset=True) == (0, 0)
"""


def child(code, **kw):
    r = subprocess.run([sys.executable, "-c", (HEAD + code).format(here=HERE, root=os.path.dirname(HERE), **kw)],
                       capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


@pytest.mark.parametrize("first", ["decode", "cross"])
@pytest.mark.parametrize("D", [64, 256])
def test_attention(D, first):
    child(ATTENTION, D=D, first=first)


def test_tables_and_store():
    child(STORE)
