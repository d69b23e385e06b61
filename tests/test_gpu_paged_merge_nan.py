"""tpk_merge_lse carries a NaN partial, alone or beside others, and leaves an empty
accumulator as it is where every partial is empty."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import Pages
from test_gpu_paged_decode import Decode

pytestmark = pytest.mark.gpu
NINF, NAN = float("-inf"), float("nan")


def test_partials():
    gen = torch.Generator().manual_seed(1)
    o = torch.randn(2, 6, 256, generator=gen)
    lse = torch.tensor([[NAN, NAN, 1.0, NINF, NINF, 2.0], [NINF, 0.5, NAN, NINF, NAN, 1.0]])
    o[torch.isnan(lse)] = NAN
    acc, al = torch.zeros(6, 256, device="cuda"), torch.full((6,), NINF, device="cuda")
    tpk.merge_lse(2, 6, 256, o.cuda(), lse.cuda(), acc, al)
    acc, al = acc.cpu(), al.cpu()
    for r in (0, 1, 2, 4):
        assert torch.isnan(acc[r]).all() and torch.isnan(al[r])
    assert (acc[3] == 0).all() and al[3] == NINF
    w = torch.softmax(lse[:, 5].double(), 0)
    want = (w[:, None] * o[:, 5].double()).sum(0)
    # two weights and the log-sum behind them, each within a few float32 roundings
    assert (acc[5].double() - want).abs().max() <= 16 * 2.0 ** -24 * o[:, 5].abs().max()
    assert abs(al[5].double() - torch.logsumexp(lse[:, 5].double(), 0)) <= 8 * 2.0 ** -23


def test_decode_partials_of_a_nan_query():
    """Both halves of a history are NaN for a NaN query, and so is what they fold into."""
    pg = Pages([1500], 2, 256, "bf16", 8)
    first, second = Decode(pg, 8, o_f32=True), Decode(pg, 8, begin=[777], o_f32=True)
    first.dq[0, 3 * 256 + 5] = NAN
    second.dq = first.dq
    first.lens = torch.tensor([777], dtype=torch.int32, device="cuda")
    first.call()
    second.call()
    acc, lse = torch.zeros_like(first.o), torch.full_like(first.lse, NINF)
    tpk.merge_lse(2, 16, 256, torch.stack([first.o, second.o]), torch.stack([first.lse, second.lse]), acc, lse)
    bad = torch.isnan(lse[0]).cpu()
    assert bad.tolist() == [j == 3 for j in range(16)]
    assert torch.equal(torch.isnan(acc[0].view(16, 256)).all(1).cpu(), bad)
