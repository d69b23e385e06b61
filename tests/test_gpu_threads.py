"""Calls from host threads that have made no CUDA call before, in a process that has (what the
library looks up once is there already)."""
import threading

import numpy as np
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from paged_util import Pages
from test_gpu_paged_cross import Cross
from test_gpu_paged_decode import Decode
from tiered_paged_kv_gb300 import synth
from tpk_testutil import DevWorkload, oracle_records

pytestmark = pytest.mark.gpu


def run(*jobs):
    """Runs each job in a thread of its own, all at once; raises what they raised."""
    errors = []

    def guarded(job):
        try:
            job()
        except BaseException as e:  # noqa: B902
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_two_threads():
    """Each on its own stream with its own buffers."""
    sets = []
    for i in (0, 1):
        sets.append([Decode(Pages([900 + i, 33], 2, 128, "bf16", 5 + i), 8), Cross(Pages([500, 64 + i], 2, 128, "bf16", 7 + i), [200, 3], 2),
                     Cross(Pages([64, 500], 2, 64, "f16", 9 + i), [2, 5], 1)])
    streams = [torch.cuda.Stream() for _ in sets]
    for c in sets[0]:
        c.call()
    torch.cuda.synchronize()

    def job(calls, stream):
        for _ in range(50):
            for c in calls:
                c.call(stream)
        with pytest.raises(tpk.TpkError, match="n_req"):
            tpk.decode_attn_paged(calls[0].shape, 0, 16, 64, 16, 16, 16, 16, None, 16, 64, False, 16, 16, 0)

    run(*(lambda c=c, s=s: job(c, s) for c, s in zip(sets, streams)))
    for s in sets:
        for c in s:
            c.check()
    assert tpk.get_device_status(reset=True) == (0, 0)


def test_hybrid():
    w = synth.make_workload([64 * 20 + 7], 512, H=2, seed=43, key_sigma="outliers")
    d = DevWorkload(w, tpk.IMPL_TENSOR)
    d.load_records(oracle_records(w))
    want = d.hybrid()
    o, lse = (torch.full_like(torch.from_numpy(x), float("nan"), dtype=torch.float32, device="cuda") for x in want)
    nbytes = tpk.hybrid_workspace_bytes(d.shape, w.B)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    run(lambda: tpk.decode_hybrid_batched(d.shape, w.B, d.q, d.k, d.v, d.rec, d.pt, d.off, w.n_ex, d.pt8, d.off8, w.n8, o, lse,
                                          ws, nbytes))
    torch.cuda.synchronize()
    assert np.array_equal(o.double().cpu().numpy(), want[0]) and np.array_equal(lse.double().cpu().numpy(), want[1])
