"""Steps without tokens: an empty tensor's pointer is null, and the calls that allow a count
of 0 take it (no GPU needed: nothing is launched)."""
import pytest
import torch

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


class Ptr:
    def data_ptr(self):
        return 16


X = Ptr()
S = tpk.PagedShape(2, 4, 64, kv_slots=10, max_pages=3)


def none(*shape, dtype=torch.bfloat16):
    x = torch.empty(0, *shape, dtype=dtype)
    assert x.data_ptr() == 0
    return x


def cross(**kw):
    d = dict(shape=S, n_req=2, n_q=0, q=none(512), q_stride=512, q_off=X, k_pool=X, v_pool=X, page_table=X, n_tokens=X,
             kv_range=none(2, dtype=torch.int32), o=none(512), o_stride=512, lse=none(8, dtype=torch.float32),
             ws=none(dtype=torch.uint8), ws_bytes=0)
    d.update(kw)
    tpk.cross_attn_paged(**d)


def rope(**kw):
    d = dict(shape=S, n_tokens=0, q=none(512), q_stride=512, k=none(128), k_stride=128, v=none(128), v_stride=128,
             positions=none(dtype=torch.int32), n_axes=1, axis_of=None, inv_freq=X, rot_dim=64, interleaved=False,
             slot_map=none(dtype=torch.int64), q_out=none(512), q_out_stride=512, k_pool=X, v_pool=X)
    d.update(kw)
    tpk.kv_rope_append(**d)


def test_no_queries():
    cross()
    cross(kv_range=None, q=X, o=X, lse=X, ws=X, ws_bytes=1 << 30)
    for kw in [{"n_req": 0}, {"n_q": 1}, {"n_q": -1}, {"q_off": None}, {"shape": tpk.PagedShape(2, 4, 64, kv_slots=10)}]:
        with pytest.raises(tpk.TpkError):
            cross(**kw)


def test_no_tokens():
    rope()
    rope(k=X, v=X, slot_map=X)  # queries alone are empty
    rope(rot_dim=0, positions=None, inv_freq=None)
    rope(q=X, q_out=X, k=None, v=None, k_pool=None, v_pool=None, slot_map=None)  # no keys asked for
    for kw in [{"n_tokens": 1}, {"k": X}, {"q": X}, {"k_pool": None}, {"rot_dim": 72}, {"inv_freq": None}, {"n_axes": 0}]:
        with pytest.raises(tpk.TpkError):
            rope(**kw)
