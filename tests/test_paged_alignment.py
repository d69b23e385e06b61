"""Arrays that are not aligned to their elements are refused (no GPU needed: nothing is
launched)."""
import pytest

import tiered_paged_kv_gb300 as tpk
from tiered_paged_kv_gb300 import build

S = tpk.PagedShape(1, 1, 64, kv_slots=4, max_pages=2)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def refused(f, good, names, bad):
    for name in names:
        with pytest.raises(tpk.TpkError, match="align"):
            f(**{**good, name: bad})


def test_tables():
    names = ["len_old", "len_new", "page_table", "free_slots", "n_free_in", "n_free_out", "len_out", "granted", "tok_off",
             "slot_map", "positions", "token_req"]
    good = dict({k: 16 for k in names}, n_req=1, max_pages=2, free_cap=4, max_tokens=3)
    refused(tpk.kv_tables_update, good, names, 18)
    refused(tpk.kv_tables_update, good, ["slot_map"], 20)


def test_rope():
    good = dict(shape=S, n_tokens=2, q=16, q_stride=64, k=16, k_stride=64, v=16, v_stride=64, positions=16, n_axes=1,
                axis_of=None, inv_freq=16, rot_dim=64, interleaved=False, slot_map=16, q_out=16, q_out_stride=64, k_pool=16,
                v_pool=16)
    refused(tpk.kv_rope_append, good, ["positions", "inv_freq", "slot_map"], 17)
    refused(tpk.kv_rope_append, good, ["slot_map"], 20)


def test_attention():
    good = dict(shape=S, n_req=1, q=16, q_stride=64, k_pool=16, v_pool=16, page_table=16, n_tokens=16, tok_begin=16, o=16,
                o_stride=64, o_f32=False, lse=16, ws=16, ws_bytes=1 << 40)
    refused(tpk.decode_attn_paged, good, ["page_table", "n_tokens", "tok_begin", "lse"], 18)
    del good["tok_begin"], good["o_f32"]
    good.update(n_q=1, q_off=16, kv_range=16)
    refused(tpk.cross_attn_paged, good, ["page_table", "n_tokens", "q_off", "kv_range", "lse"], 18)
