"""Refusals of the streaming operators' outputs that share bytes with what a call reads (host only: nothing is launched)."""
import ctypes

import pytest

import head_wise_dynamic_b200 as hw
from head_wise_dynamic_b200 import streaming as st

P = 1 << 30  # a well-aligned address that is never read
FAR = P + (1 << 28)


def _rope(**kw):
    a = dict(n_tokens=8, n_heads=2, n_rot_heads=2, x=P, x_token_stride=384, x_head_stride=64, out=FAR, out_token_stride=384,
             out_head_stride=64, x_is_fp32=0, out_is_fp32=0, pos=FAR, inverse=0)
    a.update(kw)
    cfg = hw.make_rope((32, 32))
    return hw.lib().saf3r_rope(ctypes.byref(cfg), ctypes.byref(st.saf3r_rope_args(**a)), None)


@pytest.mark.parametrize("kw", [dict(out=P + 16), dict(out=P - 16), dict(out=P + 128), dict(out=P + 112 + 128), dict(out=P + 768),
                                dict(out=P + 7 * 768 + 112), dict(out=P - 7 * 768 + 112), dict(out=P, out_is_fp32=1),
                                dict(out=P, out_head_stride=128), dict(out=P + 256, out_token_stride=512),
                                dict(out=P + 128, n_tokens=1), dict(out=P + 16, x_head_stride=0, n_tokens=1),
                                dict(x_token_stride=0, out=P + 112), dict(out=P + 128, out_is_fp32=1, out_token_stride=192)])
def test_rope_refuses_an_output_over_its_input(kw):
    assert _rope(**kw) == hw.ERR_INVALID


CACHE = dict(n_pages=4, n_heads=2, page=64, type=1, k=FAR, v=FAR + (1 << 20), k_scale=FAR + (2 << 20), v_scale=FAR + (3 << 20))
BATCH = dict(n_seqs=1, n_tokens=8, max_new=8, max_pages=2, cu_tokens=P, kv_lens=P, page_table=P)
POOL = 4 * 2 * 64 * 64


def _attn(q=P, out=P + (1 << 20), fp32=0, ts=768, hs=64, out_ts=768, out_hs=64):
    c, b, w = st.saf3r_kv_cache(**CACHE), st.saf3r_kv_batch(**BATCH), st.saf3r_window(4, 2, 4, 1)
    r = st.saf3r_query_rows(4, fp32, q, ts, hs, out, out_ts, out_hs)
    return hw.lib().saf3r_kv_attn(*(ctypes.byref(x) for x in (c, b, w, r)), P, None)


@pytest.mark.parametrize("kw", [dict(out=P + 16), dict(out=P + 1536), dict(out=P + 3 * 128), dict(out=P + 512 - 16),
                                dict(out=P - 7 * 1536 - 112), dict(out=P + 1536 * 5 + 256), dict(out=P + 512, out_ts=512),
                                dict(out=P + 256, fp32=1, out_ts=384), dict(out=P + 128, hs=128, out_hs=192),
                                dict(out=FAR), dict(out=FAR + POOL - 16), dict(out=FAR + (1 << 20) - 16), dict(out=FAR + (2 << 20) + 16),
                                dict(out=FAR + (3 << 20))])
def test_attention_refuses_an_output_over_its_queries_or_the_cache(kw):
    assert _attn(**kw) == hw.ERR_INVALID


@pytest.mark.parametrize("k", [FAR, FAR + POOL - 16, FAR + (1 << 20), FAR - 16, FAR + (2 << 20)])
def test_append_refuses_rows_that_lie_in_the_cache(k):
    c, b = st.saf3r_kv_cache(**CACHE), st.saf3r_kv_batch(**BATCH)
    for rows in [dict(k=k, v=P), dict(k=P, v=k)]:
        r = st.saf3r_kv_rows(k_token_stride=128, k_head_stride=64, v_token_stride=128, v_head_stride=64, pos=None, **rows)
        assert hw.lib().saf3r_kv_append(ctypes.byref(c), ctypes.byref(b), None, ctypes.byref(r), None) == hw.ERR_INVALID
