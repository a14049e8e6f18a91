"""Streaming operators on the host: the oracle's own checks, argument checks of the entry points
and of their bindings (no GPU: nothing is launched)."""
import ctypes

import numpy as np
import pytest

import head_wise_dynamic_b200 as hw
from head_wise_dynamic_b200 import streaming as st
from oracle import streaming as O

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ the oracle

def test_e4m3_rounding_matches_torch():
    """Every value between two codes, the ties among them, against torch's conversion."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    codes = np.unique(codes[np.isfinite(codes)])
    mids = (codes[1:] + codes[:-1]) / 2
    x = np.concatenate([codes, mids, mids * (1 + 1e-6), mids * (1 - 1e-6), [0.0, 2.0 ** -11, 2.0 ** -10, -2.0 ** -10]])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.round_e4m3(x), want)
    assert np.isnan(O.round_e4m3(np.array([np.inf, -np.inf, np.nan]))).all()
    assert O.round_e4m3(np.array([1e9, -1e9])).tolist() == [448.0, -448.0]


def test_bf16_rounding_matches_torch():
    x = np.random.default_rng(0).standard_normal(4096)
    assert np.array_equal(O.round_bf16(x.astype(np.float32)), torch.from_numpy(x).float().bfloat16().double().numpy())


@pytest.mark.parametrize("m,e", [(448.0, 0), (448.0000001, 1), (0.0, -100), (1e-40, -100), (7.0, -6), (7.1, -5),
                                 (3e38, 119)])
def test_scale_is_the_least_power_of_two_that_fits(m, e):
    assert O.scale_of(m) == 2.0 ** e
    if m > 0 and -100 < e < 119:
        assert m / O.scale_of(m) <= 448 < 2 * m / O.scale_of(m)


@pytest.mark.parametrize("pairing", [O.HALF, O.PAIRS, O.SECTIONS])
def test_rope_adjoint_and_differences(pairing):
    """<R x, y> = <x, R' y>, R' R x = x, and the gradient of <R x, y> by differences is R' y."""
    rng = np.random.default_rng(1)
    dims, pos = (16, 24, 16), rng.integers(-50, 50, (5, 3))
    x, y = rng.standard_normal((2, 5, 2, 64))
    f = lambda z: float((O.rope(z, pos, dims, 100.0, pairing) * y).sum())  # noqa: E731
    g = O.rope(y, pos, dims, 100.0, pairing, inverse=True)
    assert abs(f(x) - float((x * g).sum())) < 1e-11
    assert np.abs(O.rope(O.rope(x, pos, dims, 100.0, pairing), pos, dims, 100.0, pairing, inverse=True) - x).max() < 1e-13
    for i in [(0, 0, 0), (1, 1, 17), (4, 0, 39), (2, 1, 63)]:
        d = np.zeros_like(x)
        d[i] = 1e-4
        assert abs((f(x + d) - f(x - d)) / 2e-4 - g[i]) < 1e-9


def test_rope_pairs_cover_the_rotated_dims_once():
    for dims in [(64,), (32, 32), (16, 24, 24), (8, 8, 8, 8), (40,)]:
        for pairing in (O.HALF, O.PAIRS, O.SECTIONS):
            used = sorted(d for a, b, _, _ in O.rope_pairs(dims, 100.0, pairing) for d in (a, b))
            assert used == list(range(sum(dims)))


def test_window_of_all_views_is_causal_attention():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 12, 64))
    pos = np.arange(12)
    s = q @ k.T / 8
    s[pos[:, None] < pos] = -np.inf
    w = np.exp(s - s.max(1, keepdims=True))
    assert np.allclose(O.attend(q, k, v, pos, 1, 0, 0, True), w / w.sum(1, keepdims=True) @ v, atol=1e-13)
    # a window at least as long changes nothing, nor do sinks inside it; views of 4: block-causal
    assert np.array_equal(O.attend(q, k, v, pos, 1, 12, 3, True), O.attend(q, k, v, pos, 1, 0, 0, True))
    assert O.seen(5, 12, 4, 1, 2, True).tolist() == [True] * 2 + [False] * 2 + [True] * 4 + [False] * 4
    assert O.seen(5, 12, 4, 1, 2, False).tolist() == [True] * 2 + [False] * 2 + [True] * 4 + [False] * 4
    assert O.seen(1, 12, 4, 2, 9, True).tolist() == [True] * 4 + [False] * 8
    assert O.seen(1, 12, 4, 2, 9, False).tolist() == [True] * 9 + [False] * 3


# ------------------------------------------------------------------ argument checks of the C entry points

P = 0x10000  # a well-aligned address that is never read


def _rope_args(**kw):
    a = dict(n_tokens=8, n_heads=2, n_rot_heads=2, x=P, x_token_stride=128, x_head_stride=64, out=P + (1 << 20),
             out_token_stride=128, out_head_stride=64, x_is_fp32=0, out_is_fp32=0, pos=P, inverse=0)
    a.update(kw)
    return st.saf3r_rope_args(**a)


def _rope_status(cfg=None, **kw):
    cfg = hw.make_rope((32, 32)) if cfg is None else cfg
    a = _rope_args(**kw)
    return hw.lib().saf3r_rope(ctypes.byref(cfg), ctypes.byref(a), None)


@pytest.mark.parametrize("dims,base,pairing", [((0, 8), 100.0, 0), ((12,), 100.0, 0), ((64, 8), 100.0, 0),
                                               ((128,), 100.0, 0), ((32,), 0.5, 0), ((32,), float("nan"), 0),
                                               ((32,), 1e13, 0), ((32,), 100.0, 3), ((-8,), 100.0, 0)])
def test_rope_refuses_bad_configurations(dims, base, pairing):
    assert _rope_status(hw.make_rope(dims, base, pairing)) == hw.ERR_INVALID
    with pytest.raises(ValueError):
        hw.make_rope(())


@pytest.mark.parametrize("kw", [dict(x=None), dict(out=None), dict(pos=None), dict(x=P + 8), dict(out=P + 4), dict(pos=P + 2),
                                dict(n_tokens=-1), dict(n_heads=-1), dict(n_rot_heads=3), dict(n_rot_heads=-1),
                                dict(x_token_stride=124), dict(x_head_stride=-64), dict(out_head_stride=60),
                                dict(out_token_stride=0), dict(out_head_stride=0), dict(out_token_stride=64),
                                dict(n_tokens=1 << 31), dict(x=P, out=P, x_is_fp32=1), dict(x=P, out=P, x_head_stride=1024)])
def test_rope_refuses_bad_arguments(kw):
    assert _rope_status(**kw) == hw.ERR_INVALID


def test_empty_calls_return_before_any_device_work():
    assert _rope_status(n_tokens=0, x=None, out=None, pos=None) == hw.OK
    assert _rope_status(n_heads=0, n_rot_heads=0) == hw.OK
    assert _append_status(n_seqs=0) == hw.OK
    assert _append_status(n_tokens=0, max_new=0) == hw.OK


CACHE = dict(n_pages=4, n_heads=2, page=64, type=1, k=P, v=P, k_scale=P, v_scale=P)
BATCH = dict(n_seqs=1, n_tokens=8, max_new=8, max_pages=2, cu_tokens=P, kv_lens=P, page_table=P)
ROWS = dict(k=P, k_token_stride=128, k_head_stride=64, v=P, v_token_stride=128, v_head_stride=64, pos=P)


def _append_status(rope=None, **kw):
    c, b, r = dict(CACHE), dict(BATCH), dict(ROWS)
    for k, v in kw.items():
        d, k = (c, k[6:]) if k.startswith("cache_") else (b, k) if k in b else (r, k)
        d[k] = v
    c, b, r = st.saf3r_kv_cache(**c), st.saf3r_kv_batch(**b), st.saf3r_kv_rows(**r)
    return hw.lib().saf3r_kv_append(ctypes.byref(c), ctypes.byref(b), None if rope is None else ctypes.byref(rope),
                                    ctypes.byref(r), None)


@pytest.mark.parametrize("kw", [dict(cache_n_pages=0), dict(cache_n_heads=0), dict(cache_n_heads=65), dict(cache_page=48),
                                dict(cache_page=256), dict(cache_type=2), dict(cache_k=None), dict(cache_v=P + 8),
                                dict(cache_k_scale=None), dict(cache_v_scale=P + 4), dict(n_seqs=-1), dict(n_seqs=65536),
                                dict(n_tokens=-1), dict(max_new=9), dict(max_new=-1), dict(max_pages=-1),
                                dict(cu_tokens=None), dict(kv_lens=None), dict(page_table=None), dict(kv_lens=P + 1),
                                dict(k=None), dict(v=None), dict(k=P + 8), dict(k_token_stride=100), dict(v_head_stride=-64)])
def test_append_refuses_bad_arguments(kw):
    assert _append_status(**kw) == hw.ERR_INVALID


def test_append_refuses_a_bad_rope_and_sizes_past_31_bits():
    assert _append_status(hw.make_rope((20,))) == hw.ERR_INVALID
    assert _append_status(hw.make_rope((32,)), pos=None) == hw.ERR_INVALID
    assert _append_status(cache_n_pages=1 << 24) == hw.ERR_UNSUPPORTED
    assert _append_status(max_pages=1 << 26) == hw.ERR_UNSUPPORTED


WINDOW = dict(view_tokens=4, window=2, n_sink=4, causal=1)
QUERIES = dict(n_heads=4, out_is_fp32=0, q=P, q_token_stride=256, q_head_stride=64, out=P + (1 << 20), out_token_stride=256,
               out_head_stride=64)


def _attn_status(workspace=P, **kw):
    c, b, w, r = dict(CACHE), dict(BATCH), dict(WINDOW), dict(QUERIES)
    for k, v in kw.items():
        d, k = (c, k[6:]) if k.startswith("cache_") else (b, k) if k in b else (w, k) if k in w else (r, k)
        d[k] = v
    c, b, w, r = st.saf3r_kv_cache(**c), st.saf3r_kv_batch(**b), st.saf3r_window(**w), st.saf3r_query_rows(**r)
    return hw.lib().saf3r_kv_attn(*(ctypes.byref(x) for x in (c, b, w, r)), workspace, None)


@pytest.mark.parametrize("kw", [dict(workspace=None), dict(workspace=P + 8), dict(view_tokens=0), dict(window=-1), dict(n_sink=-1),
                                dict(n_heads=0), dict(n_heads=3), dict(n_heads=66), dict(q=None), dict(out=None), dict(q=P + 8),
                                dict(out=P + (1 << 20) + 4), dict(out=P), dict(out=P, out_is_fp32=1), dict(q_token_stride=252),
                                dict(q_head_stride=0), dict(out_head_stride=32), dict(out_token_stride=128), dict(max_new=9),
                                dict(cache_page=8), dict(cache_k=None), dict(kv_lens=None)])
def test_attention_refuses_bad_arguments(kw):
    assert _attn_status(**kw) == hw.ERR_INVALID


def test_attention_of_nothing_returns_before_any_device_work():
    assert _attn_status(n_seqs=0) == hw.OK
    assert _attn_status(n_tokens=0, max_new=0, q=None, out=None) == hw.OK


def test_window_attention_refuses_bad_arguments_and_an_output_over_its_inputs():
    lay = hw.make_layout(S=2, grid_h=3, grid_w=3, H=2, n_special=1)
    n = 2 * 2 * 10 * 128  # bytes of a tensor

    def status(q=P, k=P, v=P, out=P + n, fp32=0, ws=P, **kw):
        w = st.saf3r_window(**{**WINDOW, **kw})
        return hw.lib().saf3r_window_attn(ctypes.byref(lay), ctypes.byref(w), q, k, v, out, fp32, ws, None)

    for kw in [dict(q=None), dict(k=P + 8), dict(v=None), dict(out=None), dict(ws=None), dict(ws=P + 4), dict(view_tokens=0),
               dict(window=-1), dict(out=P), dict(out=P + n - 16), dict(out=P - n + 16), dict(out=P - n, fp32=1),
               dict(k=P + n), dict(v=P + n + 16), dict(v=P + n, fp32=1)]:
        assert status(**kw) == hw.ERR_INVALID, kw


# ------------------------------------------------------------------ checks of the bindings

def _cpu_batch(n=1, t=8):
    i = torch.int32
    return hw.KVBatch(torch.zeros(n + 1, dtype=i), torch.zeros(n, dtype=i), torch.zeros((n, 2), dtype=i), t, t)


def test_bindings_refuse_wrong_tensors():
    bf = torch.bfloat16
    x, pos = torch.zeros((8, 2, 64), dtype=bf), torch.zeros((8, 2), dtype=torch.int32)
    r = hw.make_rope((32, 32))
    for bad in [(x[:, :, :32], pos, x), (x, pos.long(), x), (x, pos[:, :1], x), (x, pos[:4], x), (x.half(), pos, x),
                (x, pos, x[:4]), (x.transpose(0, 1), pos, x), (x, pos, x), (x.repeat(1, 1, 2)[..., ::2], pos, x)]:
        with pytest.raises(ValueError):  # the last but one: good shapes, but not on a GPU
            hw.saf3r_rope(r, *bad)
    cache = hw.PagedKV.empty(4, 2, 64, hw.KV_E4M3, device="cpu")
    with pytest.raises(ValueError):
        hw.saf3r_kv_append(cache, _cpu_batch(), x, x)            # no GPU
    with pytest.raises(ValueError):
        hw.saf3r_kv_append(cache, _cpu_batch(), x.float(), x)
    with pytest.raises(ValueError):
        hw.saf3r_kv_append(cache, _cpu_batch(), x[:, :1], x)
    with pytest.raises(ValueError):
        hw.saf3r_kv_append(cache, _cpu_batch(), x, x, r)          # a rope without positions


def test_handles_refuse_wrong_tensors():
    k = torch.zeros((4, 2, 64, 64), dtype=torch.bfloat16)
    f8, s = k.to(torch.float8_e4m3fn), torch.ones((4, 2))
    hw.PagedKV(k, k.clone()), hw.PagedKV(f8, f8.clone(), s, s.clone())
    for bad in [(k, k[:2]), (k, f8), (f8, f8), (f8, f8, s, s[:2]), (f8, f8, s.double(), s), (k.float(), k.float()),
                (k[..., :32], k[..., :32]), (k.transpose(1, 2), k.transpose(1, 2))]:
        with pytest.raises(ValueError):
            hw.PagedKV(*bad)
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    hw.KVBatch(i, i[:2], t, 8, 8)
    for bad in [(i.long(), i[:2], t), (i[:2], i[:2], t), (i, i[:2], t[:1]), (i, i[:2], t.T), (i, i[:2], i)]:
        with pytest.raises(ValueError):
            hw.KVBatch(*bad, 8, 8)
