"""Attention over the paged cache and over views held at once, on the GPU against the fp64 oracle.

Tolerance, of an output o = sum p_j v_j with A = sum p_j |v_j|: the weights are rounded once to the type of the
product (bf16: half a unit is 2^-8; fp16 for few rows over 8-bit caches: 2^-11, and 2^-25 of the largest below its normal
range, over n keys at most n 2^-24 max |v|); a logit summed in fp32 is off by at most d = 2^-18 of
sum |q_d k_d| / 8, which moves weights and sum by 2d; exponentials and sums add less than 2^-12 (the tensor-core
kernel's polynomial exponential: 8.6e-5).  A bf16 output adds 2^-8 |o|.
"""
import numpy as np
import pytest

from oracle import streaming as O
from test_gpu_streaming import Paged, _hw, _np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def check_rows(got, q, k, v, pos, mask, fp16, bf16_out, what):
    """got [t, 64] against the oracle over k, v [n, 64]."""
    want = O.attend(q, k, v, pos, *mask)
    fin = np.isfinite(v)
    vv = np.where(fin, v, 0.0)
    a = O.attend(q, k, np.abs(vv), pos, *mask)
    d = 2.0 ** -18 * (np.abs(q) @ np.nan_to_num(np.abs(k), posinf=0.0).max(0) / 8)[:, None]
    tol = a * ((2.0 ** -11 if fp16 else 2.0 ** -8) + 2 * d + 2.0 ** -12)
    if fp16:
        tol = tol + len(k) * 2.0 ** -24 * np.abs(vv).max()
    if bf16_out:
        tol = tol + np.abs(want) * 2.0 ** -8
    ok = np.isfinite(want)
    assert np.array_equal(ok, np.isfinite(got)), what
    assert np.array_equal(np.isnan(want), np.isnan(got)), what
    assert np.array_equal(want[~ok & ~np.isnan(want)], got[~ok & ~np.isnan(want)]), what
    err = np.abs(np.where(ok, got, 0) - np.where(ok, want, 0))
    assert (err <= np.where(ok, tol, 0) * 1.001 + 1e-30).all(), f"{what}: {err.max():.3e}, {(err / (tol + 1e-30)).max():.2f} of the tolerance"


def few_rows(batch, heads, kv_heads):
    """Whether a step takes the kernel for few rows (whose 8-bit products are fp16 ones)."""
    return batch.max_new * (heads // kv_heads) <= 64


def check_step(c, batch, new, heads, mask, out_dtype=torch.bfloat16, seed=0, token_major=False, q=None, kv=None, rows=None):
    """Attention of a step's tokens over the cache c; returns (q, out).  `rows`: how many tokens of a sequence are checked."""
    hw = _hw()
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    T = batch.n_tokens
    if q is None:
        q = (2 * torch.randn((T, heads, 64) if token_major else (heads, T, 64), device="cuda", generator=g)).bfloat16()
        q = q if token_major else q.transpose(0, 1)
    out = torch.full((T, heads, 64) if token_major else (heads, T, 64), 7.5, device="cuda", dtype=out_dtype)
    out = out if token_major else out.transpose(0, 1)
    win = hw.make_window(*mask)
    ws = torch.full((hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, heads),), 0xAB, dtype=torch.uint8, device="cuda")
    hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
    hw.saf3r_check()
    Q, got, t, gr = _np(q), _np(out), 0, heads // c.heads
    for b, n in enumerate(new):
        n = int(n)
        end = int(c.lens[b])
        k = O.cached_rows(c.k, c.ks, c.table[b], end, c.page)
        v = O.cached_rows(c.v, c.vs, c.table[b], end, c.page)
        idx = np.arange(n) if rows is None or n <= rows else np.unique(
            np.concatenate([np.arange(3), np.random.default_rng(seed).integers(0, n, rows - 6), np.arange(n - 3, n)]))
        for h in range(heads):
            if n:
                check_rows(got[t + idx, h], Q[t + idx, h], k[:, h // gr], v[:, h // gr], end - n + idx, mask,
                           c.e4m3 and few_rows(batch, heads, c.heads),
                           out_dtype == torch.bfloat16, f"sequence {b}, head {h}")
        t += n
    assert (got[t:] == 7.5).all()  # rows behind the last sequence
    return q, out


MASKS = [(1, 0, 0, True), (1, 33, 4, True), (1, 5, 0, True), (7, 3, 7, True), (7, 0, 0, False), (7, 2, 40, False), (50, 1, 1, True),
         (1, 0, 0, False), (1, 1, 0, True)]


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 2), (5, 1), (16, 1)])
def test_single_tokens_match_the_oracle(e4m3, page, heads, kv_heads):
    hw = _hw()
    c = Paged(hw, 5, kv_heads, page, -(-700 // page), e4m3, seed=page)
    c.step([1, 600, 63, 130, 0], 1.0, seed=1)
    for i, mask in enumerate(MASKS):
        new = [1, 1, 1, 1, i % 2]
        batch = c.step(new, 1.0 + i % 3, seed=i + 2, extra=i % 2)
        check_step(c, batch, new, heads, mask, torch.bfloat16 if i % 2 else torch.float32, seed=i, token_major=bool(i % 3))


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("heads,kv_heads,new", [(4, 4, [17, 0, 1, 64]), (8, 2, [16, 3, 0, 5]), (6, 2, [1, 2, 7, 21])])
def test_short_chunks_match_the_oracle(e4m3, heads, kv_heads, new):
    hw = _hw()
    c = Paged(hw, 4, kv_heads, 32, 24, e4m3, seed=3)
    c.step([0, 500, 31, 1], 1.0, seed=1)
    for i, mask in enumerate(MASKS):
        batch = c.step(new, 0.5 + i % 3, seed=i + 2)
        check_step(c, batch, new, heads, mask, seed=i, token_major=bool(i % 2))
        if c.lens.max() + 64 > 24 * 32:
            break


def _spoil(c, b, j, what, value):
    """Writes `value` over the key or value row of token j of sequence b, in the cache and its twin."""
    pg, r = int(c.table[b, j // c.page]), j % c.page
    t = getattr(c.kv, what)
    if c.e4m3:
        t[pg, :, r] = torch.full((c.heads, 64), float("nan") if not np.isfinite(value) else value, device="cuda").to(t.dtype)
        value = np.nan if not np.isfinite(value) else value
    else:
        t[pg, :, r] = value
    getattr(c, what)[pg, :, r] = value


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("new", [[1], [9]])
def test_masked_rows_may_hold_anything(e4m3, new):
    """Not-a-number and infinite keys and values outside a row's window; the rows that see them get them."""
    hw = _hw()
    c = Paged(hw, 1, 2, 64, 10, e4m3, seed=3)
    c.step([500], 1.0, seed=1)
    batch = c.step(new, seed=2)
    for j in (10, 100, 447, 450, 453):   # a window of 50: the query at 500 sees 451.., the one at 504 no longer 453
        _spoil(c, 0, j, "v", np.nan)
    for j in (20, 440):
        _spoil(c, 0, j, "k", np.nan)
        _spoil(c, 0, j, "v", -np.inf)
    q, out = check_step(c, batch, new, 4, (1, 50, 4, True), torch.float32)
    assert torch.isnan(out[0]).any() and (new == [1] or torch.isfinite(out[8]).all())
    _spoil(c, 0, 453, "v", 1.0)
    q, out = check_step(c, batch, new, 4, (1, 50, 4, True), torch.float32)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("heads,new", [(2, [1, 1]), (4, [9, 3]), (8, [16, 16])])
def test_few_rows_over_bf16_keep_16_bits_of_a_weight(heads, new):
    """Weights in two bf16 terms are off by 2^-8 of 2^-8, so nearly all that is left of an fp32 output's error is
    the logits' (2d) and the exponentials' (2^-22 each, as the sum's), in rows of a few weights as in rows of many."""
    hw = _hw()
    c = Paged(hw, 2, 2, 64, 16, False, seed=5)
    c.step([900, 3], 1.0, seed=1)
    for i, scale in enumerate((0.25, 2.0)):
        batch = c.step(new, 1.0, seed=i + 2)
        T = batch.n_tokens
        q = (scale * torch.randn((T, heads, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(i))).bfloat16()
        out = torch.empty((T, heads, 64), device="cuda")
        win = hw.make_window()
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, heads), dtype=torch.uint8, device="cuda")
        hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
        hw.saf3r_check()
        Q, got, t = _np(q), _np(out), 0
        for b, n in enumerate(new):
            end, at = int(c.lens[b]), np.arange(n)
            k, v = (O.cached_rows(x, s, c.table[b], end, c.page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
            for h in range(heads):
                k1, v1, q1, pos = k[:, h // (heads // 2)], v[:, h // (heads // 2)], Q[t + at, h], end - n + at
                want, a = (O.attend(q1, k1, x, pos, 1, 0, 0, True) for x in (v1, np.abs(v1)))
                d = 2.0 ** -18 * (np.abs(q1) @ np.abs(k1).max(0) / 8)[:, None]
                assert (np.abs(got[t + at, h] - want) <= a * (2.0 ** -16 + 2 * d + 2.0 ** -18)).all(), (scale, b, h)
            t += n


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("new", [[1], [5], [90]])
def test_values_in_every_rows_sight_may_be_infinite(e4m3, new):
    hw = _hw()
    c = Paged(hw, 1, 2, 64, 10, e4m3, seed=3)
    c.step([400], 1.0, seed=1)
    batch = c.step(new, seed=2)
    _spoil(c, 0, 30, "v", np.inf)  # 8-bit values hold no infinity: not a number
    q, out = check_step(c, batch, new, 4, (1000, 0, 0, False), torch.float32, q=torch.zeros((4, batch.n_tokens, 64), device="cuda",
                                                                                          dtype=torch.bfloat16).transpose(0, 1))
    assert (torch.isnan(out) if e4m3 else out == np.inf).all()


def test_pages_out_of_sight_are_not_read():
    """Their table entries may be anything; a page in sight that is not there is reported."""
    hw = _hw()
    for new in ([1, 1], [9, 2]):
        c = Paged(hw, 2, 2, 16, 40, True, seed=3)
        c.step([300, 200], 1.0, seed=1)
        batch = c.step(new, seed=2)
        mask = (1, 70, 5, True)
        for b in range(2):
            first = int(c.lens[b]) - new[b] - 69
            for j in range(1, first // 16):
                c.table[b, j] = [-1, 2 ** 31 - 1, c.n_pages][j % 3]
            c.table[b, -(-int(c.lens[b]) // 16):] = -5
        batch.page_table.copy_(torch.from_numpy(c.table))
        check_step(c, batch, new, 4, mask)
        batch.page_table[1, int(c.lens[1] - 1) // 16 - 1] = c.n_pages
        with pytest.raises(hw.Saf3rError) as e:
            check_step(c, batch, [0, 0], 4, mask)
        assert e.value.status == hw.ERR_INDEX
        hw.saf3r_check()


def test_attention_reports_numbers_that_do_not_fit():
    hw = _hw()
    for new in (1,):
        c = Paged(hw, 1, 2, 16, 20, False, seed=1)
        good = c.step([new], seed=1)
        check_step(c, good, [new], 2, (1, 0, 0, True), rows=8)
        i32 = dict(dtype=torch.int32, device="cuda")
        for cu, n, m in [([0, new + 1], new + 1, new), ([-1, new], new + 1, new), ([new, 0], new, new), ([0, new], 321, new),
                         ([0, new], new - 1, new)]:
            bad = hw.KVBatch(torch.tensor(cu, **i32), torch.tensor([n], **i32), good.page_table, new, m)
            q = torch.zeros((new, 2, 64), device="cuda").bfloat16()
            win = hw.make_window()
            ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, bad, win, 2), dtype=torch.uint8, device="cuda")
            hw.saf3r_kv_attn(c.kv, bad, win, q, torch.empty_like(q), ws)
            with pytest.raises(hw.Saf3rError) as e:
                hw.saf3r_check()
            assert e.value.status == hw.ERR_INDEX
            hw.saf3r_check()


LONG = [(1, 0, 0, True), (1, 130, 4, True), (1, 70, 200, True), (37, 3, 37, True), (37, 0, 0, False), (37, 2, 300, False),
        (400, 1, 1, True), (1, 1, 0, True), (1, 0, 0, False)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,kv_heads,page,new", [(2, 2, 64, [65]), (1, 1, 16, [300, 1, 0, 129]), (6, 2, 32, [33, 257, 0, 5]),
                                                     (5, 1, 128, [100, 0, 7, 52])])
def test_many_rows_match_the_oracle(e4m3, heads, kv_heads, page, new):
    """The tensor-core kernel: one tile and two, several items, items cut by shares' borders, empty sequences."""
    hw = _hw()
    n = len(new)
    c = Paged(hw, n, kv_heads, page, -(-4200 // page), e4m3, seed=page)
    c.step([700, 31, 0, 450][:n], 1.0, seed=1)
    for i, mask in enumerate(LONG):
        batch = c.step(new, 0.5 + i % 3, seed=i + 2, extra=i % 2)
        assert not few_rows(batch, heads, kv_heads)
        check_step(c, batch, new, heads, mask, torch.bfloat16 if i % 2 else torch.float32, seed=i, token_major=bool(i % 3), rows=24)
        hw.saf3r_check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_long_item_is_shared_by_many_blocks(e4m3):
    hw = _hw()
    c = Paged(hw, 1, 1, 64, 400, e4m3, seed=3)
    c.step([20000], 1.0, seed=1)
    for i, (new, mask) in enumerate([([70], (1, 0, 0, True)), ([200], (50, 0, 0, False)), ([256], (1, 15000, 100, True)), ([257], (1, 0, 0, True))]):
        batch = c.step(new, 1.0, seed=i + 2)
        check_step(c, batch, new, 1, mask, seed=i, rows=12)


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_rows_masked_rows_may_hold_anything(e4m3):
    hw = _hw()
    c = Paged(hw, 1, 2, 64, 20, e4m3, seed=3)
    c.step([500], 1.0, seed=1)
    new = [150]
    batch = c.step(new, seed=2)
    for j in (10, 100, 447, 450, 460, 530):   # a window of 50: the query at 509 is the last to see 460
        _spoil(c, 0, j, "v", np.nan)
    for j in (20, 440):
        _spoil(c, 0, j, "k", np.nan)
        _spoil(c, 0, j, "v", -np.inf)
    q, out = check_step(c, batch, new, 4, (1, 50, 4, True), torch.float32)
    assert torch.isnan(out[9]).all() and torch.isfinite(out[10:30]).all() and torch.isnan(out[79]).all()
    assert torch.isfinite(out[80:]).all()


def test_many_rows_pages_out_of_sight_are_not_read():
    hw = _hw()
    new = [90, 70]
    c = Paged(hw, 2, 2, 16, 40, True, seed=3)
    c.step([300, 200], 1.0, seed=1)
    batch = c.step(new, seed=2)
    mask = (1, 70, 5, True)
    for b in range(2):
        first = int(c.lens[b]) - new[b] - 69
        for j in range(1, first // 16):
            c.table[b, j] = [-1, 2 ** 31 - 1, c.n_pages][j % 3]
        c.table[b, -(-int(c.lens[b]) // 16):] = -5
    batch.page_table.copy_(torch.from_numpy(c.table))
    check_step(c, batch, new, 4, mask, rows=12)
    batch.page_table[1, int(c.lens[1] - 1) // 16 - 1] = c.n_pages
    with pytest.raises(hw.Saf3rError) as e:
        check_step(c, batch, [0, 0], 4, mask)
    assert e.value.status == hw.ERR_INDEX
    hw.saf3r_check()


@pytest.mark.parametrize("S,grid,H", [(1, 1, 1), (3, 5, 2), (4, 9, 3), (5, 12, 1)])
def test_window_attention_matches_the_oracle(S, grid, H):
    hw = _hw()
    L = hw.make_layout(S, grid, H=H)
    V = grid * grid + 5
    N = S * V
    g = torch.Generator(device="cuda").manual_seed(S)
    q, k, v = (torch.randn((H, N, 64), device="cuda", generator=g).bfloat16() for _ in range(3))
    idx = np.unique(np.random.default_rng(S).integers(0, N, 40))
    for i, mask in enumerate([(V, 0, 0, False), (V, 1, 0, False), (V, 2, V, True), (V, 1, 5, False), (1, 70, 3, True), (7, 0, 0, True)]):
        fp32 = i % 2 == 0
        out = torch.full((H, N, 64), 7.5, device="cuda", dtype=torch.float32 if fp32 else torch.bfloat16)
        win = hw.make_window(*mask)
        ws = torch.full((hw.saf3r_window_attn_workspace_bytes(L, win),), 0xAB, dtype=torch.uint8, device="cuda")
        hw.saf3r_window_attn(L, win, q, k, v, out, ws)
        hw.saf3r_check()
        for h in range(H):
            check_rows(_np(out[h])[idx], _np(q[h])[idx], _np(k[h]), _np(v[h]), idx, mask, False, not fp32, f"mask {mask}, head {h}")


def test_window_attention_over_everything_is_dense_attention():
    """Both kernels of the framework on the same call."""
    hw = _hw()
    L = hw.make_layout(4, 16, H=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((4, 4 * 261, 64), device="cuda", generator=g).bfloat16() for _ in range(3))
    a, b = (torch.empty((4, 4 * 261, 64), device="cuda") for _ in range(2))
    win = hw.make_window(261, 0, 0, False)
    hw.saf3r_window_attn(L, win, q, k, v, a, torch.empty(hw.saf3r_window_attn_workspace_bytes(L, win), dtype=torch.uint8, device="cuda"))
    hw.saf3r_dense_attn(L, q, k, v, b, torch.empty(hw.saf3r_workspace_bytes(L, None, hw.OP_DENSE), dtype=torch.uint8, device="cuda"))
    hw.saf3r_check()
    # two roundings of the weights to bf16, and the sums' error, of sum p |v| <= max |v|
    assert (a - b).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -12) * v.float().abs().max()
    assert (a - b).norm() <= 2.0 ** -8 * b.norm()


def test_an_expired_wait_is_reported_and_the_next_call_is_clean():
    """One softmax warp withholds one arrival: the product warp's wait runs out, nothing hangs."""
    hw = _hw()
    c = Paged(hw, 1, 1, 64, 40, False, seed=3)
    batch = c.step([700], 1.0, seed=1)
    hw.saf3r_set_wait_budget(20_000_000)
    try:
        hw.saf3r_test_withhold_arrive()
        q = torch.zeros((700, 1, 64), device="cuda").bfloat16()
        win = hw.make_window()
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, 1), dtype=torch.uint8, device="cuda")
        hw.saf3r_kv_attn(c.kv, batch, win, q, torch.empty_like(q), ws)
        with pytest.raises(hw.Saf3rError) as e:
            hw.saf3r_check()
        assert e.value.status == hw.ERR_TIMEOUT
        hw.saf3r_check()
        check_step(c, batch, [700], 1, (1, 0, 0, True), rows=12)
    finally:
        hw.saf3r_set_wait_budget(0)
