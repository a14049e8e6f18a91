"""Streaming attention where single keys, values or pages are far from the others.

Tolerances are those of check_rows, written out at the head of test_gpu_streaming_attn.py.
"""
import numpy as np
import pytest

from oracle import streaming as O
from test_gpu_streaming import Paged, _hw, _np
from test_gpu_streaming_attn import check_rows, check_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ALL = (1, 0, 0, False)  # every row sees every key


def _loud_rows(rows, key):
    """Query rows [rows, 1, 64] whose logits at a key of `key` in its first dim (0 at keys without one) go from 60 to 2000."""
    q = torch.zeros((rows, 1, 64), device="cuda")
    q[:, 0, 0] = 8.0 / key * 60.0 * (2000.0 / 60.0) ** (torch.arange(rows, device="cuda") / (rows - 1))
    return q.bfloat16()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("block", [1, 4])
def test_one_key_far_above_the_rest_of_its_row(e4m3, block):
    """Whatever its place among the 16 keys of a group, and however far above the row's first block its logit is."""
    hw = _hw()
    rows, old = 130, 500
    for at in range(16):
        c = Paged(hw, 1, 1, 64, 12, e4m3, seed=3)
        g = torch.Generator(device="cuda").manual_seed(at)
        kv = torch.randn((old + rows, 2, 1, 64), device="cuda", generator=g)
        kv[:, 0] = 0.0
        kv[128 * block + 32 + at, 0, 0, 0] = 16.0
        kv = kv.bfloat16()
        c.step([old], k=kv[:old, 0], v=kv[:old, 1])
        batch = c.step([rows], k=kv[old:, 0], v=kv[old:, 1])
        check_step(c, batch, [rows], 1, ALL, torch.float32, q=_loud_rows(rows, 16.0))


def test_window_attention_with_one_key_far_above_the_rest():
    hw = _hw()
    L = hw.make_layout(4, 10, H=1)
    V, N = 105, 420
    win = hw.make_window(V, 0, 0, False)
    ws = torch.empty(hw.saf3r_window_attn_workspace_bytes(L, win), dtype=torch.uint8, device="cuda")
    q = _loud_rows(N, 16.0).transpose(0, 1).contiguous()
    for at in range(16):
        g = torch.Generator(device="cuda").manual_seed(at)
        v = torch.randn((1, N, 64), device="cuda", generator=g).bfloat16()
        k = torch.zeros_like(v)
        k[0, 272 + at, 0] = 16.0
        out = torch.empty((1, N, 64), device="cuda")
        hw.saf3r_window_attn(L, win, q, k, v, out, ws)
        hw.saf3r_check()
        idx = np.arange(0, N, 3)
        check_rows(_np(out[0])[idx], _np(q[0])[idx], _np(k[0]), _np(v[0]), idx, (V, 0, 0, False), False, False, f"key {at}")


@pytest.mark.parametrize("over", ["bf16 cache", "8-bit cache", "views"])
def test_a_key_in_sight_that_is_not_a_number_is_seen_at_every_place(over):
    """Its values are finite: the rows learn of it by their weights alone."""
    hw = _hw()
    L = hw.make_layout(4, 10, H=1)
    N = 420
    for at in range(16):
        g = torch.Generator(device="cuda").manual_seed(at)
        q, k, v = torch.randn((3, N, 1, 64), device="cuda", generator=g).bfloat16()
        k[272 + at] = float("nan")
        out = torch.zeros((N, 1, 64), device="cuda")
        if over == "views":
            win = hw.make_window(105, 0, 0, False)
            ws = torch.empty(hw.saf3r_window_attn_workspace_bytes(L, win), dtype=torch.uint8, device="cuda")
            hw.saf3r_window_attn(L, win, *(t.transpose(0, 1).contiguous() for t in (q, k, v)), out.view(1, N, 64), ws)
        else:
            c = Paged(hw, 1, 1, 64, 7, over == "8-bit cache", seed=3)
            batch = c.step([N], k=k, v=v)
            win = hw.make_window(*ALL)
            ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, 1), dtype=torch.uint8, device="cuda")
            hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
        hw.saf3r_check()
        assert torch.isnan(out).all(), at


def _check_by_own_keys(c, batch, new, heads, mask, q, rows):
    """Rows `rows` of the step's only sequence, with a tolerance from the keys that count in each: a logit summed in fp32 is off
    by 2^-18 of sum |q_d k_d| / 8 (d) and moves weights and sum by 2d, whatever other keys hold; weights in fp16, their
    exponentials and sums 2^-11 + 2^-12, and n 2^-24 of the largest value in sight."""
    hw = _hw()
    out = torch.empty(q.shape, device="cuda")
    win = hw.make_window(*mask)
    ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, heads), dtype=torch.uint8, device="cuda")
    hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
    hw.saf3r_check()
    end = int(c.lens[0])
    k, v = (O.cached_rows(x, s, c.table[0], end, c.page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
    for h in range(heads):
        for r in rows:
            p, k1, v1, q1 = end - new + r, k[:, h // (heads // c.heads)], v[:, h // (heads // c.heads)], _np(q[r, h])
            j = O.seen(p, end, *mask)
            s = k1[j] @ q1 / 8
            w = np.exp(s - s.max())
            w /= w.sum()
            far = w > 1e-30
            d = 2.0 ** -18 * (np.abs(k1[j][far]) @ np.abs(q1)).max() / 8
            tol = (w @ np.abs(v1[j])) * (2.0 ** -11 + 2.0 ** -12 + 2 * d) + j.sum() * 2.0 ** -24 * np.abs(v1[j]).max()
            err = np.abs(_np(out[r, h]) - w @ v1[j])
            assert (err <= tol).all(), (h, r, err.max(), (err / tol).max())


@pytest.mark.parametrize("new", [9, 150])
@pytest.mark.parametrize("spread", [30, 45, 80])
@pytest.mark.parametrize("negative", [False, True])
def test_8bit_keys_of_far_apart_scales(new, spread, negative):
    """A page of huge keys out of a row's window, or one whose logits are far below the others, leaves the other keys' bits alone."""
    hw = _hw()
    c = Paged(hw, 1, 2, 16, 44, True, seed=3)
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(i)
        kv = torch.randn(((500, new)[i], 2, 2, 64), device="cuda", generator=g)
        if i == 0:
            kv[464:480, 0] = (-kv[464:480, 0].abs() if negative else kv[464:480, 0]) * 2.0 ** spread
            kv[448:464, 0] = 0.0  # a page of zeros beside it
        kv = kv.bfloat16()
        batch = c.step([len(kv)], k=kv[:, 0], v=kv[:, 1])
    q = torch.randn((new, 4, 64), device="cuda", generator=g)
    q = (q.abs() if negative else q).bfloat16()
    if negative:
        _check_by_own_keys(c, batch, new, 4, (1, 0, 0, True), q, range(0, new, max(1, new // 9)))
    # of 150 rows with a window of 50 those from 29 on no longer see the page, of 9 with a window of 12 none does
    window = 50 if new > 29 else 12
    _check_by_own_keys(c, batch, new, 4, (1, window, 0, True), q, range(29 if new > 29 else 0, new, max(1, new // 9)))


def _with_zero_pages(hw, where, magnitude, keys=1024, page=16, heads=2):
    """An 8-bit cache of one sequence whose value pages `where` are zero, the others of `magnitude`."""
    c = Paged(hw, 1, heads, page, keys // page + 2, True, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn((keys, 2, heads, 64), device="cuda", generator=g)
    kv[:, 1] *= magnitude
    for i in where:
        kv[i * page:(i + 1) * page, 1] = 0.0
    kv = kv.bfloat16()
    c.step([keys], k=kv[:, 0], v=kv[:, 1])
    return c


@pytest.mark.parametrize("where", [[0], [0, 1, 2, 3, 4], [1], [2, 17, 30], [63], list(range(64)), list(range(1, 64)), list(range(63))])
@pytest.mark.parametrize("magnitude", [2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 110])
@pytest.mark.parametrize("new", [1, 5])
def test_8bit_pages_of_zero_values(where, magnitude, new):
    """Their keys count in the sum of the weights, wherever the pages lie; rows that see only them are zero."""
    hw = _hw()
    c = _with_zero_pages(hw, where, magnitude)
    k, v = torch.randn((2, new, 2, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).bfloat16()
    batch = c.step([new], k=k, v=(v.float() * magnitude).bfloat16())
    for mask in [(1, 0, 0, True), (1, 60, 20, True)]:
        check_step(c, batch, [new], 4, mask, torch.float32)
        check_step(c, batch, [new], 4, mask, torch.float32, q=torch.zeros((new, 4, 64), device="cuda").bfloat16())


def test_a_value_that_is_not_a_number_on_a_page_of_zeros():
    hw = _hw()
    for first in (0, 9):
        c = _with_zero_pages(hw, [first], 1.0)
        c.kv.v[c.table[0, first], :, 3, 5] = torch.full((2,), float("nan"), device="cuda").to(torch.float8_e4m3fn)
        c.v[c.table[0, first], :, 3, 5] = np.nan
        batch = c.step([1], seed=4)
        q, out = check_step(c, batch, [1], 4, (1, 0, 0, True), torch.float32)
        assert torch.isnan(out[..., 5]).all() and torch.isfinite(out[..., 6:]).all()


def test_a_page_of_zero_values_costs_no_more_than_another():
    """Rows next to it went key by key, 400 times as long; 3 times leaves room for a busy machine."""
    hw = _hw()
    times = []
    for where in ([], [0], [500]):
        c = _with_zero_pages(hw, where, 1.0, keys=16384)
        batch = c.step([1], seed=4)
        q = torch.randn((1, 4, 64), device="cuda").bfloat16()
        out, win = torch.empty_like(q), hw.make_window()
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, 4), dtype=torch.uint8, device="cuda")
        best = float("inf")
        for _ in range(10):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        hw.saf3r_check()
        times.append(best)
    print("us with no page of zeros, the first, one in the middle:", times)
    assert max(times) < 3 * times[0], times


def test_rows_that_go_key_by_key_end_before_others_give_up_waiting():
    """Ten sequences of 4,200 keys whose value scales are too far apart for the products, 64 heads of 70 rows each: a warp's 32
    rows of an item take less than a wait budget of 25 ms (60 ms at 0.46 us a key), and are right."""
    hw = _hw()
    seqs, heads, page, end, new = 10, 64, 64, 4200, 70
    per = -(-end // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = hw.PagedKV.empty(seqs * per, heads, page, hw.KV_E4M3)
    for t in (kv.k, kv.v):
        t.copy_(torch.randn(t.shape, device="cuda", generator=g).to(t.dtype))
    kv.k_scale.fill_(1.0)
    kv.v_scale.fill_(1.0)
    kv.v_scale[3::per] = 2.0 ** 30
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = hw.KVBatch(torch.arange(seqs + 1, **i32) * new, torch.full((seqs,), end, **i32),
                       torch.arange(seqs * per, **i32).view(seqs, per), seqs * new, new)
    q = torch.randn((seqs * new, heads, 64), device="cuda", generator=g).bfloat16()
    out, win = torch.empty(q.shape, device="cuda"), hw.make_window()
    ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(kv, batch, win, heads), dtype=torch.uint8, device="cuda")
    hw.saf3r_set_wait_budget(50_000_000)
    try:
        hw.saf3r_kv_attn(kv, batch, win, q, out, ws)
        hw.saf3r_check()
    finally:
        hw.saf3r_set_wait_budget(0)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    hw.saf3r_kv_attn(kv, batch, win, q, out, ws)
    b.record()
    b.synchronize()
    hw.saf3r_check()
    print("us with all rows key by key:", a.elapsed_time(b) * 1000)
    for s, r, h in [(0, 0, 0), (3, 69, 5), (9, 33, 63), (5, 64, 31), (7, 12, 12)]:
        pages, n = slice(s * per, (s + 1) * per), end - new + r + 1
        k = kv.k[pages, h].reshape(-1, 64)[:n].double()
        v = (kv.v[pages, h].double() * kv.v_scale[pages, h].double()[:, None, None]).reshape(-1, 64)[:n]
        w = torch.softmax(k @ q[s * new + r, h].double() / 8, 0)
        # fp32 logits (2^-18 of sum |q k| / 8, twice: weights and sum), exponentials and sums
        tol = (w @ v.abs()) * (2.0 ** -17 * (k.abs() @ q[s * new + r, h].double().abs()).max() / 8 + 2.0 ** -18)
        assert ((out[s * new + r, h].double() - w @ v).abs() <= tol).all(), (s, r, h)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,old,new", [(2, 4000, 1), (2, 4000, 9), (2, 300, 80), (1, 9000, 80), (32, 700, 70)])
def test_values_next_to_the_largest_number(e4m3, heads, old, new):
    """Means of values near the end of the range, of one sign and of both, though their sums leave it."""
    c = Paged(_hw(), 1, heads, 64, 160, e4m3, seed=3)
    batch = None
    for i, n in enumerate((old, new)):
        g = torch.Generator(device="cuda").manual_seed(i)
        kv = torch.randn((n, 2, heads, 64), device="cuda", generator=g)
        kv[:, 1, :, :32] = 2.9e38 * (0.5 + 0.5 * torch.rand((n, heads, 32), device="cuda", generator=g))
        kv[:, 1, :, 32:] = 2.9e38 * torch.sign(kv[:, 1, :, 32:])
        kv[:, 1, :, 60:] = 1.0
        kv = kv.bfloat16()
        batch = c.step([n], k=kv[:, 0], v=kv[:, 1])
    for mask in [(1, 0, 0, True), (1, 250, 3, True)]:
        check_step(c, batch, [new], heads, mask, torch.float32, rows=12)


def test_window_attention_over_values_next_to_the_largest_number():
    hw = _hw()
    L = hw.make_layout(4, 10, H=2)
    N = 420
    q, k = torch.randn((2, 2, N, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    v = (3e38 * torch.sign(torch.randn((2, N, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)))).bfloat16()
    v[..., :32] = v[..., :32].abs()
    out = torch.empty((2, N, 64), device="cuda")
    for mask in [(105, 0, 0, False), (105, 2, 0, True)]:
        win = hw.make_window(*mask)
        hw.saf3r_window_attn(L, win, q, k, v, out, torch.empty(hw.saf3r_window_attn_workspace_bytes(L, win), dtype=torch.uint8, device="cuda"))
        hw.saf3r_check()
        idx = np.arange(0, N, 7)
        for h in range(2):
            check_rows(_np(out[h])[idx], _np(q[h])[idx], _np(k[h]), _np(v[h]), idx, mask, False, False, f"head {h}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,old,new", [(2, 4000, 1), (2, 40, 1), (2, 4000, 9), (2, 300, 80), (1, 9000, 80), (32, 200, 70)])
def test_rows_of_infinite_logits(e4m3, heads, old, new):
    """Minus infinity at every key (as at any with plus infinity) is not a number; the rows beside such a one are as always."""
    hw = _hw()
    c = Paged(hw, 1, heads, 64, 160, e4m3, seed=3)
    for i, n in enumerate((old, new)):
        kv = torch.randn((n, 2, heads, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        kv[:, 0, :, 0] = 0.5 + kv[:, 0, :, 0].abs()
        kv = kv.bfloat16()
        batch = c.step([n], k=kv[:, 0], v=kv[:, 1])
    for value in (-float("inf"), float("inf")):
        q = torch.randn((new, heads, 64), device="cuda").bfloat16()
        q[new // 2:, :, 0] = value
        for mask in [(1, 0, 0, True), (1, 250, 3, True)]:
            out = torch.zeros(q.shape, device="cuda")
            win = hw.make_window(*mask)
            ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, heads), dtype=torch.uint8, device="cuda")
            hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
            hw.saf3r_check()
            assert torch.isfinite(out[:new // 2]).all() and torch.isnan(out[new // 2:]).all(), (value, mask)


@pytest.mark.parametrize("new", [1, 9, 80])
def test_a_key_of_minus_infinity_takes_no_part(new):
    hw = _hw()
    c = Paged(hw, 1, 2, 64, 12, False, seed=3)
    batch = None
    for i, n in enumerate((500, new)):
        kv = torch.randn((n, 2, 2, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        if i == 0:
            kv[:16, 0, :, 0] = -float("inf")  # at every place of a group, and first in a row's first block
            kv[296:300, 0, :, 0] = -float("inf")
        kv = kv.bfloat16()
        batch = c.step([n], k=kv[:, 0], v=kv[:, 1])
    q = torch.randn((new, 4, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    q[..., 0] = q[..., 0].abs() + 0.1
    q = q.bfloat16()
    out = torch.empty(q.shape, device="cuda")
    for mask in [(1, 0, 0, True), (1, 1000, 0, False), (1, 250, 8, True)]:
        win = hw.make_window(*mask)
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, 4), dtype=torch.uint8, device="cuda")
        hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
        hw.saf3r_check()
        k, v = (O.cached_rows(x, None, c.table[0], 500 + new, 64) for x in (c.k, c.v))
        far = np.where(np.isinf(k), 0.0, k)  # for the tolerance
        for h in range(4):
            for r in range(0, new, 7):
                j = O.seen(500 + r, 500 + new, *mask)
                s = k[j, h // 2] @ _np(q[r, h]) / 8
                w = np.exp(s - s.max())
                w /= w.sum()
                tol = (w @ np.abs(v[j, h // 2])) * (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -17 * (np.abs(far[j, h // 2]) @ np.abs(_np(q[r, h]))).max() / 8)
                assert (np.abs(_np(out[r, h]) - w @ v[j, h // 2]) <= tol).all(), (mask, h, r)


def _random_rows(rng, tokens, heads, size, written):
    """Strides (elements) of rows of 64 in one of the orders; rows that are only read may be repeated."""
    unit = 16 // size
    if rng.integers(2):
        hs = 64 + unit * int(rng.integers(0, 9))
        ts = (heads - 1) * hs + 64 + unit * int(rng.integers(0, 40))
    else:
        ts = 64 + unit * int(rng.integers(0, 9))
        hs = (tokens - 1) * ts + 64 + unit * int(rng.integers(0, 40))
    if not written and rng.integers(4) == 0:
        ts, hs = (0, hs) if rng.integers(2) else (ts, 0)
    return ts, hs


def _units(at, ts, hs, tokens, heads, size):
    """The 16-byte units of every row."""
    i = at + (np.arange(tokens)[:, None] * ts + np.arange(heads) * hs) * size // 16
    return (i[..., None] + np.arange(4 * size)).ravel()


def test_rows_of_one_buffer_interleave_or_are_refused():
    """Rotation between two sets of rows of one buffer, against a count of the bytes that they share."""
    hw = _hw()
    rng = np.random.default_rng(1)
    cfg = hw.make_rope((32, 32))
    ran = refused = careful = 0
    for _ in range(1500):
        T, H = int(rng.integers(1, 6)), int(rng.integers(1, 5))
        sx, so = (int(rng.choice([2, 4])) for _ in range(2))
        xt, xh = _random_rows(rng, T, H, sx, False)
        ot, oh = _random_rows(rng, T, H, so, True)
        if rng.integers(2):  # one packed buffer: the same steps
            so, (xt, xh) = sx, _random_rows(rng, T, H, sx, True)
            gap = 64 * int(rng.integers(1, 4))
            xt, xh = (xt + gap, xh) if xt > xh else (xt, xh + gap)
            ot, oh = xt, xh
        a, b = (int(n) for n in rng.integers(0, 200, 2))
        ux, uo = _units(a, xt, xh, T, H, sx), _units(b, ot, oh, T, H, so)
        if sx == so and a == b and (xt if T > 1 else 0, xh if H > 1 else 0) == (ot if T > 1 else 0, oh if H > 1 else 0):
            continue  # in place
        buf = torch.randn(int(max(ux.max(), uo.max()) + 8) * 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
        view = lambda n, s, ts, hs: buf.view(torch.float32 if s == 4 else torch.bfloat16).as_strided((T, H, 64), (ts, hs, 1), n * 16 // s)  # noqa: E731
        if sx == 2 or so == 2:
            buf = torch.randn(2 * buf.numel(), device="cuda").bfloat16().view(torch.float32)
        x, out = view(a, sx, xt, xh), view(b, so, ot, oh)
        pos = torch.randint(0, 40, (T, 2), device="cuda").int()
        shared = bool(np.intersect1d(ux, uo).size)
        same_steps = xt * sx == ot * so or T == 1 or xt == 0
        apart = ux.max() < uo.min() or uo.max() < ux.min()
        if shared or not (same_steps or apart):
            with pytest.raises(hw.Saf3rError) as e:
                hw.saf3r_rope(cfg, x, pos, out)
            assert e.value.status == hw.ERR_INVALID
            refused += shared
            careful += not shared
            continue
        ran += not apart
        want, before = torch.empty((T, H, 64), device="cuda", dtype=out.dtype), buf.clone()
        hw.saf3r_rope(cfg, x.clone(), pos, want)
        hw.saf3r_rope(cfg, x, pos, out)
        assert torch.equal(out.nan_to_num(1e9), want.nan_to_num(1e9))
        out.zero_()
        buf2, buf = buf, before
        view(b, so, ot, oh).zero_()
        assert torch.equal(buf2.view(torch.int32), buf.view(torch.int32))
    hw.saf3r_check()
    assert min(ran, refused) > 50 and careful > 0, (ran, refused, careful)


@pytest.mark.parametrize("new", [3, 90])
def test_queries_and_output_of_one_packed_buffer(new):
    hw = _hw()
    c = Paged(hw, 1, 2, 64, 12, False, seed=3)
    c.step([300], 1.0, seed=1)
    batch = c.step([new], seed=2)
    win = hw.make_window(1, 100, 3)
    ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, 4), dtype=torch.uint8, device="cuda")
    packed = torch.randn((new, 3, 4, 64), device="cuda").bfloat16()
    keep, want = packed.clone(), torch.empty((new, 4, 64), device="cuda", dtype=torch.bfloat16)
    hw.saf3r_kv_attn(c.kv, batch, win, keep[:, 1], want, ws)
    hw.saf3r_kv_attn(c.kv, batch, win, packed[:, 1], packed[:, 2], ws)
    keep[:, 2] = want
    assert torch.equal(packed, keep)
    rows = packed.view(new, 12, 64)
    for q, out in [(rows[:, :4], rows[:, 3:7]), (rows[:, 4:8], rows[:, 1:5]), (rows[:-1, :4], rows[1:, 2:6])]:
        b = batch if len(q) == new else hw.KVBatch(batch.cu_tokens, batch.kv_lens, batch.page_table, new - 1, new - 1)
        with pytest.raises(hw.Saf3rError) as e:
            hw.saf3r_kv_attn(c.kv, b, win, q, out, ws)
        assert e.value.status == hw.ERR_INVALID
    hw.saf3r_check()


@pytest.mark.parametrize("heads,kv_heads,page,new", [(2, 2, 64, [65]), (6, 2, 32, [33, 257, 0, 5]), (5, 1, 128, [100, 0, 7, 52])])
def test_many_rows_over_8bit_keep_11_bits_of_a_weight(heads, kv_heads, page, new):
    """fp16 weights: 2^-11 of each, and of n keys at most n 2^-24 of the largest value in all (check_rows' fp16 tolerance)."""
    hw = _hw()
    c = Paged(hw, len(new), kv_heads, page, -(-2200 // page), True, seed=page)
    c.step([700, 31, 0, 450][:len(new)], 1.0, seed=1)
    for i, mask in enumerate([(1, 0, 0, True), (1, 130, 4, True), (37, 3, 37, True), (37, 2, 300, False), (1, 1, 0, True)]):
        batch = c.step(new, 0.5 + i % 3, seed=i + 2)
        g = torch.Generator(device="cuda").manual_seed(i)
        q = (2 * torch.randn((batch.n_tokens, heads, 64), device="cuda", generator=g)).bfloat16()
        out, win = torch.empty(q.shape, device="cuda"), hw.make_window(*mask)
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, heads), dtype=torch.uint8, device="cuda")
        hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)
        hw.saf3r_check()
        t = 0
        for b, n in enumerate(new):
            end, idx = int(c.lens[b]), np.arange(0, n, 5)
            k, v = (O.cached_rows(x, s, c.table[b], end, page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
            for h in range(heads if n else 0):
                check_rows(_np(out[t:t + n, h])[idx], _np(q[t:t + n, h])[idx], k[:, h // (heads // kv_heads)],
                           v[:, h // (heads // kv_heads)], end - n + idx, mask, True, False, f"mask {mask}, sequence {b}, head {h}")
            t += n


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_rows_report_numbers_that_do_not_fit(e4m3):
    hw = _hw()
    new = 100
    c = Paged(hw, 1, 2, 16, 20, e4m3, seed=1)
    good = c.step([new], seed=1)
    check_step(c, good, [new], 2, (1, 0, 0, True), rows=8)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros((new, 2, 64), device="cuda").bfloat16()
    win = hw.make_window()
    for cu, n, m in [([0, new + 1], new + 1, new), ([-1, new], new + 1, new), ([new, 0], new, new), ([0, new], 321, new),
                     ([0, new], new - 1, new), ([0, new], new, new - 1), ([0, new], -5, new)]:
        bad = hw.KVBatch(torch.tensor(cu, **i32), torch.tensor([n], **i32), good.page_table, new, m)
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, bad, win, 2), dtype=torch.uint8, device="cuda")
        hw.saf3r_kv_attn(c.kv, bad, win, q, torch.empty_like(q), ws)
        with pytest.raises(hw.Saf3rError) as e:
            hw.saf3r_check()
        assert e.value.status == hw.ERR_INDEX
        hw.saf3r_check()
    check_step(c, good, [new], 2, (1, 0, 0, True), rows=8)


def test_an_expired_wait_over_an_8bit_cache_is_reported_and_the_next_call_is_clean():
    """One softmax warp withholds one arrival: the product warp's wait runs out, nothing hangs."""
    hw = _hw()
    c = Paged(hw, 1, 1, 64, 40, True, seed=3)
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


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("new", [1, 90])
def test_pages_behind_the_first_four_gigabytes(e4m3, new):
    """The same step over a small cache and over one whose pages in use lie at the far end of pools of 5 GB: the same bits."""
    hw = _hw()
    heads, page, per, seqs = 8, 64, 8, 2
    n_big = 5 * 2 ** 30 // (heads * page * 64 * (1 if e4m3 else 2))
    g = torch.Generator(device="cuda").manual_seed(new)
    i32 = dict(dtype=torch.int32, device="cuda")
    cfg, win = hw.make_rope((32, 32)), hw.make_window(1, 200, 5)
    steps = []
    for n in (300, new):
        k, v = torch.randn((2, seqs * n, heads, 64), device="cuda", generator=g).bfloat16()
        steps.append((n, k, v, torch.randint(0, 99, (seqs * n, 2), device="cuda", generator=g).int()))
    q = torch.randn((seqs * new, 2 * heads, 64), device="cuda", generator=g).bfloat16()
    outs = []
    for n_pages in (seqs * per, n_big):
        kv = hw.PagedKV.empty(n_pages, heads, page, hw.KV_E4M3 if e4m3 else hw.KV_BF16)
        table = (n_pages - 1 - torch.arange(seqs * per, **i32)).view(seqs, per)
        done = 0
        for n, k, v, pos in steps:
            done += n
            batch = hw.KVBatch(torch.arange(seqs + 1, **i32) * n, torch.full((seqs,), done, **i32), table, seqs * n, n)
            hw.saf3r_kv_append(kv, batch, k, v, cfg, pos)
        out = torch.empty(q.shape, device="cuda")
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(kv, batch, win, 2 * heads), dtype=torch.uint8, device="cuda")
        hw.saf3r_kv_attn(kv, batch, win, q, out, ws)
        hw.saf3r_check()
        rows = table.long().flatten()
        outs.append((out, kv.k[rows][:, :, :50].view(torch.uint8).clone(), kv.v[rows][:, :, :50].view(torch.uint8).clone()))
        del kv
    assert torch.equal(outs[0][0], outs[1][0]) and torch.isfinite(outs[0][0]).all()
    used = [i for i in range(seqs * per) if i % per < (300 + new) // page]
    for a, b in zip(outs[0][1:], outs[1][1:]):
        assert torch.equal(a[used], b[used])
