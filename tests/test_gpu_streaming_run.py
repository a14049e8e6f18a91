"""The streaming operators together, as a model that takes its views one after another uses them, and the calls that are easy
to get wrong: captured and replayed steps, streams, many sequences, padded rows, far-apart scales and logits.

Tolerances are those of the attention tests (check_rows); where a step's queries are rotated first, the oracle takes the
rotated bf16 queries that the step itself used, so that no tolerance has to cover two roundings at once.
"""
import numpy as np
import pytest

from oracle import streaming as O
from test_gpu_streaming import Paged, _hw, _np
from test_gpu_streaming_attn import check_rows, check_step, few_rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _attn(hw, c, batch, win, q, out=None, stream=None, ws=None):
    out = torch.empty_like(q) if out is None else out
    if ws is None:
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, q.shape[1]), dtype=torch.uint8, device="cuda")
    hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws, stream=stream)
    return out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (8, 2)])
def test_views_one_after_another(e4m3, heads, kv_heads):
    """Packed projections rotated, appended and attended view by view, then token by token."""
    hw = _hw()
    V, n_views = 41, 4
    dims = (32, 32)
    rope = (hw.make_rope(dims, 100.0, hw.ROPE_HALF), dims, 100.0, O.HALF)
    c = Paged(hw, 2, kv_heads, 16, 20, e4m3, seed=1)
    win = hw.make_window(V, 2, V)
    g = torch.Generator(device="cuda").manual_seed(9)
    for step in range(n_views + 3):
        new = [V, V] if step < n_views else [1, 1]
        batch = c.step(new, 1.0, rope=rope, seed=step + 20)
        T = batch.n_tokens
        packed = torch.randn((T, heads, 64), device="cuda", generator=g).bfloat16()
        pos = torch.randint(0, 40, (T, 2), device="cuda", generator=g).int()
        q = torch.empty((heads, T, 64), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
        hw.saf3r_rope(rope[0], packed, pos, q)
        check_step(c, batch, new, heads, (V, 2, V, True), q=q, rows=12)
    hw.saf3r_check()


def test_stepwise_and_offline_attention_agree():
    """The same mask over a cache, view by view, and over all views at once: the same bf16 products."""
    hw = _hw()
    S, grid, H = 5, 8, 3
    V = grid * grid + 5
    N = S * V
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((H, N, 64), device="cuda", generator=g).bfloat16() for _ in range(3))
    L = hw.make_layout(S, grid, H=H)
    win = hw.make_window(V, 2, V)
    whole = torch.empty((H, N, 64), device="cuda")
    hw.saf3r_window_attn(L, win, q, k, v, whole, torch.empty(hw.saf3r_window_attn_workspace_bytes(L, win), dtype=torch.uint8, device="cuda"))
    c = Paged(hw, 1, H, 32, -(-N // 32), False, seed=2)
    parts = torch.empty((N, H, 64), device="cuda")
    for s in range(S):
        rows = slice(s * V, (s + 1) * V)
        batch = c.step([V], k=k[:, rows].transpose(0, 1), v=v[:, rows].transpose(0, 1))
        _attn(hw, c, batch, win, q[:, rows].transpose(0, 1), parts[rows])
    hw.saf3r_check()
    # the weights' bf16 rounding (2^-8 of sum p |v| <= max |v|) and the sums', on both sides
    assert (whole.transpose(0, 1) - parts).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -12) * v.float().abs().max()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 90])
def test_a_captured_step_follows_its_arrays(e4m3, n):
    """Append and attention in one graph; lengths, table and rows change between replays."""
    hw = _hw()
    heads = 2
    c = Paged(hw, 2, heads, 16, 30, e4m3, seed=5)
    c.step([50, 37], 1.0, seed=1)
    start = c.lens.copy()
    T = 2 * n
    kv = torch.zeros((T, 2, heads, 64), device="cuda", dtype=torch.bfloat16)
    k, v = kv[:, 0], kv[:, 1]
    q = torch.zeros((T, heads, 64), device="cuda", dtype=torch.bfloat16)
    out = torch.zeros((T, heads, 64), device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, lens = torch.tensor([0, n, 2 * n], **i32), torch.tensor(start + n, **i32)
    batch = hw.KVBatch(cu, lens, torch.from_numpy(c.table).cuda(), T, n)
    win = hw.make_window(1, 60, 4)
    ws = torch.full((hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, heads),), 0xAB, dtype=torch.uint8, device="cuda")

    def step():
        hw.saf3r_kv_append(c.kv, batch, k, v)
        hw.saf3r_kv_attn(c.kv, batch, win, q, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [t.clone() for t in (c.kv.k.view(torch.uint8), c.kv.v.view(torch.uint8))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()  # once before the capture
    torch.cuda.current_stream().wait_stream(side)
    for t, old in zip((c.kv.k, c.kv.v), keep):
        t.view(torch.uint8).copy_(old)
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(4)
    for i, new in enumerate([[n, n], [n, max(n - 3, 0)], [0, n]]):
        c.lens += np.asarray(new)
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32))
        lens.copy_(torch.tensor(c.lens, **i32))
        kv.copy_(torch.randn(kv.shape, device="cuda", generator=g))
        q.copy_(2 * torch.randn(q.shape, device="cuda", generator=g))
        out.fill_(7.5)
        if e4m3 and i == 0:  # the scales that the twin has are those before the first, uncaptured step
            for name, twin in (("k_scale", c.ks), ("v_scale", c.vs)):
                getattr(c.kv, name).copy_(torch.from_numpy(twin))
        graph.replay()
        torch.cuda.synchronize()
        O.append(c.k, c.ks, _np(k), cu.cpu().numpy(), c.lens, c.table, 16)
        O.append(c.v, c.vs, _np(v), cu.cpu().numpy(), c.lens, c.table, 16)
        t = 0
        for b, m in enumerate(new):
            end = int(c.lens[b])
            kk, vv = O.cached_rows(c.k, c.ks, c.table[b], end, 16), O.cached_rows(c.v, c.vs, c.table[b], end, 16)
            for h in range(heads):
                check_rows(_np(out)[t:t + m, h], _np(q)[t:t + m, h], kk[:, h], vv[:, h], end - m + np.arange(m), (1, 60, 4, True),
                           e4m3 and n == 1, False, f"replay {i}, sequence {b}, head {h}")
            t += m
        assert (out[t:] == 7.5).all()
    hw.saf3r_check()


def test_two_streams_at_once():
    """Each with a workspace of its own, one step of few rows and one of many on either."""
    hw = _hw()
    steps = []
    for i in range(4):
        c = Paged(hw, 1, 2, 64, 40, i % 2 == 1, seed=i)
        c.step([1500], 1.0, seed=i)
        batch = c.step([1 if i < 2 else 200], 1.0, seed=i + 9)
        q = torch.randn((batch.n_tokens, 4, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)).bfloat16()
        win = hw.make_window(1, 700, 3)
        ws = torch.empty(hw.saf3r_kv_attn_workspace_bytes(c.kv, batch, win, 4), dtype=torch.uint8, device="cuda")
        steps.append((c, batch, win, q, ws, _attn(hw, c, batch, win, q, ws=ws).clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(s[3]) for s in steps]
    for _ in range(20):
        for i in (0, 2, 1, 3):
            c, batch, win, q, ws, _ = steps[i]
            _attn(hw, c, batch, win, q, outs[i], stream=streams[i % 2], ws=ws)
    torch.cuda.synchronize()
    hw.saf3r_check()
    for s, o in zip(steps, outs):
        assert torch.equal(s[5], o)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("seqs,heads,new", [(300, 4, 1), (1100, 64, 2)])
def test_many_sequences(e4m3, seqs, heads, new):
    """More sequences than a block has threads (few rows), and than the plan has entries (many rows)."""
    hw = _hw()
    c = Paged(hw, seqs, 1, 16, 6, e4m3, seed=2)
    rng = np.random.default_rng(seqs)
    c.step(list(rng.integers(0, 70, seqs)), 1.0, seed=1)
    counts = rng.integers(0, new + 1, seqs)
    batch = c.step(list(counts), 1.0, seed=2)
    if batch.max_new < new:
        pytest.skip("no sequence got the most")
    assert few_rows(batch, heads, 1) == (heads == 4)
    q = torch.randn((batch.n_tokens, heads, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    win = hw.make_window(1, 40, 2)
    out = _attn(hw, c, batch, win, q, torch.empty(q.shape, device="cuda"))
    hw.saf3r_check()
    cu = np.concatenate([[0], np.cumsum(counts)])
    for b in list(range(6)) + list(rng.integers(0, seqs, 20)) + [seqs - 1]:
        n, end = int(counts[b]), int(c.lens[b])
        if n == 0:
            continue
        kk, vv = O.cached_rows(c.k, c.ks, c.table[b], end, 16), O.cached_rows(c.v, c.vs, c.table[b], end, 16)
        for h in (0, heads - 1):
            rows = slice(int(cu[b]), int(cu[b]) + n)
            check_rows(_np(out)[rows, h], _np(q)[rows, h], kk[:, 0], vv[:, 0], end - n + np.arange(n), (1, 40, 2, True),
                       e4m3 and heads == 4, False, f"sequence {b}, head {h}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [[2], [130]])
def test_strided_rows_and_nothing_beside_them(e4m3, new):
    hw = _hw()
    c = Paged(hw, 1, 2, 32, 20, e4m3, seed=3)
    c.step([300], 1.0, seed=1)
    batch = c.step(new, seed=2)
    T = batch.n_tokens
    g = torch.Generator(device="cuda").manual_seed(5)
    qw = torch.randn((T, 3, 4, 72), device="cuda", generator=g).bfloat16()
    q = qw[:, 1, :, :64]
    win = hw.make_window(1, 100, 8)
    plain = _attn(hw, c, batch, win, q.contiguous(), torch.empty((T, 4, 64), device="cuda"))
    wide = torch.full((T, 5, 96), 3.25, device="cuda")
    _attn(hw, c, batch, win, q, wide[:, :4, 16:80])
    hw.saf3r_check()
    assert torch.equal(wide[:, :4, 16:80], plain)
    wide[:, :4, 16:80] = 3.25
    assert (wide == 3.25).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [[1], [9], [140]])
@pytest.mark.parametrize("grow", [4.0, 40.0, 400.0])
def test_logits_that_keep_growing(e4m3, new, grow):
    """Each page's keys are larger than the last one's: references far below later logits."""
    hw = _hw()
    c = Paged(hw, 1, 2, 16, 40, e4m3, seed=3)
    for i in range(20):
        g = torch.Generator(device="cuda").manual_seed(i)
        kv = torch.randn((16, 2, 2, 64), device="cuda", generator=g)
        kv[:, 0] *= grow ** (i / 20)
        kv = kv.bfloat16()
        c.step([16], k=kv[:, 0], v=kv[:, 1])
    batch = c.step(new, 1.0, seed=40)
    for mask in [(1, 0, 0, True), (1, 90, 3, True)]:
        check_step(c, batch, new, 4, mask, torch.float32, rows=16)
    hw.saf3r_check()


@pytest.mark.parametrize("new", [[1], [9], [140]])
def test_pages_of_far_apart_scales(new):
    """8-bit pages whose value scales are 2^30 to 2^90 apart; rows that see only small ones keep their bits."""
    hw = _hw()
    for spread in (20, 45, 90):
        c = Paged(hw, 1, 2, 16, 40, True, seed=3)
        for i in range(22):
            g = torch.Generator(device="cuda").manual_seed(i)
            kv = torch.randn((16, 2, 2, 64), device="cuda", generator=g)
            kv[:, 1] *= 2.0 ** (spread if i % 5 == 1 else 0)
            if i == 3:
                kv[:] = 0.0  # a page of zeros
            kv = kv.bfloat16()
            c.step([16], k=kv[:, 0], v=kv[:, 1])
        batch = c.step(new, 1.0, seed=40)
        for mask in [(1, 0, 0, True), (1, 30, 0, True)]:
            check_step(c, batch, new, 4, mask, torch.float32, rows=16)
    hw.saf3r_check()


def test_masks_of_the_largest_numbers():
    hw = _hw()
    top = 2 ** 31 - 1
    for new in ([3, 1], [100, 40]):
        c = Paged(hw, 2, 1, 16, 40, False, seed=3)
        c.step([200, 0], 1.0, seed=1)
        batch = c.step(new, seed=2)
        for mask in [(top, top, top, False), (1, top, 0, False), (top, 0, 0, True), (1, 1, top, True)]:
            check_step(c, batch, new, 2, mask, rows=12)
    hw.saf3r_check()


def test_a_step_without_new_tokens():
    hw = _hw()
    c = Paged(hw, 2, 1, 16, 4, True, seed=3)
    c.step([20, 3], 1.0, seed=1)
    for new_rows in (1, 100):
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = hw.KVBatch(torch.zeros(3, **i32), torch.tensor(c.lens, **i32), torch.from_numpy(c.table).cuda(), new_rows, new_rows)
        q = torch.zeros((new_rows, 2, 64), device="cuda").bfloat16()
        before = c.kv.k.view(torch.uint8).clone()
        hw.saf3r_kv_append(c.kv, batch, q[:, :1], q[:, :1])
        out = _attn(hw, c, batch, hw.make_window(), q, torch.full(q.shape, 7.5, device="cuda"))
        hw.saf3r_check()
        assert (out == 7.5).all() and torch.equal(c.kv.k.view(torch.uint8), before)
