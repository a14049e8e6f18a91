"""Streaming operators on the GPU against the fp64 oracle: rotary positions and the paged append.

Tolerances.  Rotation in fp32: the angle is exact to 2^-33 turns and its conversion to fp32 rounds half turns by
2^-24 of a value of at most 1, so the sine and cosine are off by at most pi * 2^-24 + 2^-23 < 4.4e-7 (two
half-unit errors of sincospif within 2 ulp); a cos x - b sin x then by at most (|a| + |b|) * (4.4e-7 + 2 * 2^-24)
< 6e-7 (|a| + |b|).  A bf16 output adds half a unit, 2^-8 of the value; an e4m3 code half a step: 2^-4 of the value,
or 2^-10 of the scale below 2^-6 of it.
"""
import numpy as np
import pytest

from oracle import streaming as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32 = 6e-7  # of |a| + |b|


def _hw():
    import head_wise_dynamic_b200 as hw
    return hw


def _np(t):
    return t.detach().double().cpu().numpy()


def _pair_sum(x, dims, pairing, n_rot):
    """|a| + |b| of the pair that each value belongs to (0 where nothing turns)."""
    m = np.zeros_like(x)
    for a, b, _, _ in O.rope_pairs(dims, 10.0, pairing):
        m[:, :n_rot, a] = m[:, :n_rot, b] = np.abs(x[:, :n_rot, a]) + np.abs(x[:, :n_rot, b])
    return m


@pytest.mark.parametrize("pairing", [0, 1, 2])
@pytest.mark.parametrize("dims,base", [((32, 32), 100.0), ((16, 24, 24), 10000.0), ((64,), 10000.0), ((8, 16), 1.0),
                                       ((8, 8, 8, 8), 100.0), ((40,), 1e12)])
@pytest.mark.parametrize("tokens,heads,n_rot", [(1, 1, 1), (33, 5, 3), (261, 12, 12)])
def test_rope_matches_the_oracle(pairing, dims, base, tokens, heads, n_rot):
    hw = _hw()
    g = torch.Generator(device="cuda").manual_seed(tokens * 7 + len(dims))
    pos = torch.randint(-5, 2 ** 31 - 1 if tokens == 33 else 40, (tokens, len(dims)), device="cuda", generator=g).int()
    cfg = hw.make_rope(dims, base, pairing)
    for din, dout in [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                      (torch.float32, torch.bfloat16)]:
        x = torch.randn((tokens, heads, 64), device="cuda", generator=g).to(din)
        for inverse in (False, True):
            out = torch.full((heads, tokens, 64), float("nan"), device="cuda", dtype=dout).transpose(0, 1)
            hw.saf3r_rope(cfg, x, pos, out, n_rot_heads=n_rot, inverse=inverse)
            assert hw.saf3r_last_launch_count() == 1
            want = O.rope(_np(x), pos.cpu().numpy(), dims, base, pairing, n_rot, inverse)
            tol = F32 * _pair_sum(_np(x), dims, pairing, n_rot) + (np.abs(want) * 2.0 ** -8 if dout == torch.bfloat16 else 0)
            assert (np.abs(_np(out) - want) <= tol * 1.001).all()
    hw.saf3r_check()


def test_rope_strides_in_place_and_broadcast():
    hw = _hw()
    g = torch.Generator(device="cuda").manual_seed(3)
    cfg, T = hw.make_rope((32, 32)), 70
    pos = torch.randint(0, 40, (T, 2), device="cuda", generator=g).int()
    packed = torch.randn((T, 3, 4, 80), device="cuda", generator=g).bfloat16()  # rows 80 apart
    q = packed[:, 1, :, 8:72]
    want = O.rope(_np(q), pos.cpu().numpy(), (32, 32), 100.0, 0)
    keep = packed.clone()
    out = torch.empty((T, 4, 64), device="cuda", dtype=torch.bfloat16)
    hw.saf3r_rope(cfg, q, pos, out)
    assert torch.equal(packed, keep)
    hw.saf3r_rope(cfg, q, pos, q)  # in place
    assert torch.equal(q, out)
    keep[:, 1, :, 8:72] = out
    assert torch.equal(packed, keep)  # nothing else was written
    assert (np.abs(_np(out) - want) <= (np.abs(want) * 2.0 ** -8 + F32 * _pair_sum(_np(keep[:, 1, :, 8:72]), (32, 32), 0, 4) * 4)).all()
    one = torch.randn((T, 1, 64), device="cuda", generator=g)  # one head for all
    wide = torch.empty((T, 5, 64), device="cuda")
    hw.saf3r_rope(cfg, one.expand(T, 5, 64), pos, wide)
    alone = torch.empty((T, 1, 64), device="cuda")
    hw.saf3r_rope(cfg, one, pos, alone)
    assert torch.equal(wide, alone.expand(T, 5, 64))


def test_rope_on_another_stream_and_in_a_graph():
    hw = _hw()
    g = torch.Generator(device="cuda").manual_seed(4)
    cfg = hw.make_rope((32, 32))
    x = torch.randn((50, 6, 64), device="cuda", generator=g)
    pos = torch.randint(0, 40, (50, 2), device="cuda", generator=g).int()
    ref, out = torch.empty_like(x), torch.zeros_like(x)
    hw.saf3r_rope(cfg, x, pos, ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hw.saf3r_rope(cfg, x, pos, out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hw.saf3r_rope(cfg, x, pos, out)
    x.copy_(torch.randn((50, 6, 64), device="cuda", generator=g))
    hw.saf3r_rope(cfg, x, pos, ref)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


# ------------------------------------------------------------------ append

class Paged:
    """A cache on the GPU beside its fp64 twin: same page table, same codes at the start."""

    def __init__(self, hw, seqs, heads, page, max_pages, e4m3, seed, spare=3):
        self.hw, self.page, self.e4m3, self.heads = hw, page, e4m3, heads
        rng = np.random.default_rng(seed)
        self.n_pages = seqs * max_pages + spare
        self.table = rng.permutation(self.n_pages)[:seqs * max_pages].reshape(seqs, max_pages).astype(np.int32)
        self.kv = hw.PagedKV.empty(self.n_pages, heads, page, hw.KV_E4M3 if e4m3 else hw.KV_BF16)
        self.kv.k.view(torch.uint8).fill_(0x7f)  # NaN everywhere: only written rows may count
        self.kv.v.view(torch.uint8).fill_(0x7f)
        shape = (self.n_pages, heads, page, 64)
        self.k, self.v = np.full(shape, np.nan), np.full(shape, np.nan)
        self.ks = self.vs = None
        if e4m3:
            self.kv.k_scale.fill_(float("nan"))
            self.kv.v_scale.fill_(float("nan"))
            self.ks, self.vs = np.full(shape[:2], np.nan), np.full(shape[:2], np.nan)
        self.lens = np.zeros(seqs, dtype=np.int64)

    def step(self, new, scale_of_rows=1.0, rope=None, seed=0, extra=0, k=None, v=None, pad_rows=0):
        """Append new[b] rows to every sequence; `extra` rows lie behind the last sequence."""
        hw = self.hw
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1]) + extra
        g = torch.Generator(device="cuda").manual_seed(seed)
        if k is None:
            kv = (torch.randn((max(T, 1), 2, self.heads, 64), device="cuda", generator=g) * scale_of_rows).bfloat16()[:T]
            k, v = kv[:, 0], kv[:, 1]
        self.lens += np.asarray(new)
        batch = hw.KVBatch(torch.from_numpy(cu).cuda(), torch.from_numpy(self.lens.astype(np.int32)).cuda(),
                           torch.from_numpy(self.table).cuda(), T, max(list(new) + [0]))
        pos = None
        kk = _np(k)
        if rope is not None:
            cfg, dims, base, pairing = rope
            pos = torch.randint(0, 100000, (T, len(dims)), device="cuda", generator=g).int()
            kk = O.rope(kk, pos.cpu().numpy(), dims, base, pairing)
        hw.saf3r_kv_append(self.kv, batch, k, v, None if rope is None else rope[0], pos)
        O.append(self.k, self.ks, kk, cu, self.lens, self.table, self.page)
        O.append(self.v, self.vs, _np(v), cu, self.lens, self.table, self.page)
        return batch

    def compare(self, exact, slack=0.0):
        """Every written row against the twin; rows that nothing was written to hold what they held."""
        for name, want, ws in (("k", self.k, self.ks), ("v", self.v, self.vs)):
            t = getattr(self.kv, name)
            got = _np(t.float())
            if self.e4m3:
                gs = _np(getattr(self.kv, name + "_scale"))
                assert np.array_equal(np.isnan(gs), np.isnan(ws))
                assert np.array_equal(np.nan_to_num(gs), np.nan_to_num(ws))
            written = np.zeros(want.shape[:3], dtype=bool)
            for b, n in enumerate(self.lens):
                for i in range(int(n)):
                    written[self.table[b, i // self.page], :, i % self.page] = True
            raw = t.view(torch.uint8).cpu().numpy().reshape(*want.shape[:3], -1)
            assert (raw[~written] == 0x7f).all()
            a, b = got[written], want[written]
            assert np.array_equal(np.isnan(a), np.isnan(b))
            if exact or name == "v":
                assert np.array_equal(np.nan_to_num(a), np.nan_to_num(b))
            else:  # a value next to a rounding border may fall to its other side: one step, on few
                step = np.maximum(np.abs(b) * 2.0 ** -3, 2.0 ** -9) if self.e4m3 else np.abs(b) * 2.0 ** -7 + 1e-30
                d = np.abs(a - b)
                assert (d <= step * 1.001).all()
                assert (d > 0).mean() < 1e-3  # borders are 2^-18 wide at most beside steps of 2^-8 and more


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [1, 5, 16])
def test_append_ragged_steps(e4m3, page, heads):
    """Steps of none, one and many tokens over page borders, rows behind the last sequence, growing scales."""
    hw = _hw()
    c = Paged(hw, 4, heads, page, -(-400 // page), e4m3, seed=page + heads)
    for i, (new, mag) in enumerate([([1, 0, 3, 17], 0.1), ([1, 1, 1, 1], 1.0), ([0, page, 5, 130], 8.0), ([1, 0, 0, 1], 0.01),
                                    ([200, 1, page - 1, 2], 50.0)]):
        c.step(new, mag, seed=i, extra=i % 3)
        c.compare(exact=True)
    hw.saf3r_check()


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("dims,pairing", [((32, 32), 0), ((16, 24, 24), 1), ((16, 24, 24), 2), ((40,), 0)])
def test_append_rotates_the_keys(e4m3, dims, pairing):
    hw = _hw()
    c = Paged(hw, 3, 6, 64, 5, e4m3, seed=1)
    rope = (hw.make_rope(dims, 100.0, pairing), dims, 100.0, pairing)
    for i, new in enumerate([[70, 1, 0], [1, 1, 1], [100, 200, 3]]):
        c.step(new, 2.0 ** i, rope, seed=i)
    c.compare(exact=False)
    hw.saf3r_check()


def test_append_special_values():
    """Zeros, infinities, NaN, the largest and smallest magnitudes; a page of zeros that grows; subnormal codes."""
    hw = _hw()
    big = 3.3895313892515355e38
    rows = [0.0, 1.0, float("inf"), -float("inf"), float("nan"), big, -big, 1e-38, 1e-45, 448.0, 449.0, 1e-3]
    for e4m3 in (True, False):
        c = Paged(hw, 1, 2, 16, 4, e4m3, seed=0)
        for i, r in enumerate(rows):
            x = torch.zeros((1, 2, 64), device="cuda")
            x[..., :8] = r
            x[:, 1, 8:16] = 2.0 ** -12
            x = x.bfloat16()
            c.step([1], k=x, v=-x)
            c.compare(exact=True)
    hw.saf3r_check()


def test_append_reports_numbers_that_do_not_fit():
    """Bad page ids, lengths and row ranges: SAF3R_ERR_INDEX, nothing written outside the rows that fit."""
    hw = _hw()
    x = torch.ones((8, 2, 64), device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")

    def call(cu, lens, table, max_new=8):
        kv = hw.PagedKV.empty(4, 2, 16, hw.KV_BF16)
        kv.k.zero_(), kv.v.zero_()
        hw.saf3r_kv_append(kv, hw.KVBatch(torch.tensor(cu, **i32), torch.tensor(lens, **i32), torch.tensor(table, **i32),
                                          8, max_new), x, x)
        return kv

    good = call([0, 8], [20], [[1, 3]])
    hw.saf3r_check()
    assert int(good.k.abs().sum()) == 8 * 2 * 64
    for bad in [([0, 8], [20], [[1, 4]]), ([0, 8], [20], [[1, -1]]), ([0, 8], [33], [[1, 3]]), ([0, 8], [7], [[1, 3]]),
                ([0, 9], [20], [[1, 3]]), ([-1, 7], [20], [[1, 3]]), ([4, 0], [20], [[1, 3]]), ([0, 8], [20], [[1, 3]], 7)]:
        kv = call(*bad)
        with pytest.raises(hw.Saf3rError) as e:
            hw.saf3r_check()
        assert e.value.status == hw.ERR_INDEX
        assert int(kv.k.abs().sum()) <= 4 * 2 * 64  # rows 12..15 of page 1 fit in the first two
        hw.saf3r_check()


def test_append_in_a_graph_follows_the_device_lengths():
    hw = _hw()
    c, d = (Paged(hw, 2, 4, 64, 4, True, seed=5) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = torch.randn((2, 2, 4, 64), device="cuda", generator=g).bfloat16()
    cu, lens = torch.tensor([0, 1, 2]).int().cuda(), torch.tensor([63, 10]).int().cuda()
    batch = hw.KVBatch(cu, lens, torch.from_numpy(c.table).cuda(), 2, 1)
    c.step([62, 9], seed=1), d.step([62, 9], seed=1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hw.saf3r_kv_append(c.kv, batch, k, v)
        lens.add_(1)
    for _ in range(4):
        d.step([1, 1], k=k, v=v)
        graph.replay()
    torch.cuda.synchronize()
    for a, b in ((c.kv.k, d.kv.k), (c.kv.v, d.kv.v), (c.kv.k_scale, d.kv.k_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    hw.saf3r_check()
