"""8-bit pages whose largest rotated key lies next to a border between two scales: the scale is that of the exact rotation."""
import numpy as np
import pytest

from oracle import streaming as O
from test_gpu_streaming import _hw, _np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _crossing(a, b, freq, border):
    """The first position at which a cos x - b sin x is no longer above the border (x = position * freq, small)."""
    lo, hi = 0, int(min(2 ** 31 - 1, 1.0 / freq))
    f = lambda p: a * np.cos(p * freq) - b * np.sin(p * freq)  # noqa: E731
    assert f(lo) > border > f(hi)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if f(mid) > border else (lo, mid)
    return hi


@pytest.mark.parametrize("dims,pairing", [((64,), 0), ((64,), 1), ((64,), 2), ((40,), 0), ((24, 24), 1)])
@pytest.mark.parametrize("many", [False, True])
def test_scales_next_to_a_border(dims, pairing, many):
    """Positions around the one where the largest value crosses 448 * 2^n, 2^-26 of it apart: less than fp32 tells, and hundreds
    of times the angle's error (2^-34 turns)."""
    hw = _hw()
    base, page = 1e12, 16
    rows = []  # (pair's dims, a, b, positions)
    for first, second, axis, freq in O.rope_pairs(dims, base, pairing):
        if not 2e-11 < freq < 1e-9:
            continue
        for n in (-6, 0, 9):
            for a in (450.0, 456.0):
                p = _crossing(a, 256.0, freq, 448.0)
                off = max(1, int(448 * 2.0 ** -26 / (256.0 * freq)))
                for d in (-off, off):
                    rows.append((first, second, axis, a * 2.0 ** n, 256.0 * 2.0 ** n, p + d))
    assert len(rows) >= 24
    T, H = len(rows), 2
    per = 3 if many else 1  # new tokens of a sequence: the others are small
    k = torch.zeros((T * per, H, 64))
    pos = torch.zeros((T * per, len(dims)), dtype=torch.int32)
    for i, (first, second, axis, a, b, p) in enumerate(rows):
        k[per * i + per // 2, :, first] = a
        k[per * i + per // 2, :, second] = b
        k[per * i + per // 2, 1] *= -1.0
        pos[per * i + per // 2, axis] = p
    k = k.bfloat16()
    want = O.rope(_np(k), pos.numpy(), dims, base, pairing)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = hw.PagedKV.empty(T, H, page)
    batch = hw.KVBatch(torch.arange(T + 1, **i32) * per, torch.full((T,), per, **i32), torch.arange(T, **i32).view(T, 1), T * per, per)
    kd = k.cuda()
    hw.saf3r_kv_append(cache, batch, kd, torch.zeros_like(kd), hw.make_rope(dims, base, pairing), pos.cuda())
    hw.saf3r_check()
    scale, codes = _np(cache.k_scale), _np(cache.k.float())
    for i in range(T):
        for h in range(H):
            x = want[per * i:per * (i + 1), h]
            s = O.scale_of(np.abs(x).max())
            assert scale[i, h] == s, (rows[i], h, scale[i, h], s)
            assert np.array_equal(codes[i, h, :per], O.round_e4m3(x / s))


@pytest.mark.parametrize("pairing", [0, 1, 2])
@pytest.mark.parametrize("many", [False, True])
def test_codes_next_to_a_tie(pairing, many):
    """Values 2^-27 from the middle between two codes on either side: fp32 would put them on it."""
    hw = _hw()
    base, page, dims = 1e12, 16, (40,)
    rows = []
    for first, second, axis, freq in O.rope_pairs(dims, base, pairing):
        if not 2e-11 < freq < 1e-9:
            continue
        for a, middle in ((58.25, 58.0), (62.25, 62.0), (54.25, 54.0), (50.25, 50.0)):
            p = _crossing(a, 32.0, freq, middle)
            off = max(1, int(middle * 2.0 ** -27 / (32.0 * freq)))
            rows += [(first, second, a, p + d) for d in (-off, off)]
    T, H = len(rows), 2
    assert T >= 8
    per = 3 if many else 1
    k = torch.zeros((T * per, H, 64))
    pos = torch.zeros((T * per, 1), dtype=torch.int32)
    for i, (first, second, a, p) in enumerate(rows):
        at = per * i + per // 2
        k[at, :, first], k[at, :, second], k[at, :, 63] = a, 32.0, 448.0  # dims from 40 on are not rotated: the scale is 1
        k[at, 1] *= -1.0
        pos[at, 0] = p
    k = k.bfloat16()
    want = O.round_e4m3(O.rope(_np(k), pos.numpy(), dims, base, pairing))
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = hw.PagedKV.empty(T, H, page)
    batch = hw.KVBatch(torch.arange(T + 1, **i32) * per, torch.full((T,), per, **i32), torch.arange(T, **i32).view(T, 1), T * per, per)
    kd = k.cuda()
    hw.saf3r_kv_append(cache, batch, kd, torch.zeros_like(kd), hw.make_rope(dims, base, pairing), pos.cuda())
    hw.saf3r_check()
    assert (cache.k_scale == 1.0).all()
    codes = _np(cache.k.float())
    for i in range(T):
        assert np.array_equal(codes[i, :, :per], want[per * i:per * (i + 1)].transpose(1, 0, 2)), rows[i]
