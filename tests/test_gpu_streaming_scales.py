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
