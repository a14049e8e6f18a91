"""fp64 restatement of the streaming operators: rotary positions with several axes, appending to a
paged cache (bf16, or e4m3 with a power-of-two scale for each page and head), and attention with
views, a sliding window and sinks.  Plain loops over numpy arrays; shares no code with the library."""
import math

import numpy as np

HALF, PAIRS, SECTIONS = range(3)
BF16, E4M3 = range(2)
MIN_EXP, MAX_EXP = -100, 119


# ------------------------------------------------------------------ roundings

def round_bf16(x):
    """fp64 -> nearest bf16 (ties to even), normal range."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(x), where=(x != 0) & np.isfinite(x), out=np.zeros_like(x)))
    step = np.exp2(np.maximum(e, -126) - 7)
    return np.where(np.isfinite(x), np.rint(x / step) * step, x)


def round_e4m3(x):
    """fp64 -> nearest e4m3 value (ties to even, saturating at 448); infinities and NaN become NaN."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    a = np.where(ok, np.abs(x), 0.0)
    _, e = np.frexp(np.maximum(a, 2.0 ** -30))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    r = np.minimum(np.rint(a / step) * step, 448.0)
    return np.where(ok, np.copysign(r, x), np.nan)


# ------------------------------------------------------------------ rotary positions

def rope_pairs(dims, base, pairing):
    """[(first dim, second dim, axis, frequency)] of every rotated pair."""
    out, at, width = [], 0, sum(dims)
    for axis, d in enumerate(dims):
        for i in range(d // 2):
            j = at // 2 + i
            if pairing == HALF:
                out.append((at + i, at + d // 2 + i, axis, base ** (-2.0 * i / d)))
            elif pairing == PAIRS:
                out.append((at + 2 * i, at + 2 * i + 1, axis, base ** (-2.0 * i / d)))
            else:
                out.append((j, j + width // 2, axis, base ** (-2.0 * j / width)))
        at += d
    return out


def rope(x, pos, dims, base, pairing, n_rot=None, inverse=False):
    """x [T, h, 64] with its first n_rot heads rotated by pos [T, axes]."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    n = x.shape[1] if n_rot is None else n_rot
    for a, b, axis, freq in rope_pairs(dims, base, pairing):
        ang = np.asarray(pos)[:, axis].astype(np.float64) * freq
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1.0 if inverse else 1.0)
        y[:, :n, a] = x[:, :n, a] * c - x[:, :n, b] * s
        y[:, :n, b] = x[:, :n, a] * s + x[:, :n, b] * c
    return y


# ------------------------------------------------------------------ the paged cache

def scale_of(m):
    """Power-of-two scale that the magnitude m needs."""
    if m == 0:
        return 2.0 ** MIN_EXP
    f, e = math.frexp(m)  # m = f * 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
    return 2.0 ** min(max(e - 9 + (f > 0.875), MIN_EXP), MAX_EXP)


def append(pool, scale, x, cu, kv_lens, table, page):
    """Rows x [T, heads, 64] (fp64) into pool [pages, heads, page, 64] (the values that codes stand for before
    scaling, fp64), in place; scale [pages, heads] fp64 or None (bf16)."""
    for b in range(len(kv_lens)):
        new = int(cu[b + 1] - cu[b])
        p, end, t = int(kv_lens[b]) - new, int(kv_lens[b]), int(cu[b])
        while p < end:
            pg, r = int(table[b][p // page]), p % page
            n = min(page - r, end - p)
            for h in range(x.shape[1]):
                rows = x[t:t + n, h]
                if scale is None:
                    pool[pg, h, r:r + n] = round_bf16(rows)
                    continue
                fine = np.abs(rows[np.isfinite(rows)])
                s = scale_of(float(fine.max()) if fine.size else 0.0)
                if r > 0:
                    if s > scale[pg, h]:
                        pool[pg, h, :r] = round_e4m3(pool[pg, h, :r] * (scale[pg, h] / s))
                    s = max(s, float(scale[pg, h]))
                scale[pg, h] = s
                pool[pg, h, r:r + n] = round_e4m3(rows / s)
            p, t = p + n, t + n


def cached_rows(pool, scale, table, n, page):
    """The first n rows of one sequence, [n, heads, 64] (rows of pages that the table does not hold: NaN)."""
    out = np.full((n, pool.shape[1], pool.shape[3]), np.nan)
    for i in range(0, n, page):
        pg = int(table[i // page])
        if 0 <= pg < pool.shape[0]:
            rows = pool[pg] if scale is None else pool[pg] * scale[pg][:, None, None]
            m = min(page, n - i)
            out[i:i + m] = rows[:, :m].transpose(1, 0, 2)
    return out


# ------------------------------------------------------------------ attention

def seen(p, n, view, window, sink, causal):
    """[n] truth values: which tokens the query at position p sees."""
    j = np.arange(n)
    f, g = p // view, j // view
    side = g <= f if causal else np.ones(n, dtype=bool)
    near = side if window == 0 else side & (g > f - window) & (g < f + window)
    return near | (side & (j < sink))


def attend(q, k, v, pos, view, window, sink, causal):
    """q [t, 64] at positions pos over k, v [n, 64]: rows that see nothing are zero."""
    out = np.zeros((len(q), v.shape[1]))
    for i, p in enumerate(pos):
        j = seen(int(p), len(k), view, window, sink, causal)
        if j.any():
            s = k[j] @ q[i] / 8.0
            w = np.exp(s - s.max())
            out[i] = (w / w.sum()) @ v[j]
    return out
