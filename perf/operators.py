"""Cases of the streaming operators: rotary positions with several axes, appending keys and values
to a paged cache, attention over that cache, and the same mask over views held at once.

A model with global attention over views takes its views one after another here: the new tokens'
queries and keys are rotated by their (time, row, column), the keys and values go into a paged
cache (bf16, or e4m3 with a power-of-two scale for each page and head), and the new tokens attend
to the views of a sliding window and to the first tokens of the sequence.

`own` false: the operators in elementary torch operations (32 bits; angles in 64).  `own` true:
this repository's calls.
"""
import math

import numpy as np
import torch

own = False

D = 64
VIEW = 37 * 37 + 5       # tokens of one view: a 37 x 37 patch grid and five special tokens
SMALL_VIEW = 16 * 16 + 5
SCALE = 1.0 / math.sqrt(D)
MIN_EXP, MAX_EXP = -100, 119  # range of a page's power-of-two scale
AXES = {1: (64,), 2: (32, 32), 3: (16, 24, 24)}  # rotated dims of each position axis


def listed():
    return [
        # the adjoint of the rotation for a small four-view layer: fp32 gradients of q and k, three
        # axes, adjacent pairs
        {"name": "rope_grad_s4", "op": "rope", "tokens": 4 * SMALL_VIEW, "heads": 32, "rot": 32, "axes": 3,
         "pairing": "pairs", "base": 10000.0, "view": SMALL_VIEW, "dtype": "fp32", "inverse": True},
        # q, k, v of 32 views out of one projection, token-major, to the head-major rows that the
        # attention takes: q and k rotated by (row, column), v as it is
        {"name": "rope_s32", "op": "rope", "tokens": 32 * VIEW, "heads": 48, "rot": 32, "axes": 2,
         "pairing": "half", "base": 100.0, "view": VIEW, "dtype": "bf16", "inverse": False},
        # 64 streams, one token each, into pages that already hold older tokens
        {"name": "append_tokens64_8bit", "op": "append", "kv": "e4m3", "seqs": 64, "new": 1, "ragged": True,
         "old": 997, "kv_heads": 16, "page": 64, "axes": 2},
        # one view of a stream, from the middle of a page
        {"name": "append_view_8bit", "op": "append", "kv": "e4m3", "seqs": 1, "new": VIEW, "ragged": False,
         "old": 2 * VIEW, "kv_heads": 16, "page": 64, "axes": 2},
        # a view of each of 16 streams, small pages, values held in bf16
        {"name": "append_views16_bf16", "op": "append", "kv": "bf16", "seqs": 16, "new": VIEW, "ragged": False,
         "old": VIEW, "kv_heads": 16, "page": 16, "axes": 3},
        # one token of one stream over four views: latency
        {"name": "attn_token_bf16", "op": "attn", "kv": "bf16", "seqs": 1, "new": 1, "ragged": False,
         "old": 4 * VIEW, "heads": 16, "kv_heads": 16, "page": 64, "view": 1, "window": 0, "sink": 0},
        # one token of each of 64 streams of unequal length, four query heads to a key head
        {"name": "attn_tokens64_8bit", "op": "attn", "kv": "e4m3", "seqs": 64, "new": 1, "ragged": True,
         "old": 16 * VIEW, "heads": 16, "kv_heads": 4, "page": 64, "view": 1, "window": 0, "sink": 0},
        # chunks of unequal length of eight streams, causal by token, a window of tokens and four sinks
        {"name": "attn_chunks8_8bit", "op": "attn", "kv": "e4m3", "seqs": 8, "new": 517, "ragged": True,
         "old": 9001, "heads": 16, "kv_heads": 4, "page": 32, "view": 1, "window": 4096, "sink": 4},
        # one view of one stream over a window of 16 views and the first view
        {"name": "attn_view_8bit", "op": "attn", "kv": "e4m3", "seqs": 1, "new": VIEW, "ragged": False,
         "old": 31 * VIEW, "heads": 16, "kv_heads": 16, "page": 64, "view": VIEW, "window": 16, "sink": VIEW},
        # one view of each of four streams over all their views
        {"name": "attn_views4_bf16", "op": "attn", "kv": "bf16", "seqs": 4, "new": VIEW, "ragged": False,
         "old": 15 * VIEW, "heads": 16, "kv_heads": 16, "page": 64, "view": VIEW, "window": 0, "sink": 0},
        # a small layer with all its views in hand: neighbouring views both ways, and the first
        {"name": "window_s4", "op": "window", "views": 4, "grid": 16, "heads": 4, "window": 2, "sink": SMALL_VIEW,
         "causal": False},
        # 32 views, each over its last eight and the first
        {"name": "window_s32", "op": "window", "views": 32, "grid": 37, "heads": 16, "window": 8, "sink": VIEW,
         "causal": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "window"])
    if op == "rope":
        heads = rng.choice([4, 12, 16, 24, 48])
        return {"op": op, "tokens": _log(rng, 1, 32 * VIEW), "heads": heads,
                "rot": rng.choice([heads, heads - heads // 4, heads // 2]), "axes": rng.choice([1, 2, 3]),
                "pairing": rng.choice(["half", "pairs", "sections"]), "base": rng.choice([100.0, 10000.0]),
                "view": rng.choice([1, SMALL_VIEW, VIEW]), "dtype": rng.choice(["bf16", "fp32"]),
                "inverse": rng.random() < 0.3}
    if op == "append":
        new = rng.choice([1, _log(rng, 2, VIEW), VIEW])
        return {"op": op, "kv": rng.choice(["e4m3", "bf16"]), "seqs": _log(rng, 1, 64 if new == 1 else 16), "new": new,
                "ragged": rng.random() < 0.5, "old": _log(rng, 1, 2 * VIEW), "kv_heads": rng.choice([1, 2, 4, 8, 16]),
                "page": rng.choice([16, 32, 64, 128]), "axes": rng.choice([0, 1, 2, 3])}
    if op == "attn":
        new = rng.choice([1, 1, _log(rng, 2, VIEW), VIEW])
        heads = rng.choice([4, 8, 16])
        view = 1 if new < SMALL_VIEW else rng.choice([1, new])
        windowed = rng.random() < 0.6
        return {"op": op, "kv": rng.choice(["e4m3", "bf16"]), "seqs": _log(rng, 1, 32 if new == 1 else 4), "new": new,
                "ragged": rng.random() < 0.5, "old": _log(rng, 1, 12 * VIEW), "heads": heads,
                "kv_heads": rng.choice([k for k in (1, 2, 4, 8, 16) if heads % k == 0 and heads // k <= 8]),
                "page": rng.choice([16, 32, 64, 128]), "view": view,
                "window": (rng.choice([2, 5]) if view > 1 else _log(rng, 64, 8192)) if windowed else 0,
                "sink": rng.choice([0, 4, view]) if windowed else 0}
    grid = rng.randint(4, 37)
    views = rng.randint(1, max(1, min(32, 32 * VIEW // (grid * grid + 5))))
    return {"op": op, "views": views, "grid": grid, "heads": rng.choice([1, 4, 16]), "window": rng.randint(1, 8),
            "sink": rng.choice([0, 5, grid * grid + 5]), "causal": rng.random() < 0.5}


# ---------------------------------------------------------------- sizes that follow from a case

def _lengths(case):
    """(new tokens, cached tokens with them) of every sequence."""
    q, kv = [], []
    for b in range(case["seqs"]):
        new, old = case["new"], case["old"]
        if case["ragged"]:
            new = 1 + (new - 1) * ((b * 7 + 5) % 11) // 10
            old = 1 + (old - 1) * ((b * 5 + 8) % 13) // 12
        q.append(new)
        kv.append(old + new)
    return q, kv


def _bounds(pos, kv_len, view, window, sink, causal):
    """First and last-plus-one key of the window and end of the sinks, for queries at `pos` (arrays)."""
    f = pos // view
    lo = np.zeros_like(pos) if window == 0 else np.maximum(f - window + 1, 0) * view
    if causal:
        hi = np.minimum((f + 1) * view, kv_len)
        sk = np.minimum(sink, hi)
    else:
        hi = np.full_like(pos, kv_len) if window == 0 else np.minimum((f + window) * view, kv_len)
        sk = np.full_like(pos, min(sink, kv_len))
    return lo, hi, sk


def _pairs_and_keys(pos, kv_len, view, window, sink, causal):
    lo, hi, sk = _bounds(pos, kv_len, view, window, sink, causal)
    pairs = int((hi - lo + np.minimum(sk, lo)).sum())
    keys = int(hi.max() - lo.min() + min(sk.max(), lo.min()))
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "rope":
        el = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * case["heads"] * D
        return {"bytes": 2 * n * el + 4 * case["tokens"] * case["axes"], "flops": 3 * case["tokens"] * case["rot"] * D}
    if op == "append":
        q, _ = _lengths(case)
        n = sum(q) * case["kv_heads"] * D * 2
        return {"bytes": n * 2 + n * (1 if case["kv"] == "e4m3" else 2) + 4 * sum(q) * case["axes"], "flops": 3 * n}
    if op == "attn":
        el = 1 if case["kv"] == "e4m3" else 2
        q, kv = _lengths(case)
        total = {"bytes": sum(q) * case["heads"] * D * 4, "flops": 0}
        for n, m in zip(q, kv):
            pairs, keys = _pairs_and_keys(np.arange(m - n, m), m, case["view"], case["window"], case["sink"], True)
            total["bytes"] += keys * case["kv_heads"] * D * 2 * el
            total["flops"] += 4 * D * pairs * case["heads"]
        return total
    v = case["grid"] ** 2 + 5
    n = case["views"] * v
    pairs, _ = _pairs_and_keys(np.arange(n), n, v, case["window"], case["sink"], case["causal"])
    return {"bytes": n * case["heads"] * D * 8,
            "flops": 4 * D * pairs * case["heads"]}


# ---------------------------------------------------------------- inputs

def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def _positions(g, tokens, axes, view):
    """(time, row, column) of consecutive views' tokens, special tokens at row and column 0; the
    stream began at any time.  One axis: the time of each token."""
    i = torch.arange(tokens, device="cuda")
    start = torch.randint(0, 100000, (1,), device="cuda", generator=g)
    if axes == 1:
        return (start + i).to(torch.int32)[:, None].contiguous()
    patch = torch.clamp(i % view - 5, min=-1)
    side = max(1, math.isqrt(max(view - 5, 1)))
    row = torch.where(patch >= 0, patch // side + 1, 0)
    col = torch.where(patch >= 0, patch % side + 1, 0)
    cols = [start + i // view, row, col] if axes == 3 else [row, col]
    return torch.stack(cols, 1).to(torch.int32).contiguous()


def _pairing(axes, pairing, base):
    """The 32 pairs at most: first dim, second dim, axis and frequency of each."""
    dims, a, b, ax, fr, at = AXES[axes], [], [], [], [], 0
    width = sum(dims)
    for n, d in enumerate(dims):
        for i in range(d // 2):
            if pairing == "half":
                a.append(at + i), b.append(at + i + d // 2), fr.append(base ** (-2.0 * i / d))
            elif pairing == "pairs":
                a.append(at + 2 * i), b.append(at + 2 * i + 1), fr.append(base ** (-2.0 * i / d))
            else:  # one rotation over the whole width, whose frequencies are dealt out to the axes
                j = at // 2 + i
                a.append(j), b.append(j + width // 2), fr.append(base ** (-2.0 * j / width))
            ax.append(n)
        at += d
    return a, b, ax, fr


def _tables(s, case_axes, pairing, base):
    a, b, ax, fr = _pairing(case_axes, pairing, base)
    s["a"], s["b"], s["ax"] = (torch.tensor(x, device="cuda") for x in (a, b, ax))
    s["fr"] = torch.tensor(fr, dtype=torch.float64, device="cuda")


def _paged(s, case, g, need=None):
    """Pools, page table and lengths of a batch; `need(b, page)`: whether a page is still held."""
    q, kv = _lengths(case)
    page, hk = case["page"], case["kv_heads"]
    counts = [-(-m // page) for m in kv]
    held = [[p for p in range(n) if need is None or need(b, p)] for b, n in enumerate(counts)]
    pages = sum(len(h) for h in held) + 3
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).cpu().numpy()
    table, at = np.full((case["seqs"], max(counts)), -1, dtype=np.int32), 0
    for b, h in enumerate(held):
        table[b, h] = ids[at:at + len(h)]
        at += len(h)
    s["table"] = torch.from_numpy(table).cuda()
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(q)]).astype(np.int32)).cuda()
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["tokens"], s["max_new"], s["max_kv"] = sum(q), max(q), max(kv)
    shape = (pages, hk, page, D)
    for n in ("k", "v"):
        x = torch.randn(shape, device="cuda", generator=g)
        if case["kv"] == "e4m3":
            s[n + "_pool"] = (x * 96).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[n + "_scale"] = torch.exp2(-torch.randint(6, 8, (pages, hk), device="cuda", generator=g).float())
        else:
            s[n + "_pool"], s[n + "_scale"] = x.to(torch.bfloat16), None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        s["x"] = torch.randn((t, h, D), device="cuda", generator=g).to(_dtype(case["dtype"]))
        s["pos"] = _positions(g, t, case["axes"], case["view"])
        s["out"] = torch.empty((h, t, D), dtype=s["x"].dtype, device="cuda").transpose(0, 1)
        _tables(s, case["axes"], case["pairing"], case["base"])
    elif op == "append":
        _paged(s, case, g)
        kv = torch.randn((s["tokens"], 2, case["kv_heads"], D), device="cuda", generator=g).to(torch.bfloat16)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        if case["axes"]:
            s["pos"] = _positions(g, s["tokens"], case["axes"], VIEW)
            _tables(s, case["axes"], "half", 100.0)
    elif op == "attn":
        q, kv = _lengths(case)
        span = []  # of each sequence: the sinks' end and the first key of the window
        for n, m in zip(q, kv):
            lo, _, sk = _bounds(np.arange(m - n, m), m, case["view"], case["window"], case["sink"], True)
            span.append((int(sk.max()), int(lo.min())))
        page = case["page"]
        _paged(s, case, g, lambda b, p: p * page < span[b][0] or (p + 1) * page > span[b][1])
        s["q"] = (2 * torch.randn((case["heads"], s["tokens"], D), device="cuda", generator=g)).to(
            torch.bfloat16).transpose(0, 1)
        s["out"] = torch.empty((case["heads"], s["tokens"], D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    else:
        n = case["views"] * (case["grid"] ** 2 + 5)
        for name in ("q", "k", "v"):
            x = torch.randn((case["heads"], n, D), device="cuda", generator=g)
            s[name] = (2 * x if name == "q" else x).to(torch.bfloat16)
        s["out"] = torch.empty((case["heads"], n, D), dtype=torch.bfloat16, device="cuda")
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    """What a program that makes the framework's calls keeps: configurations, cache and batch handles, workspace."""
    import head_wise_dynamic_b200 as hw
    op = case["op"]
    pairing = {"half": hw.ROPE_HALF, "pairs": hw.ROPE_PAIRS, "sections": hw.ROPE_SECTIONS}
    if op == "rope":
        s["rope"] = hw.make_rope(AXES[case["axes"]], case["base"], pairing[case["pairing"]])
    if op in ("append", "attn"):
        s["cache"] = hw.PagedKV(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        s["batch"] = hw.KVBatch(s["cu"], s["kv_lens"], s["table"], s["tokens"], s["max_new"])
    if op == "append":
        s["rope"] = hw.make_rope(AXES[case["axes"]], 100.0, hw.ROPE_HALF) if case["axes"] else None
    if op == "attn":
        s["mask"] = hw.make_window(case["view"], case["window"], case["sink"])
        s["ws"] = torch.empty(hw.saf3r_kv_attn_workspace_bytes(s["cache"], s["batch"], s["mask"], case["heads"]),
                              dtype=torch.uint8, device="cuda")
    if op == "window":
        s["layout"] = hw.make_layout(case["views"], case["grid"], H=case["heads"])
        s["mask"] = hw.make_window(case["grid"] ** 2 + 5, case["window"], case["sink"], case["causal"])
        s["ws"] = torch.empty(hw.saf3r_window_attn_workspace_bytes(s["layout"], s["mask"]), dtype=torch.uint8,
                              device="cuda")


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import head_wise_dynamic_b200 as hw
        if op == "rope":
            hw.saf3r_rope(s["rope"], s["x"], s["pos"], s["out"], n_rot_heads=s["case"]["rot"], inverse=s["case"]["inverse"])
            return s["out"]
        if op == "append":
            hw.saf3r_kv_append(s["cache"], s["batch"], s["k"], s["v"], s["rope"], s.get("pos"))
            return _cache_out(s)
        if op == "attn":
            hw.saf3r_kv_attn(s["cache"], s["batch"], s["mask"], s["q"], s["out"], s["ws"])
            return s["out"]
        hw.saf3r_window_attn(s["layout"], s["mask"], s["q"], s["k"], s["v"], s["out"], s["ws"])
        return s["out"]
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "window": _plain_window}[op](s)


def _cache_out(s):
    """The cache after an append: its values (8-bit ones as float8) and scales."""
    return {n: s[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale") if s[n] is not None}


def _rotate(s, x, inverse=False):
    """x [T, h, 64] in 32 bits, rotated (angles in 64)."""
    ang = s["pos"].double()[:, s["ax"]] * s["fr"]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if inverse:
        sin = -sin
    y = x.clone()
    a, b = x[..., s["a"]], x[..., s["b"]]
    y[..., s["a"]] = a * cos - b * sin
    y[..., s["b"]] = a * sin + b * cos
    return y


def _plain_rope(s):
    c = s["case"]
    x = s["x"].float()
    y = torch.cat([_rotate(s, x[:, :c["rot"]], c["inverse"]), x[:, c["rot"]:]], 1)
    s["out"].copy_(y)
    return s["out"]


def _slots(s):
    """Sequence, page and row in the page of every new token, and its page's first row that is new."""
    t = torch.arange(s["tokens"], device="cuda")
    cu, page = s["cu"].long(), s["case"]["page"]
    b = torch.searchsorted(cu, t, right=True) - 1
    start = (s["kv_lens"] - (s["cu"][1:] - s["cu"][:-1])).long()[b]
    p = start + t - cu[b]
    first = torch.clamp(start - p // page * page, min=0)
    return s["table"].long()[b, p // page], p % page, first


def _plain_append(s):
    k, v = s["k"].float(), s["v"].float()
    if "pos" in s:
        k = _rotate(s, k)
    pages, rows, first = _slots(s)
    for n, x in (("k", k), ("v", v)):
        pool, scale = s[n + "_pool"], s[n + "_scale"]
        if scale is None:
            pool[pages, :, rows] = x.to(torch.bfloat16)
            continue
        fine = torch.isfinite(x)
        amax = torch.where(fine, x.abs(), 0.0).amax(-1)                                       # [T, heads]
        most = torch.zeros_like(scale).index_reduce_(0, pages, amax, "amax")
        m, e = torch.frexp(most)
        e = torch.where(most > 0, e - 9 + (m > 0.875), MIN_EXP).clamp(MIN_EXP, MAX_EXP)
        need = ((e + 127) << 23).to(torch.int32).view(torch.float32)
        start = torch.zeros(pool.shape[0], dtype=torch.long, device="cuda").index_put_((pages,), first)
        at = torch.zeros(pool.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, pages, True).nonzero()[:, 0]
        was, start = scale[at], start[at]
        now = torch.where(start[:, None] > 0, torch.maximum(need[at], was), need[at])
        old = pool[at]
        kept = torch.arange(old.shape[2], device="cuda") < start[:, None]
        again = (old.float() * (was / now)[:, :, None, None]).to(pool.dtype)
        bits = torch.where(kept[:, None, :, None], again.view(torch.uint8), old.view(torch.uint8))
        pool.view(torch.uint8)[at] = bits
        scale[at] = now
        x = torch.where(fine, (x / scale[pages][:, :, None]).clamp(-448, 448), float("nan"))
        pool.view(torch.uint8)[pages, :, rows] = x.to(pool.dtype).view(torch.uint8)
    return _cache_out(s)


def _softmax_rows(q, k, v, keep):
    """Masked attention in 32 bits: q [..., n, 64], k and v [..., m, 64], keep [..., n, m]."""
    x = (q @ k.transpose(-1, -2)).mul_(SCALE).masked_fill_(~keep, float("-inf"))
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    return x @ v


def _keep(pos, kv_len, keys, view, window, sink, causal):
    """[..., queries, keys] truth values: which keys a query at `pos` sees."""
    f, g = pos[..., :, None] // view, keys // view
    near = g <= f if causal else torch.ones_like(g <= f)
    recent = near if window == 0 else near & (g > f - window) & (g < f + window)
    return (recent | (near & (keys < sink))) & (keys < kv_len)


def _values(s, n):
    """The cached keys or values of every sequence as 32-bit rows [seqs, heads, keys, 64]."""
    at = s["table"].long().clamp(min=0)
    x = s[n + "_pool"][at].float()
    if s[n + "_scale"] is not None:
        x *= s[n + "_scale"][at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, D)


def _plain_attn(s):
    c = s["case"]
    k, v = _values(s, "k"), _values(s, "v")
    cu, n = s["cu"].long(), s["max_new"]
    new = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=s["tokens"] - 1)
    pos = s["kv_lens"].long()[:, None] - new[:, None] + torch.minimum(i, new[:, None] - 1)
    keep = _keep(pos, s["kv_lens"].long()[:, None, None], torch.arange(k.shape[2], device="cuda"), c["view"],
                 c["window"], c["sink"], True)[:, None]
    q = s["q"].float()[at].transpose(1, 2)                                                    # [seqs, heads, n, 64]
    b = torch.searchsorted(cu, torch.arange(s["tokens"], device="cuda"), right=True) - 1
    row = torch.arange(s["tokens"], device="cuda") - cu[b]
    g = c["heads"] // c["kv_heads"]
    for h in range(c["kv_heads"]):
        o = _softmax_rows(q[:, h * g:(h + 1) * g], k[:, h:h + 1], v[:, h:h + 1], keep)
        s["out"][:, h * g:(h + 1) * g] = o[b, :, row].to(s["out"].dtype)
    return s["out"]


def _plain_window(s):
    c = s["case"]
    i = torch.arange(s["q"].shape[1], device="cuda")
    keep = _keep(i, len(i), i, c["grid"] ** 2 + 5, c["window"], c["sink"], c["causal"])
    for h in range(c["heads"]):
        s["out"][h] = _softmax_rows(s["q"][h].float(), s["k"][h].float(), s["v"][h].float(), keep).to(s["out"].dtype)
    return s["out"]


# ---------------------------------------------------------------- 64 bits, from the definitions

def _turned(x, pos, axes, pairing, base, inverse=False):
    """x [T, h, 64] as complex numbers a + ib times e^(i angle)."""
    a, b, ax, fr = _pairing(axes, pairing, base)
    ang = torch.stack([pos[:, n].double() * f for n, f in zip(ax, fr)], 1)
    z = torch.complex(x[..., a].double(), x[..., b].double()) * torch.polar(
        torch.ones_like(ang), -ang if inverse else ang)[:, None]
    y = x.double().clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_append(s, case):
    q, kv = _lengths(case)
    page = case["page"]
    table = s["table"].cpu().numpy()
    rows = {"k": _turned(s["k"], s["pos"], case["axes"], "half", 100.0) if case["axes"] else s["k"].double(),
            "v": s["v"].double()}
    got = {}
    for n, x in rows.items():
        pool, scale = s[n + "_pool"].double(), s[n + "_scale"]
        scale = None if scale is None else scale.double()
        t = 0
        for b, (new, end) in enumerate(zip(q, kv)):
            p = end - new
            while p < end:  # page by page
                r, here = p % page, int(table[b, p // page])
                m = min(page - r, end - p)
                part = x[t:t + m].transpose(0, 1)
                if scale is not None:
                    most = part.abs().amax((1, 2)).clamp(min=2.0 ** -120)
                    e = torch.ceil(torch.log2(most / 448.0)).clamp(MIN_EXP, MAX_EXP)
                    want = torch.exp2(e)
                    if r > 0:
                        want = torch.maximum(want, scale[here])
                        old = pool[here, :, :r] * (scale[here] / want)[:, None, None]
                        pool[here, :, :r] = old.float().to(torch.float8_e4m3fn).double()
                    scale[here] = want
                    part = (part / want[:, None, None]).float().to(torch.float8_e4m3fn).double()
                pool[here, :, r:r + m] = part
                t += m
                p += m
        got[n + "_pool"] = pool
        if scale is not None:
            got[n + "_scale"] = scale
    return got


def _exact_rows(q, k, v, seen):
    x = torch.einsum("hnd,hmd->hnm", q, k) * SCALE
    return torch.einsum("hnm,hmd->hnd", torch.softmax(torch.where(seen, x, float("-inf")), -1), v)


def _seen(pos, kv_len, view, window, sink, causal):
    lo, hi, sk = (torch.from_numpy(np.asarray(x)).cuda()[:, None] for x in _bounds(pos, kv_len, view, window, sink, causal))
    j = torch.arange(kv_len, device="cuda")
    return ((j >= lo) & (j < hi)) | (j < sk)


def _exact_attn(s, case):
    q, kv = _lengths(case)
    g, t = case["heads"] // case["kv_heads"], 0
    out = torch.empty((s["tokens"], case["heads"], D), dtype=torch.float64, device="cuda")
    for b, (new, end) in enumerate(zip(q, kv)):
        at = s["table"][b, :-(-end // case["page"])].long().clamp(min=0)
        k, v = ((s[n + "_pool"][at].double() * (1.0 if s[n + "_scale"] is None else
                                                s[n + "_scale"][at].double()[..., None, None]))
                .transpose(0, 1).reshape(case["kv_heads"], -1, D)[:, :end] for n in ("k", "v"))
        for i in range(0, new, 256):
            n = min(256, new - i)
            seen = _seen(np.arange(end - new + i, end - new + i + n), end, case["view"], case["window"], case["sink"], True)
            for h in range(case["kv_heads"]):
                x = s["q"][t + i:t + i + n, h * g:(h + 1) * g].double().transpose(0, 1)
                o = _exact_rows(x, k[h:h + 1].expand(g, -1, -1), v[h:h + 1].expand(g, -1, -1), seen)
                out[t + i:t + i + n, h * g:(h + 1) * g] = o.transpose(0, 1)
        t += new
    return out


def _exact_window(s, case):
    n, v = s["q"].shape[1], case["grid"] ** 2 + 5
    out = torch.empty((case["heads"], n, D), dtype=torch.float64, device="cuda")
    for i in range(0, n, 4096):
        pos = np.arange(i, min(i + 4096, n))
        seen = _seen(pos, n, v, case["window"], case["sink"], case["causal"])
        for h in range(case["heads"]):
            out[h, i:i + len(pos)] = _exact_rows(s["q"][h:h + 1, i:i + len(pos)].double(), s["k"][h:h + 1].double(),
                                                 s["v"][h:h + 1].double(), seen)[0]
    return out


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "rope":
        x, r = s["x"], case["rot"]
        return torch.cat([_turned(x[:, :r], s["pos"], case["axes"], case["pairing"], case["base"], case["inverse"]),
                          x[:, r:].double()], 1)
    if case["op"] == "append":
        return _exact_append(s, case)
    return _exact_attn(s, case) if case["op"] == "attn" else _exact_window(s, case)
