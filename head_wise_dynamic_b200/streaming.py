"""Streaming operators: views taken one after another.

Rotary positions with several axes, appending keys and values to a paged cache (bf16, or 8-bit with
a scale for each page and head), attention of the new tokens over the cache, and the same
sliding-window mask over views held at once.  Bindings of the entry points of include/saf3r.h; they
check shapes, types and devices, and launch on the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import head_wise_dynamic_b200 as _hw

__all__ = ["ROPE_HALF", "ROPE_PAIRS", "ROPE_SECTIONS", "KV_BF16", "KV_E4M3", "make_rope", "PagedKV", "KVBatch",
           "make_window", "saf3r_rope", "saf3r_kv_append", "saf3r_kv_attn", "saf3r_kv_attn_workspace_bytes",
           "saf3r_window_attn", "saf3r_window_attn_workspace_bytes"]

# saf3r_rope_pairing
ROPE_HALF, ROPE_PAIRS, ROPE_SECTIONS = range(3)
# saf3r_kv_type
KV_BF16, KV_E4M3 = range(2)

torch = None  # loaded by the first call or handle that takes tensors


def _load_torch():
    global torch
    import torch as t
    torch = t


_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_ref = ctypes.byref


class saf3r_rope_cfg(ctypes.Structure):
    _fields_ = [("n_axes", _i32), ("pairing", _i32), ("dims", _i32 * 4), ("base", ctypes.c_double)]


class saf3r_rope_args(ctypes.Structure):
    _fields_ = [("n_tokens", _i64), ("n_heads", _i32), ("n_rot_heads", _i32),
                ("x", _vp), ("x_token_stride", _i64), ("x_head_stride", _i64),
                ("out", _vp), ("out_token_stride", _i64), ("out_head_stride", _i64),
                ("x_is_fp32", _i32), ("out_is_fp32", _i32), ("pos", _vp), ("inverse", _i32)]


class saf3r_kv_cache(ctypes.Structure):
    _fields_ = [("n_pages", _i32), ("n_heads", _i32), ("page", _i32), ("type", _i32),
                ("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp)]


class saf3r_kv_batch(ctypes.Structure):
    _fields_ = [("n_seqs", _i32), ("n_tokens", _i32), ("max_new", _i32), ("max_pages", _i32),
                ("cu_tokens", _vp), ("kv_lens", _vp), ("page_table", _vp)]


class saf3r_kv_rows(ctypes.Structure):
    _fields_ = [("k", _vp), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v", _vp), ("v_token_stride", _i64), ("v_head_stride", _i64), ("pos", _vp)]


class saf3r_window(ctypes.Structure):
    _fields_ = [("view_tokens", _i32), ("window", _i32), ("n_sink", _i32), ("causal", _i32)]


class saf3r_query_rows(ctypes.Structure):
    _fields_ = [("n_heads", _i32), ("out_is_fp32", _i32), ("q", _vp), ("q_token_stride", _i64), ("q_head_stride", _i64),
                ("out", _vp), ("out_token_stride", _i64), ("out_head_stride", _i64)]


def declare(L) -> None:
    """Argument types of the streaming entry points of the loaded library."""
    P = ctypes.POINTER
    L.saf3r_rope.argtypes = [P(saf3r_rope_cfg), P(saf3r_rope_args), _vp]
    L.saf3r_kv_append.argtypes = [P(saf3r_kv_cache), P(saf3r_kv_batch), P(saf3r_rope_cfg), P(saf3r_kv_rows), _vp]
    L.saf3r_kv_attn.argtypes = [P(saf3r_kv_cache), P(saf3r_kv_batch), P(saf3r_window), P(saf3r_query_rows), _vp, _vp]
    L.saf3r_window_attn.argtypes = [P(_hw.saf3r_layout), P(saf3r_window), _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp]
    for f in (L.saf3r_rope, L.saf3r_kv_append, L.saf3r_kv_attn, L.saf3r_window_attn):
        f.restype = ctypes.c_int
    L.saf3r_kv_attn_workspace_bytes.argtypes = [P(saf3r_kv_cache), P(saf3r_kv_batch), P(saf3r_window), ctypes.c_int]
    L.saf3r_window_attn_workspace_bytes.argtypes = [P(_hw.saf3r_layout), P(saf3r_window)]
    for f in (L.saf3r_kv_attn_workspace_bytes, L.saf3r_window_attn_workspace_bytes):
        f.restype = ctypes.c_size_t


# ------------------------------------------------------------------ configurations

def make_rope(dims: Sequence[int], base: float = 100.0, pairing: int = ROPE_HALF) -> saf3r_rope_cfg:
    """Rotary positions with one axis for each entry of `dims` (rotated dims of the axis)."""
    if not 1 <= len(dims) <= 4:
        raise ValueError("1 to 4 axes")
    return saf3r_rope_cfg(len(dims), int(pairing), (_i32 * 4)(*[int(d) for d in dims]), float(base))


def make_window(view_tokens: int = 1, window: int = 0, n_sink: int = 0, causal: bool = True) -> saf3r_window:
    """Which tokens a query sees: the last `window` views (0: all) and the first n_sink tokens."""
    return saf3r_window(int(view_tokens), int(window), int(n_sink), int(bool(causal)))


# ------------------------------------------------------------------ checks
#
# A small step's call is as long as its checks: they compare first and word an error only when there is one.

def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _dense(t, dtype, shape, device, what: str):
    """A contiguous tensor of this type, shape and device: its address."""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor {tuple(shape)} on {device} is wanted, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _row_strides(t, tokens: int, heads: int, device, what: str):
    """A [tokens, heads, 64] tensor in any order of its rows: its token and head strides."""
    if t.shape != (tokens, heads, 64) or t.device != device:
        raise ValueError(f"{what}: a tensor [{tokens}, {heads}, 64] on {device} is wanted, got {tuple(t.shape)} on {t.device}")
    a, b, c = t.stride()
    if c != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    # the stride of a dimension of one says nothing: any valid one will do
    return (a if tokens > 1 else 64), (b if heads > 1 else 64)


def _workspace(t, n: int, device):
    if t.device != device or t.numel() * t.element_size() < n or not t.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor of at least {n} bytes on {device} is wanted")
    return t.data_ptr()


def _launch(device, stream, call, *args):
    """call(*args, stream) with the tensors' device as the current one; without `stream` on torch's current stream."""
    if device.type != "cuda":
        raise ValueError(f"CUDA tensors are wanted, got some on {device}")
    index = device.index
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        status = call(*args, stream)
    else:
        with torch.cuda.device(device):
            status = call(*args, stream)
    if status:
        _hw._check(status, call.__name__)


# ------------------------------------------------------------------ handles

class PagedKV:
    """A paged cache: pools k and v [n_pages, kv heads, page, 64] (bf16, or float8_e4m3fn with the
    fp32 scales [n_pages, kv heads]).  The tensors stay the caller's."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if torch is None:
            _load_torch()
        _need(k.dim() == 4 and k.shape[3] == 64, "k: a pool [n_pages, kv heads, page, 64] is wanted")
        _need(k.dtype in (torch.bfloat16, torch.float8_e4m3fn), f"k: bfloat16 or float8_e4m3fn is wanted, got {k.dtype}")
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.device
        self.n_pages, self.n_heads, self.page = (int(n) for n in k.shape[:3])
        eight = k.dtype == torch.float8_e4m3fn
        kp = _dense(k, k.dtype, k.shape, k.device, "k")
        vp = _dense(v, k.dtype, k.shape, k.device, "v")
        sk = sv = None
        if eight:
            _need(k_scale is not None and v_scale is not None, "an 8-bit cache has k_scale and v_scale")
            sk = _dense(k_scale, torch.float32, k.shape[:2], k.device, "k_scale")
            sv = _dense(v_scale, torch.float32, k.shape[:2], k.device, "v_scale")
        self.c = saf3r_kv_cache(self.n_pages, self.n_heads, self.page, KV_E4M3 if eight else KV_BF16, kp, vp, sk, sv)
        self.ref = _ref(self.c)

    @classmethod
    def empty(cls, n_pages: int, n_heads: int, page: int = 64, kv_type: int = KV_E4M3, device="cuda") -> "PagedKV":
        """A cache over newly allocated tensors (nothing in them needs a start value)."""
        if torch is None:
            _load_torch()
        shape = (n_pages, n_heads, page, 64)
        dt = torch.float8_e4m3fn if kv_type == KV_E4M3 else torch.bfloat16
        k, v = (torch.empty(shape, dtype=dt, device=device) for _ in range(2))
        if kv_type != KV_E4M3:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))


class KVBatch:
    """The new tokens of one step (see saf3r_kv_batch): int32 tensors cu_tokens [n_seqs + 1], kv_lens
    [n_seqs] (with the new tokens) and page_table [n_seqs, max_pages], the rows n_tokens of the step's
    tensors and the most new tokens of one sequence.  The tensors' contents may change between calls."""

    def __init__(self, cu_tokens, kv_lens, page_table, n_tokens: int, max_new: int):
        if torch is None:
            _load_torch()
        n = kv_lens.shape[0]
        self.cu_tokens, self.kv_lens, self.page_table, self.device = cu_tokens, kv_lens, page_table, kv_lens.device
        self.n_seqs, self.n_tokens, self.max_new = int(n), int(n_tokens), int(max_new)
        _need(page_table.dim() == 2, "page_table: a tensor [n_seqs, max_pages] is wanted")
        self.c = saf3r_kv_batch(
            self.n_seqs, self.n_tokens, self.max_new, int(page_table.shape[1]),
            _dense(cu_tokens, torch.int32, (n + 1,), self.device, "cu_tokens"),
            _dense(kv_lens, torch.int32, (n,), self.device, "kv_lens"),
            _dense(page_table, torch.int32, (n, page_table.shape[1]), self.device, "page_table"))
        self.workspace_bytes = {}
        self.ref = _ref(self.c)


# ------------------------------------------------------------------ the calls

def saf3r_rope(rope, x, pos, out, n_rot_heads: Optional[int] = None, inverse: bool = False, stream=None):
    """Rotate the first n_rot_heads heads (default: all) of x [tokens, heads, 64] by pos [tokens, axes]
    (int32) into out [tokens, heads, 64]; the other heads are copied.  x and out are bf16 or fp32, their rows
    in any order (out may be a transposed head-major tensor).  inverse: the adjoint."""
    if torch is None:
        _load_torch()
    T, H, dev = x.shape[0], x.shape[1], x.device
    xf, of = x.dtype == torch.float32, out.dtype == torch.float32
    _need((xf or x.dtype == torch.bfloat16) and (of or out.dtype == torch.bfloat16), "x and out: bfloat16 or float32")
    xt, xh = _row_strides(x, T, H, dev, "x")
    ot, oh = _row_strides(out, T, H, dev, "out")
    a = saf3r_rope_args(T, H, H if n_rot_heads is None else int(n_rot_heads), x.data_ptr(), xt, xh, out.data_ptr(), ot, oh,
                        xf, of, _dense(pos, torch.int32, (T, rope.n_axes), dev, "pos"), bool(inverse))
    _launch(dev, stream, _hw.lib().saf3r_rope, _ref(rope), _ref(a))


def saf3r_kv_append(cache: PagedKV, batch: KVBatch, k, v, rope=None, pos=None, stream=None):
    """Append the step's rows k, v [n_tokens, kv heads, 64] (bf16) to the cache; with `rope` the keys
    are rotated by pos [n_tokens, axes] (int32) on the way."""
    dev, T, H = cache.device, batch.n_tokens, cache.n_heads
    _need(batch.device == dev and k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16,
          "k and v: bfloat16 tensors, the batch on the cache's device")
    kt, kh = _row_strides(k, T, H, dev, "k")
    vt, vh = _row_strides(v, T, H, dev, "v")
    pp = None
    if rope is not None:
        _need(pos is not None, "a rope needs pos")
        pp = _dense(pos, torch.int32, (T, rope.n_axes), dev, "pos")
    a = saf3r_kv_rows(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, pp)
    _launch(dev, stream, _hw.lib().saf3r_kv_append, cache.ref, batch.ref, None if rope is None else _ref(rope), _ref(a))


def saf3r_kv_attn_workspace_bytes(cache: PagedKV, batch: KVBatch, window: saf3r_window, n_heads: int) -> int:
    """Workspace bytes of saf3r_kv_attn for n_heads query heads (ValueError for sizes it does not take)."""
    n = int(_hw.lib().saf3r_kv_attn_workspace_bytes(cache.ref, batch.ref, _ref(window), int(n_heads)))
    _need(n > 0, "sizes that saf3r_kv_attn does not take")
    return n


def saf3r_kv_attn(cache: PagedKV, batch: KVBatch, window: saf3r_window, q, out, workspace, stream=None):
    """Attention of the step's queries q [n_tokens, heads, 64] (bf16) over the cache, which holds the step's
    keys and values already, into out [n_tokens, heads, 64] (bf16 or fp32, not in q's place); rows in any order."""
    dev, T, H = cache.device, batch.n_tokens, q.shape[1]
    fp32 = out.dtype == torch.float32
    _need(batch.device == dev and q.dtype == torch.bfloat16 and (fp32 or out.dtype == torch.bfloat16),
          "q: bfloat16, out: bfloat16 or float32, the batch on the cache's device")
    qt, qh = _row_strides(q, T, H, dev, "q")
    ot, oh = _row_strides(out, T, H, dev, "out")
    sizes = (cache.n_heads, H)  # with the batch's own, all that the workspace depends on
    need = batch.workspace_bytes.get(sizes)
    if need is None:
        need = batch.workspace_bytes[sizes] = saf3r_kv_attn_workspace_bytes(cache, batch, window, H)
    ws = _workspace(workspace, need, dev)
    a = saf3r_query_rows(H, fp32, q.data_ptr(), qt, qh, out.data_ptr(), ot, oh)
    _launch(dev, stream, _hw.lib().saf3r_kv_attn, cache.ref, batch.ref, _ref(window), _ref(a), ws)


def saf3r_window_attn_workspace_bytes(layout, window: saf3r_window) -> int:
    n = int(_hw.lib().saf3r_window_attn_workspace_bytes(_ref(_hw.layout_of(layout)), _ref(window)))
    _need(n > 0, "a layout or window that saf3r_window_attn does not take")
    return n


def saf3r_window_attn(layout, window: saf3r_window, q, k, v, out, workspace, stream=None):
    """Attention with a sliding window of views and sinks over q, k, v [H, N, 64] (bf16) held at once,
    into out [H, N, 64] (bf16 or fp32, in none of their places)."""
    if torch is None:
        _load_torch()
    L = _hw.layout_of(layout)
    dev, shape = q.device, (L.H, L.S * (L.grid_h * L.grid_w + L.n_special), L.d)
    fp32 = out.dtype == torch.float32
    qp, kp, vp = (_dense(t, torch.bfloat16, shape, dev, n) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    op = _dense(out, torch.float32 if fp32 else torch.bfloat16, shape, dev, "out")
    ws = _workspace(workspace, saf3r_window_attn_workspace_bytes(L, window), dev)
    _launch(dev, stream, _hw.lib().saf3r_window_attn, _ref(L), _ref(window), qp, kp, vp, op, fp32, ws)
