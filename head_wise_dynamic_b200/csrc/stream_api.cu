// C ABI of the streaming operators: argument checks, views of the caller's buffers, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "stream.h"

using namespace saf3r;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Row strides of a tensor that is read (broadcast dims allowed) or written (rows must not overlap).
bool strides_ok(long long tokens, long long ts, long long heads, long long hs, bool fp32, bool written) {
  const long long unit = fp32 ? 4 : 8, top = 1LL << 36;
  if (ts < 0 || hs < 0 || ts % unit || hs % unit || ts > top || hs > top) return false;
  if (!written) return true;
  if ((tokens > 1 && ts < kD) || (heads > 1 && hs < kD)) return false;
  if (tokens > 1 && heads > 1) {
    // rows apart: one dim lies inside the other's step
    const bool token_major = ts >= (heads - 1) * hs + kD, head_major = hs >= static_cast<__int128>(tokens - 1) * ts + kD;
    if (!token_major && !head_major) return false;
  }
  return true;
}

bool apart(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + na <= y || y + nb <= x;
}

// The rows of a tensor, in bytes.
struct Rows {
  long long base, tokens, ts, heads, hs, row;
  Rows(const void* p, long long tokens_, long long ts_, long long heads_, long long hs_, bool fp32)
      : base(static_cast<long long>(reinterpret_cast<uintptr_t>(p))),
        tokens(ts_ ? tokens_ : 1), ts(ts_ * (fp32 ? 4 : 2)), heads(hs_ ? heads_ : 1), hs(hs_ * (fp32 ? 4 : 2)), row(kD * (fp32 ? 4 : 2)) {}
  __int128 end() const { return static_cast<__int128>(tokens - 1) * ts + static_cast<__int128>(heads - 1) * hs + base + row; }
};

// Whether a row at distance d + i * step from another one, for some i in lo..hi, shares a byte with it.
bool row_meets(__int128 d, long long step, long long lo, long long hi, long long row, long long other) {
  if (lo == hi) return d + static_cast<__int128>(lo) * step < other && d + static_cast<__int128>(lo) * step > -row;
  const __int128 n = other - 1 - d;
  __int128 i = n / step - (n % step < 0 ? 1 : 0);  // the last that begins before the other's end
  if (i > hi) i = hi;
  return i >= lo && d + i * step > -row;
}

// Whether a row of a and one of b share a byte.  Ranges that lie apart do not; rows of one packed buffer may interleave.  Where
// the ranges interleave with unequal token strides, or with more than 2^16 pairs of heads of unequal strides, the answer is yes.
bool rows_meet(Rows a, Rows b) {
  if (a.end() <= b.base || b.end() <= a.base) return false;
  if (a.tokens == 1) a.ts = b.ts;
  if (b.tokens == 1) b.ts = a.ts;
  if (a.heads == 1) a.hs = b.hs;
  if (b.heads == 1) b.hs = a.hs;
  if (a.ts != b.ts) return true;
  const __int128 d = static_cast<__int128>(a.base) - b.base;
  if (a.hs == b.hs) {
    for (long long i = 1 - b.heads; i < a.heads; ++i)
      if (row_meets(d + static_cast<__int128>(i) * a.hs, a.ts, 1 - b.tokens, a.tokens - 1, a.row, b.row)) return true;
    return false;
  }
  if (a.heads * b.heads > 65536) return true;
  for (long long i = 0; i < a.heads; ++i)
    for (long long j = 0; j < b.heads; ++j)
      if (row_meets(d + static_cast<__int128>(i) * a.hs - static_cast<__int128>(j) * b.hs, a.ts, 1 - b.tokens, a.tokens - 1, a.row, b.row))
        return true;
  return false;
}

saf3r_status check_cache(const saf3r_kv_cache* c, bool pointers) {
  if (!c) return SAF3R_ERR_INVALID;
  if (c->n_pages < 1 || c->n_heads < 1 || c->n_heads > kMaxHeads) return SAF3R_ERR_INVALID;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return SAF3R_ERR_INVALID;
  if (c->type != SAF3R_KV_BF16 && c->type != SAF3R_KV_E4M3) return SAF3R_ERR_INVALID;
  // rows of a pool are counted in 31 bits
  if (static_cast<long long>(c->n_pages) * c->n_heads * c->page >= (1LL << 31)) return SAF3R_ERR_UNSUPPORTED;
  if (!pointers) return SAF3R_OK;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return SAF3R_ERR_INVALID;
  if (c->type == SAF3R_KV_E4M3 &&
      (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
    return SAF3R_ERR_INVALID;
  return SAF3R_OK;
}

// Whether the range of the rows runs into the cache's.
bool meets_pools(const saf3r_kv_cache* c, const Rows& r) {
  const long long pages = static_cast<long long>(c->n_pages) * c->n_heads, pool = pages * c->page * kD * (c->type == SAF3R_KV_E4M3 ? 1 : 2);
  auto meets = [&](const void* p, long long bytes) {
    const long long at = static_cast<long long>(reinterpret_cast<uintptr_t>(p));
    return r.base < at + bytes && r.end() > at;
  };
  return meets(c->k, pool) || meets(c->v, pool) ||
         (c->type == SAF3R_KV_E4M3 && (meets(c->k_scale, 4 * pages) || meets(c->v_scale, 4 * pages)));
}

saf3r_status check_batch(const saf3r_kv_cache* c, const saf3r_kv_batch* b, bool pointers) {
  if (!b || b->n_seqs < 0 || b->n_seqs > 65535 || b->n_tokens < 0 || b->max_new < 0 || b->max_new > b->n_tokens ||
      b->max_pages < 0)
    return SAF3R_ERR_INVALID;
  // positions are counted in 31 bits, with room for one tile behind the last
  if (static_cast<long long>(b->max_pages) * c->page > (1LL << 31) - 1024) return SAF3R_ERR_UNSUPPORTED;
  if (pointers && b->n_seqs > 0 &&
      (!b->cu_tokens || !b->kv_lens || (b->max_pages > 0 && !b->page_table) ||
       (reinterpret_cast<uintptr_t>(b->cu_tokens) & 3) || (reinterpret_cast<uintptr_t>(b->kv_lens) & 3) ||
       (reinterpret_cast<uintptr_t>(b->page_table) & 3)))
    return SAF3R_ERR_INVALID;
  return SAF3R_OK;
}

bool window_ok(const saf3r_window* w) { return w && w->view_tokens >= 1 && w->window >= 0 && w->n_sink >= 0; }

KvView view_of(const saf3r_kv_cache* c, const saf3r_kv_batch* b, int* err) {
  KvView v;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.cu = b->cu_tokens;
  v.kv_lens = b->kv_lens;
  v.table = b->page_table;
  v.err = err;
  v.n_pages = c->n_pages;
  v.n_heads = c->n_heads;
  v.page = c->page;
  v.page_log2 = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  v.n_seqs = b->n_seqs;
  v.n_tokens = b->n_tokens;
  v.max_new = b->max_new;
  v.max_pages = b->max_pages;
  return v;
}

WindowMask mask_of(const saf3r_window* w) { return WindowMask{w->view_tokens, w->window, w->n_sink, w->causal != 0, make_div(w->view_tokens)}; }

saf3r_status device(int* sms, int** err) {
  int major = 0;
  if (!call_device(sms, &major, err)) return SAF3R_ERR_CUDA;
  return major == 10 ? SAF3R_OK : SAF3R_ERR_UNSUPPORTED;
}

saf3r_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SAF3R_OK : SAF3R_ERR_CUDA; }

}  // namespace

extern "C" {

saf3r_status saf3r_rope(const saf3r_rope_cfg* rope, const saf3r_rope_args* a, void* stream) {
  set_launch_count(0);
  RopeParams p;
  if (!build_rope_table(rope, &p.table) || !a) return SAF3R_ERR_INVALID;
  if (a->n_tokens < 0 || a->n_tokens >= (1LL << 31) || a->n_heads < 0 || a->n_heads > 65535 || a->n_rot_heads < 0 ||
      a->n_rot_heads > a->n_heads)
    return SAF3R_ERR_INVALID;
  if (a->n_tokens == 0 || a->n_heads == 0) return SAF3R_OK;
  if (!a->x || !a->out || !aligned16(a->x) || !aligned16(a->out)) return SAF3R_ERR_INVALID;
  if (a->n_rot_heads > 0 && (!a->pos || (reinterpret_cast<uintptr_t>(a->pos) & 3))) return SAF3R_ERR_INVALID;
  if (!strides_ok(a->n_tokens, a->x_token_stride, a->n_heads, a->x_head_stride, a->x_is_fp32 != 0, false) ||
      !strides_ok(a->n_tokens, a->out_token_stride, a->n_heads, a->out_head_stride, a->out_is_fp32 != 0, true))
    return SAF3R_ERR_INVALID;
  const bool in_place = a->x == a->out && (a->x_is_fp32 != 0) == (a->out_is_fp32 != 0) &&
                        a->x_token_stride == a->out_token_stride && a->x_head_stride == a->out_head_stride;
  if (!in_place && rows_meet(Rows(a->x, a->n_tokens, a->x_token_stride, a->n_heads, a->x_head_stride, a->x_is_fp32 != 0),
                             Rows(a->out, a->n_tokens, a->out_token_stride, a->n_heads, a->out_head_stride, a->out_is_fp32 != 0)))
    return SAF3R_ERR_INVALID;
  int sms = 0, *err = nullptr;
  const saf3r_status st = device(&sms, &err);
  if (st != SAF3R_OK) return st;
  p.x = a->x;
  p.out = a->out;
  p.pos = a->pos;
  p.n_tokens = a->n_tokens;
  p.x_ts = a->x_token_stride;
  p.x_hs = a->x_head_stride;
  p.out_ts = a->out_token_stride;
  p.out_hs = a->out_head_stride;
  p.n_heads = a->n_heads;
  p.n_rot = a->n_rot_heads;
  p.inverse = a->inverse != 0;
  p.heads_per_block = 0;
  int launches = 0;
  const cudaError_t e =
      launch_rope(p, a->x_is_fp32 != 0, a->out_is_fp32 != 0, sms, static_cast<cudaStream_t>(stream), &launches);
  set_launch_count(launches);
  return cuda_status(e);
}

saf3r_status saf3r_kv_append(const saf3r_kv_cache* cache, const saf3r_kv_batch* batch, const saf3r_rope_cfg* rope,
                             const saf3r_kv_rows* rows, void* stream) {
  set_launch_count(0);
  saf3r_status st = check_cache(cache, true);
  if (st != SAF3R_OK) return st;
  if ((st = check_batch(cache, batch, true)) != SAF3R_OK) return st;
  AppendParams p;
  std::memset(&p.rope, 0, sizeof(p.rope));
  if (rope && !build_rope_table(rope, &p.rope)) return SAF3R_ERR_INVALID;
  if (!rows) return SAF3R_ERR_INVALID;
  if (batch->n_seqs == 0 || batch->n_tokens == 0 || batch->max_new == 0) return SAF3R_OK;
  if (!rows->k || !rows->v || !aligned16(rows->k) || !aligned16(rows->v)) return SAF3R_ERR_INVALID;
  if (rope && (!rows->pos || (reinterpret_cast<uintptr_t>(rows->pos) & 3))) return SAF3R_ERR_INVALID;
  if (!strides_ok(batch->n_tokens, rows->k_token_stride, cache->n_heads, rows->k_head_stride, false, false) ||
      !strides_ok(batch->n_tokens, rows->v_token_stride, cache->n_heads, rows->v_head_stride, false, false))
    return SAF3R_ERR_INVALID;
  if (meets_pools(cache, Rows(rows->k, batch->n_tokens, rows->k_token_stride, cache->n_heads, rows->k_head_stride, false)) ||
      meets_pools(cache, Rows(rows->v, batch->n_tokens, rows->v_token_stride, cache->n_heads, rows->v_head_stride, false)))
    return SAF3R_ERR_INVALID;
  int sms = 0, *err = nullptr;
  if ((st = device(&sms, &err)) != SAF3R_OK) return st;
  p.kv = view_of(cache, batch, err);
  p.has_rope = rope != nullptr;
  p.heads_per_block = 0;
  p.k_rows = static_cast<const uint16_t*>(rows->k);
  p.v_rows = static_cast<const uint16_t*>(rows->v);
  p.k_ts = rows->k_token_stride;
  p.k_hs = rows->k_head_stride;
  p.v_ts = rows->v_token_stride;
  p.v_hs = rows->v_head_stride;
  p.pos = rows->pos;
  int launches = 0;
  const cudaError_t e =
      launch_append(p, cache->type == SAF3R_KV_E4M3, sms, static_cast<cudaStream_t>(stream), &launches);
  set_launch_count(launches);
  return cuda_status(e);
}

size_t saf3r_kv_attn_workspace_bytes(const saf3r_kv_cache* cache, const saf3r_kv_batch* batch,
                                     const saf3r_window* window, int n_heads) {
  if (check_cache(cache, false) != SAF3R_OK || check_batch(cache, batch, false) != SAF3R_OK || !window_ok(window) ||
      n_heads < 1 || n_heads > kMaxHeads || n_heads % cache->n_heads)
    return 0;
  const KvView kv = view_of(cache, batch, nullptr);
  const int group = n_heads / cache->n_heads;
  const size_t n = decode_takes(batch->max_new, group)
                       ? decode_workspace_bytes(kv, group)
                       : attn_workspace_bytes();
  return n < 256 ? 256 : n;
}

saf3r_status saf3r_kv_attn(const saf3r_kv_cache* cache, const saf3r_kv_batch* batch, const saf3r_window* window,
                           const saf3r_query_rows* rows, void* workspace, void* stream) {
  set_launch_count(0);
  saf3r_status st = check_cache(cache, true);
  if (st != SAF3R_OK) return st;
  if ((st = check_batch(cache, batch, true)) != SAF3R_OK) return st;
  if (!window_ok(window) || !rows || rows->n_heads < 1 || rows->n_heads > kMaxHeads || rows->n_heads % cache->n_heads)
    return SAF3R_ERR_INVALID;
  if (batch->n_seqs == 0 || batch->n_tokens == 0 || batch->max_new == 0) return SAF3R_OK;
  if (!rows->q || !rows->out || !workspace || !aligned16(rows->q) || !aligned16(rows->out) || !aligned16(workspace))
    return SAF3R_ERR_INVALID;
  if (!strides_ok(batch->n_tokens, rows->q_token_stride, rows->n_heads, rows->q_head_stride, false, true) ||
      !strides_ok(batch->n_tokens, rows->out_token_stride, rows->n_heads, rows->out_head_stride, rows->out_is_fp32 != 0,
                  true))
    return SAF3R_ERR_INVALID;
  // a row may be computed again, from the queries and the cache, after others were written
  const Rows q(rows->q, batch->n_tokens, rows->q_token_stride, rows->n_heads, rows->q_head_stride, false);
  const Rows out(rows->out, batch->n_tokens, rows->out_token_stride, rows->n_heads, rows->out_head_stride, rows->out_is_fp32 != 0);
  if (rows_meet(q, out) || meets_pools(cache, out)) return SAF3R_ERR_INVALID;
  int sms = 0, *err = nullptr;
  if ((st = device(&sms, &err)) != SAF3R_OK) return st;
  KvAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.kv = view_of(cache, batch, err);
  p.win = mask_of(window);
  p.q = static_cast<const uint16_t*>(rows->q);
  p.out = rows->out;
  p.q_ts = rows->q_token_stride;
  p.q_hs = rows->q_head_stride;
  p.out_ts = rows->out_token_stride;
  p.out_hs = rows->out_head_stride;
  p.n_heads = rows->n_heads;
  p.group = rows->n_heads / cache->n_heads;
  p.by_group = make_div(p.group);
  p.out_fp32 = rows->out_is_fp32 != 0;
  p.e4m3 = cache->type == SAF3R_KV_E4M3;
  p.ws = static_cast<uint8_t*>(workspace);
  p.num_sms = sms;
  p.wait_budget = call_wait_budget();
  int launches = 0;
  if (decode_takes(batch->max_new, p.group))
    st = launch_decode(p, static_cast<cudaStream_t>(stream), &launches);
  else {
    p.withhold = take_withhold_arrive();
    st = launch_attn(p, static_cast<cudaStream_t>(stream), &launches);
  }
  set_launch_count(launches);
  return st;
}

size_t saf3r_window_attn_workspace_bytes(const saf3r_layout* layout, const saf3r_window* window) {
  if (validate_layout(layout) != SAF3R_OK || !window_ok(window)) return 0;
  return attn_workspace_bytes();
}

saf3r_status saf3r_window_attn(const saf3r_layout* layout, const saf3r_window* window, const void* q, const void* k,
                               const void* v, void* out, int out_is_fp32, void* workspace, void* stream) {
  set_launch_count(0);
  saf3r_status st = validate_layout(layout);
  if (st != SAF3R_OK) return st;
  if (!window_ok(window) || !q || !k || !v || !out || !workspace || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(out) || !aligned16(workspace))
    return SAF3R_ERR_INVALID;
  const Dims d = make_dims(*layout);
  const size_t n = static_cast<size_t>(d.H) * d.N * kD, out_bytes = n * (out_is_fp32 ? 4 : 2);
  if (!apart(out, out_bytes, q, 2 * n) || !apart(out, out_bytes, k, 2 * n) || !apart(out, out_bytes, v, 2 * n))
    return SAF3R_ERR_INVALID;
  int sms = 0, *err = nullptr;
  if ((st = device(&sms, &err)) != SAF3R_OK) return st;
  KvAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.kv.err = err;
  p.kv.n_heads = d.H;
  p.kv.n_seqs = 1;
  p.kv.n_tokens = p.kv.max_new = d.N;
  p.win = mask_of(window);
  p.ck = static_cast<const uint16_t*>(k);
  p.cv = static_cast<const uint16_t*>(v);
  p.q = static_cast<const uint16_t*>(q);
  p.out = out;
  p.q_ts = p.out_ts = kD;
  p.q_hs = p.out_hs = static_cast<long long>(d.N) * kD;
  p.n_heads = d.H;
  p.group = 1;
  p.by_group = make_div(1);
  p.out_fp32 = out_is_fp32 != 0;
  p.ws = static_cast<uint8_t*>(workspace);
  p.num_sms = sms;
  p.wait_budget = call_wait_budget();
  p.withhold = take_withhold_arrive();
  int launches = 0;
  st = launch_attn(p, static_cast<cudaStream_t>(stream), &launches);
  set_launch_count(launches);
  return st;
}

}  // extern "C"
