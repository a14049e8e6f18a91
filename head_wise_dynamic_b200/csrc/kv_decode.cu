// Attention of a few query rows per sequence over the paged cache (single tokens and short chunks).
//
// Bound by memory: every visible key and value row is read once per kv head and 16 query rows (the
// heads of a group times the new tokens).  The keys of an item (sequence, kv head, 16 rows) are split
// into pieces for the GPU's SMs; a piece is four warps that take chunks of keys in turn, each with
// its own running maximum and sum, merged in shared memory and, over pieces, by a second small kernel.
//
// Fragments come straight from global memory, with no shared memory in between.  The matrix
// products may contract their 64 dims, and number their value columns, in any order, so the
// order is chosen for the loads: in Q K^T lane (g, t) of the m16n8k16 B fragment takes the 16 dims
// 16t.. of key g (one 16-byte load of an 8-bit row, two of a bf16 one: a warp reads whole rows), and in P V
// value column n of tile nt is dim 8n + nt, so a lane needs 8 dims in a row of each of its keys.
// An output row's lane then owns dims 16t..16t+15.
//
// 8-bit caches: codes become fp16 exactly (one conversion for two) and Q is scaled by a power of
// two per row so that it fits fp16 (its 8 significant bits do, down to 2^-24 of the row's largest); the page's key scale
// multiplies the fp32 logits.  The value scale goes into the exponent: with x = s + log2(vs), P = 2^(x - max x)
// is the weight times vs, at most 1, whatever the scales' range, and the sum takes P / vs.  bf16
// caches use bf16 products; P is rounded to bf16 there (2^-9 relative, as the tensor-core kernels do).
#include "ptx.cuh"
#include "stream.h"
#include "stream_exact.cuh"

namespace saf3r {

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;
constexpr float kLog2Scale = 0.18033688011112042f;  // log2(e) / sqrt(64)

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T>
__device__ __forceinline__ T load_stream(const void* p) {
  return __ldcs(static_cast<const T*>(p));
}

// Chunks of a whole sequence's new tokens (what its items read, at most).
__device__ __forceinline__ int seq_chunks(const WindowMask& w, const SeqInfo& s) {
  if (s.n_new <= 0) return 0;
  const Span a = span_of(w, s.len - s.n_new, s.len), z = span_of(w, s.len - 1, s.len);
  return chunks_of(runs_of(a.lo, z.hi, z.sink)).total;
}

// Chunks per piece for this call.  Run by a whole block; every block finds the same value.
__device__ __forceinline__ int chunks_per_piece(const KvAttnParams& p, int groups, int* scratch) {
  const KvView& kv = p.kv;
  int most = 0;
  long long sum = 0;
  for (int b = threadIdx.x; b < kv.n_seqs; b += blockDim.x) {
    const int c = seq_chunks(p.win, seq_info(kv, b));
    most = max(most, c);
    sum += c;
  }
  int isum = static_cast<int>(min(sum, 1LL << 24));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    isum += __shfl_xor_sync(0xffffffffu, isum, d);
  }
  if ((threadIdx.x & 31) == 0) {
    scratch[2 * (threadIdx.x >> 5)] = most;
    scratch[2 * (threadIdx.x >> 5) + 1] = isum;
  }
  __syncthreads();
  sum = 0;
  for (int w = 0; w < (blockDim.x >> 5); ++w) {
    most = max(most, scratch[2 * w]);
    sum += scratch[2 * w + 1];
  }
  sum *= kv.n_heads * groups;
  const long long target = 8LL * p.num_sms;  // pieces wanted: two rounds of four blocks per SM
  long long cps = (sum + target - 1) / target;
  cps = max(cps, static_cast<long long>((most + p.n_split - 1) / p.n_split));
  return static_cast<int>(max(cps, static_cast<long long>(kWarps)));
}

struct Stats {
  float m[kRows], l[kRows];
  int bad;  // a value that some rows must not see is not finite
  int pad[3];
};
constexpr size_t kPieceBytes = kRows * kD * sizeof(float) + sizeof(Stats);
static_assert(kPieceBytes % 16 == 0, "pieces stay aligned");

__device__ __forceinline__ uint8_t* piece_at(const KvAttnParams& p, long long item, int s) {
  return p.ws + (item * p.n_split + s) * kPieceBytes;
}

// Row r of an item: token and head.  Rows from `rows` on do not exist.
struct Item {
  int b, hk, r0, rows;
  SeqInfo s;
};
__device__ __forceinline__ Item item_of(const KvAttnParams& p, int y, int z) {
  Item it;
  it.b = z;
  it.hk = y % p.kv.n_heads;
  it.r0 = (y / p.kv.n_heads) * kRows;
  it.s = seq_info(p.kv, z);
  it.rows = min(kRows, it.s.n_new * p.group - it.r0);
  return it;
}

__device__ __forceinline__ void store_row(const KvAttnParams& p, const Item& it, int r, int col, const float* o, float inv) {
  const int i = it.r0 + r, tok = p.by_group.div(i), head = it.hk * p.group + i % p.group;
  const long long at = (it.s.row0 + tok) * p.out_ts + head * p.out_hs + col;
  if (p.out_fp32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
    d[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    d[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) =
        make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                   pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
  }
}

__device__ __forceinline__ void exact_item(const KvAttnParams& p, const Item& it, int warp, int lane) {
  for (int r = warp; r < it.rows; r += kWarps) {
    const int i = it.r0 + r, tok = p.by_group.div(i);
    exact_row(p, it.b, it.s.len, it.s.row0 + tok, it.s.len - it.s.n_new + tok, it.hk * p.group + i % p.group, lane, 0,
              kD);
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(32 * kWarps) decode_kernel(const __grid_constant__ KvAttnParams p) {
  constexpr int kT = kE4m3 ? 64 : 32;   // keys of one step of a warp: 8 KB of keys and values
  constexpr int kTiles = kT / 8;
  __shared__ float s_o[kWarps][kRows][kD + 4];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int s_scratch[2 * kWarps];
  __shared__ int s_bad;
  const KvView& kv = p.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) s_bad = 0;
  const int cps = chunks_per_piece(p, gridDim.y / kv.n_heads, s_scratch);
  const Item it = item_of(p, blockIdx.y, blockIdx.z);
  if (it.rows <= 0) return;
  const int pos0 = it.s.len - it.s.n_new;
  const int pa = pos0 + p.by_group.div(it.r0), pz = pos0 + p.by_group.div(it.r0 + it.rows - 1);
  const Span sa = span_of(p.win, pa, it.s.len), sz = span_of(p.win, pz, it.s.len);
  const Runs runs = runs_of(sa.lo, sz.hi, sz.sink);
  const Chunks ch = chunks_of(runs);
  const int c0 = blockIdx.x * cps, c1 = min(c0 + cps, ch.total);
  if (c0 >= c1) return;

  // Q fragments: rows g and g + 8, dims 16t..16t+15
  uint32_t qa[4][4];
  float qs[2] = {kLog2Scale, kLog2Scale};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    uint4 u = make_uint4(0, 0, 0, 0), w = u;
    if (r < it.rows) {
      const int a = it.r0 + r;
      const uint4* q = reinterpret_cast<const uint4*>(p.q + (it.s.row0 + p.by_group.div(a)) * p.q_ts +
                                                      (it.hk * p.group + a % p.group) * p.q_hs + 16 * t);
      u = q[0];
      w = q[1];
    }
    uint32_t v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
    if (kE4m3) {
      // the row's largest exponent; then every value times 2^-e, as fp16
      uint32_t mx = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = max(mx, max((v[j] >> 7) & 0xffu, (v[j] >> 23) & 0xffu));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = mx == 0xff ? 0 : min(max(static_cast<int>(mx) - 127, -120), 120);  // an infinity or NaN stays one
      const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      qs[i] = kLog2Scale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = pack_f16x2(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xffff0000u) * f);
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      qa[kk][i] = v[2 * kk];
      qa[kk][2 + i] = v[2 * kk + 1];
    }
  }
  // what rows g and g + 8 see
  const Span sg = span_of(p.win, pos0 + p.by_group.div(it.r0 + min(g, it.rows - 1)), it.s.len);
  const Span sh = span_of(p.win, pos0 + p.by_group.div(it.r0 + min(g + 8, it.rows - 1)), it.s.len);

  float o[8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  bool bad = false;
  const int32_t* table = kv.table + static_cast<long long>(it.b) * kv.max_pages;
  constexpr int kSteps = 64 / kT;  // steps of a chunk
  for (int st = c0 * kSteps + warp; st < c1 * kSteps; st += kWarps) {
    const int j0 = ch.key(st / kSteps) + (st % kSteps) * kT;
    // keys of this step that some row sees: [ua, ub) and below ue
    const int ue = runs.a_end, ua = runs.b_begin, ub = runs.b_end;
    if (j0 >= ub || (j0 + kT <= ua && j0 >= ue)) continue;
    const bool whole = (j0 >= sz.lo && j0 + kT <= sa.hi) || j0 + kT <= sa.sink;  // every row sees every key
    long long base[kT / 16];   // first row of each 16 keys in the pools, -1: not read
    float ks[kT / 16], lv[kT / 16], vi[kT / 16];
#pragma unroll
    for (int i = 0; i < kT / 16; ++i) {
      const int j = j0 + 16 * i;
      base[i] = -1;
      ks[i] = vi[i] = 1.f;
      lv[i] = 0.f;
      if (j < ub && (j + 16 > ua || j < ue)) {
        const int id = table[j >> kv.page_log2];
        if (id < 0 || id >= kv.n_pages) {
          atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
        } else {
          const long long at = static_cast<long long>(id) * kv.n_heads + it.hk;
          base[i] = (at << kv.page_log2) + (j & (kv.page - 1));
          if (kE4m3) {
            ks[i] = kv.k_scale[at];
            const float v = kv.v_scale[at];
            lv[i] = static_cast<float>(static_cast<int>(__float_as_uint(v) >> 23) - 127);
            vi[i] = __uint_as_float((254u << 23) - (__float_as_uint(v) & 0x7f800000u));
          }
        }
      }
    }
    auto in = [&](int j) { return j < ub && (j >= ua || j < ue); };
    // loads: keys, then values
    uint4 k[kTiles][kE4m3 ? 1 : 2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int off = 8 * (n & 1) + g;
#pragma unroll
      for (int c = 0; c < (kE4m3 ? 1 : 2); ++c) {
        k[n][c] = make_uint4(0, 0, 0, 0);
        if (base[n / 2] >= 0 && in(j0 + 16 * (n / 2) + off))
          k[n][c] = load_stream<uint4>(kv.k + ((base[n / 2] + off) * kD + 16 * t + 8 * c) * (kE4m3 ? 1 : 2));
      }
    }
    uint32_t v[kT / 16][4][kE4m3 ? 2 : 4];
#pragma unroll
    for (int i = 0; i < kT / 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int off = 2 * t + (c & 1) + 8 * (c >> 1);
        const bool have = base[i] >= 0 && in(j0 + 16 * i + off);
        const uint8_t* src = kv.v + ((base[i] + off) * kD + 8 * g) * (kE4m3 ? 1 : 2);
        if (kE4m3) {
          const uint2 x = have ? load_stream<uint2>(src) : make_uint2(0, 0);
          v[i][c][0] = x.x;
          v[i][c][1] = x.y;
        } else {
          const uint4 x = have ? load_stream<uint4>(src) : make_uint4(0, 0, 0, 0);
          v[i][c][0] = x.x;
          v[i][c][1] = x.y;
          v[i][c][kE4m3 ? 0 : 2] = x.z;
          v[i][c][kE4m3 ? 1 : 3] = x.w;
        }
      }
    // logits, in units of log2, times nothing yet but the scales
    float s[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      if (kE4m3) {
        const uint32_t w[4] = {k[n][0].x, k[n][0].y, k[n][0].z, k[n][0].w};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_f16(s[n], qa[kk], f16_of_e4m3(w[kk]), f16_of_e4m3(w[kk] >> 16));
      } else {
        const uint4 x = k[n][0], y = k[n][kE4m3 ? 0 : 1];
        mma_bf16(s[n], qa[0], x.x, x.y);
        mma_bf16(s[n], qa[1], x.z, x.w);
        mma_bf16(s[n], qa[2], y.x, y.y);
        mma_bf16(s[n], qa[3], y.z, y.w);
      }
      const float f0 = qs[0] * ks[n / 2], f1 = qs[1] * ks[n / 2];
      s[n][0] = s[n][0] * f0 + lv[n / 2];
      s[n][1] = s[n][1] * f0 + lv[n / 2];
      s[n][2] = s[n][2] * f1 + lv[n / 2];
      s[n][3] = s[n][3] * f1 + lv[n / 2];
    }
    if (!whole) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int j = j0 + 8 * n + 2 * t + c;
          const bool have = base[n / 2] >= 0;
          if (!(have && ((j >= sg.lo && j < sg.hi) || j < sg.sink))) s[n][c] = -INFINITY;
          if (!(have && ((j >= sh.lo && j < sh.hi) || j < sh.sink))) s[n][2 + c] = -INFINITY;
        }
      if (kv.max_new > 1) {
#pragma unroll
        for (int i = 0; i < kT / 16; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int w = 0; w < (kE4m3 ? 2 : 4); ++w) {
              const uint32_t x = v[i][c][w];
              if (kE4m3)
                bad |= (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;  // a code of 0x7f
              else
                bad |= (((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0;  // an exponent of ones
            }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[i], mx);
      const float use = mn == -INFINITY ? 0.f : mn;
      const float f = fast_exp2(m[i] - use);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const float a = fast_exp2(s[n][2 * i] - use), b = fast_exp2(s[n][2 * i + 1] - use);
        sum += (a + b) * vi[n / 2];
        s[n][2 * i] = a;
        s[n][2 * i + 1] = b;
      }
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        o[n][2 * i] *= f;
        o[n][2 * i + 1] *= f;
      }
    }
#pragma unroll
    for (int i = 0; i < kT / 16; ++i) {
      uint32_t pa4[4];
      if (kE4m3) {
        pa4[0] = pack_f16x2(s[2 * i][0], s[2 * i][1]);
        pa4[1] = pack_f16x2(s[2 * i][2], s[2 * i][3]);
        pa4[2] = pack_f16x2(s[2 * i + 1][0], s[2 * i + 1][1]);
        pa4[3] = pack_f16x2(s[2 * i + 1][2], s[2 * i + 1][3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = __byte_perm(v[i][0][h], v[i][1][h], 0x5140), b = __byte_perm(v[i][0][h], v[i][1][h], 0x7362);
          const uint32_t c = __byte_perm(v[i][2][h], v[i][3][h], 0x5140), d = __byte_perm(v[i][2][h], v[i][3][h], 0x7362);
          mma_f16(o[4 * h], pa4, f16_of_e4m3(a), f16_of_e4m3(c));
          mma_f16(o[4 * h + 1], pa4, f16_of_e4m3(a >> 16), f16_of_e4m3(c >> 16));
          mma_f16(o[4 * h + 2], pa4, f16_of_e4m3(b), f16_of_e4m3(d));
          mma_f16(o[4 * h + 3], pa4, f16_of_e4m3(b >> 16), f16_of_e4m3(d >> 16));
        }
      } else {
        pa4[0] = pack_bf16x2(s[2 * i][0], s[2 * i][1]);
        pa4[1] = pack_bf16x2(s[2 * i][2], s[2 * i][3]);
        pa4[2] = pack_bf16x2(s[2 * i + 1][0], s[2 * i + 1][1]);
        pa4[3] = pack_bf16x2(s[2 * i + 1][2], s[2 * i + 1][3]);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int w = kE4m3 ? 0 : h;
          mma_bf16(o[2 * h], pa4, __byte_perm(v[i][0][w], v[i][1][w], 0x5410), __byte_perm(v[i][2][w], v[i][3][w], 0x5410));
          mma_bf16(o[2 * h + 1], pa4, __byte_perm(v[i][0][w], v[i][1][w], 0x7632), __byte_perm(v[i][2][w], v[i][3][w], 0x7632));
        }
      }
    }
  }
  // merge the warps: the lane's columns of rows g and g + 8 are dims 16t + nt and 16t + 8 + nt
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    const int r = g + 8 * i;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      s_o[warp][r][16 * t + n] = o[n][2 * i];
      s_o[warp][r][16 * t + 8 + n] = o[n][2 * i + 1];
    }
    if (t == 0) {
      s_m[warp][r] = m[i];
      s_l[warp][r] = l[i];
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  const bool only = ch.total <= cps;  // the item has this piece alone
  if (only && s_bad) {
    exact_item(p, it, warp, lane);
    return;
  }
  const int r = threadIdx.x >> 3, col = (threadIdx.x & 7) * 8;
  float mm = -INFINITY, ll = 0.f, acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][r]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = fast_exp2(s_m[w][r] - (mm == -INFINITY ? 0.f : mm));
    ll += s_l[w][r] * f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += s_o[w][r][col + i] * f;
  }
  if (only) {
    if (r < it.rows) store_row(p, it, r, col, acc, ll == 0.f ? 0.f : 1.f / ll);
    return;
  }
  uint8_t* piece = piece_at(p, static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y, blockIdx.x);
  float4* po = reinterpret_cast<float4*>(reinterpret_cast<float*>(piece) + r * kD + col);
  po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  po[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  Stats* ps = reinterpret_cast<Stats*>(piece + kRows * kD * sizeof(float));
  if (col == 0) {
    ps->m[r] = mm;
    ps->l[r] = ll;
  }
  if (threadIdx.x == 0) ps->bad = s_bad;
}

// Joins the pieces of one item, in their order.
__global__ void __launch_bounds__(32 * kWarps) decode_join_kernel(const __grid_constant__ KvAttnParams p) {
  __shared__ int s_scratch[2 * kWarps];
  const KvView& kv = p.kv;
  const int cps = chunks_per_piece(p, gridDim.x / kv.n_heads, s_scratch);
  const Item it = item_of(p, blockIdx.x, blockIdx.y);
  if (it.rows <= 0) return;
  const int pos0 = it.s.len - it.s.n_new;
  const Span sa = span_of(p.win, pos0 + p.by_group.div(it.r0), it.s.len);
  const Span sz = span_of(p.win, pos0 + p.by_group.div(it.r0 + it.rows - 1), it.s.len);
  const Chunks ch = chunks_of(runs_of(sa.lo, sz.hi, sz.sink));
  if (ch.total <= cps) return;
  const int n = (ch.total + cps - 1) / cps;
  const uint8_t* base = piece_at(p, static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x, 0);
  auto stats = [&](int s) { return reinterpret_cast<const Stats*>(base + s * kPieceBytes + kRows * kD * sizeof(float)); };
  const int r = threadIdx.x >> 3, col = (threadIdx.x & 7) * 8;
  float mm = -INFINITY;
  bool bad = false;
  for (int s = 0; s < n; ++s) {
    mm = fmaxf(mm, stats(s)->m[r]);
    bad |= stats(s)->bad != 0;
  }
  if (bad) {
    exact_item(p, it, threadIdx.x >> 5, threadIdx.x & 31);
    return;
  }
  if (r >= it.rows) return;
  float ll = 0.f, acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int s = 0; s < n; ++s) {
    const float f = fast_exp2(stats(s)->m[r] - (mm == -INFINITY ? 0.f : mm));
    ll += stats(s)->l[r] * f;
    const float4* po = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base + s * kPieceBytes) + r * kD + col);
    const float4 a = po[0], b = po[1];
    acc[0] += a.x * f; acc[1] += a.y * f; acc[2] += a.z * f; acc[3] += a.w * f;
    acc[4] += b.x * f; acc[5] += b.y * f; acc[6] += b.z * f; acc[7] += b.w * f;
  }
  store_row(p, it, r, col, acc, ll == 0.f ? 0.f : 1.f / ll);
}

int row_groups(int max_new, int group) { return (max_new * group + kRows - 1) / kRows; }

// Most pieces of one item: its keys by at least 256, and not so many that idle blocks cost time.
int split_limit(const KvView& kv, const WindowMask& w, int groups) {
  long long keys = static_cast<long long>(kv.max_pages) << kv.page_log2;
  if (w.window > 0) {
    const long long views = (static_cast<long long>(kv.max_new) + w.view - 2) / w.view + 1;  // of the new tokens
    const long long seen = (views + (w.causal ? 1LL : 2LL) * w.window) * w.view + w.sink + 128;
    keys = keys < seen ? keys : seen;
  }
  const long long items = static_cast<long long>(kv.n_seqs) * kv.n_heads * groups;
  long long n = (keys + 255) / 256;
  const long long cap = items > 0 ? (16384 + items - 1) / items : 1;
  n = n < cap ? n : cap;
  n = n < 512 ? n : 512;
  return n < 1 ? 1 : static_cast<int>(n);
}

}  // namespace

bool decode_takes(int max_new, int group) { return static_cast<long long>(max_new) * group <= 64; }

size_t decode_workspace_bytes(const KvView& kv, const WindowMask& w, int group) {
  const int groups = row_groups(kv.max_new, group);
  return static_cast<size_t>(kv.n_seqs) * kv.n_heads * groups * split_limit(kv, w, groups) * kPieceBytes;
}

cudaError_t launch_decode(const KvAttnParams& p0, cudaStream_t stream, int* n_launch) {
  KvAttnParams p = p0;
  const int groups = row_groups(p.kv.max_new, p.group);
  p.n_split = split_limit(p.kv, p.win, groups);
  const dim3 grid(p.n_split, p.kv.n_heads * groups, p.kv.n_seqs);
  if (p.e4m3)
    decode_kernel<true><<<grid, 32 * kWarps, 0, stream>>>(p);
  else
    decode_kernel<false><<<grid, 32 * kWarps, 0, stream>>>(p);
  ++*n_launch;
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.n_split == 1) return e;
  decode_join_kernel<<<dim3(grid.y, grid.z), 32 * kWarps, 0, stream>>>(p);
  ++*n_launch;
  return cudaGetLastError();
}

}  // namespace saf3r
