// Appends a step's keys and values to the paged cache, the keys rotated on the way.
//
// A block owns one page of one sequence that takes new rows, for some of the kv heads: 8 warps in
// teams of page / 16, each team one head's keys or values, a warp 16 rows of the page.  A team
// holds its rows in registers between the largest magnitude (8-bit caches: it fixes the
// page's scale) and the store, so every row is read once, and has the next task's rows on their way meanwhile.  Sines and
// cosines are computed once per block and row and shared by its heads.  Because one block owns a (page, head), growing a scale
// and re-rounding the older rows needs no atomics.
//
// Scales are powers of two: x / scale is exact, and re-rounding older codes when a scale grows is too
// unless they become subnormal.
//
// Measured: 16 views of bf16 (1,374 tokens, 16 heads, pages of 16) 39 us, 70% of the measured copy rate: 4 loads that wait
// for one another before a block's first row is stored, three waves of blocks.  Fewer heads a block cost more
// (8: 44 us, 4: 60 us), as does putting the rows together in shared memory first (45 us).  One 8-bit view 16 us: instructions (37%
// of the issue slots, 6 us of pure issue: values turned twice, codes made four times over to find those next to a border) and
// the same chain.  64 single tokens 4.3 us of GPU time (a call takes 7.6 us of the host): latency.
#include "rope.cuh"
#include "stream.h"

namespace saf3r {

namespace {

constexpr int kWarps = 8;

// The new rows of one page.
struct Chunk {
  int page;    // page id, -1: nothing to do
  int row0;    // first new row inside the page
  int n;       // new rows
  int token;   // their first row in the step's tensors
};

// Block x's page: pages that take new rows are numbered sequence after sequence.  Run by one warp.
__device__ __forceinline__ Chunk find_chunk(const KvView& kv, int x, int lane) {
  int b = -1, idx = 0;  // sequence, page of its new rows
  SeqInfo s{0, 0, 0, false};
  int before = 0;
  for (int b0 = 0; b0 < kv.n_seqs && b < 0; b0 += 32) {
    SeqInfo mine{0, 0, 0, false};
    if (b0 + lane < kv.n_seqs) mine = seq_info(kv, b0 + lane);
    int cnt = 0;
    if (mine.n_new > 0)
      cnt = ((mine.len - 1) >> kv.page_log2) - ((mine.len - mine.n_new) >> kv.page_log2) + 1;
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, cnt > 0 && x >= before + incl - cnt && x < before + incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = b0 + src;
      idx = x - before - __shfl_sync(0xffffffffu, incl - cnt, src);
      s.row0 = __shfl_sync(0xffffffffu, mine.row0, src);
      s.n_new = __shfl_sync(0xffffffffu, mine.n_new, src);
      s.len = __shfl_sync(0xffffffffu, mine.len, src);
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  Chunk c{-1, 0, 0, 0};
  if (b < 0 || s.n_new <= 0) return c;
  const int start = s.len - s.n_new;
  const int pi = (start >> kv.page_log2) + idx;
  const int p0 = max(start, pi << kv.page_log2);
  const int p1 = static_cast<int>(min(static_cast<long long>(s.len), (static_cast<long long>(pi) + 1) << kv.page_log2));
  c.page = kv.table[static_cast<long long>(b) * kv.max_pages + pi];
  if (c.page < 0 || c.page >= kv.n_pages) {
    atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
    c.page = -1;
  }
  c.row0 = p0 - (pi << kv.page_log2);
  c.n = p1 - p0;
  c.token = s.row0 + (p0 - start);
  return c;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
// four codes times a power of two, rounded again
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float f) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = f32x2_of_f16x2(f16x2_of_e4m3(codes >> (16 * i)));
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
  return e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}

constexpr float kFltMax = 3.402823466e+38f;
constexpr int kMinExp = -100, kMaxExp = 119;

// Exponent of the scale that magnitude m needs: ceil(log2(m / 448)), 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float m) {
  const uint32_t b = __float_as_uint(m);
  if (b < 0x00800000u) return kMinExp;
  const int e = static_cast<int>(b >> 23) - 127;
  return min(max(e - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0), kMinExp), kMaxExp);
}

// The same in 64 bits (of a magnitude in fp32's range).
__device__ __forceinline__ int scale_exp(double m) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(m));
  const int e = static_cast<int>(b >> 52) - 1023;
  return min(max(e - 8 + ((b & 0xfffffffffffffull) > 0xc000000000000ull ? 1 : 0), kMinExp), kMaxExp);
}

// Old codes of a page's first `rows` rows, rounded again to a larger scale (f = old scale / new one); `threads` threads.
__device__ __forceinline__ void rescale_rows(uint8_t* rows_at, int rows, float f, int thread, int threads) {
  uint4* old = reinterpret_cast<uint4*>(rows_at);
  const int n = rows * 4;
  for (int i0 = thread; i0 < n; i0 += 4 * threads) {  // four loads at a time
    uint4 v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (i0 + c * threads < n) v[c] = old[i0 + c * threads];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (i0 + c * threads < n)
        old[i0 + c * threads] = make_uint4(rescale4(v[c].x, f), rescale4(v[c].y, f), rescale4(v[c].z, f), rescale4(v[c].w, f));
  }
}

__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fabsf(x[i]) <= kFltMax ? x[i] * inv : __uint_as_float(0x7fffffffu);
  return e4m3x4(y[0], y[1], y[2], y[3]);
}
// a segment's codes at p (its 4 or 8 bytes)
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[N], float inv) {
  if constexpr (N == 4)
    *reinterpret_cast<uint32_t*>(p) = codes4(x, inv);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(codes4(x, inv), codes4(x + 4, inv));
}
template <int N>
__device__ __forceinline__ float largest(const float (&x)[N], float m) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float a = fabsf(x[i]);
    m = fmaxf(m, a <= kFltMax ? a : 0.f);  // infinities and NaN do not count
  }
  return m;
}
template <int N>
__device__ __forceinline__ void store_rows(uint16_t* row, int o1, int o2, const float (&a)[N], const float (&b)[N]) {
  Segment<uint16_t, N> u, w;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    u.set2(i, a[i], a[i + 1]);
    w.set2(i, b[i], b[i + 1]);
  }
  u.store(row + o1);
  w.store(row + o2);
}

// Codes of a turned key's segments.  The fp32 rotation is off by less than 2^-21 of |a| + |b| for a pair (a, b): where that
// could carry a value over a border between two codes, the thread's pairs are turned again in 64 bits.  One in a hundred
// warps meets such a value; all in 64 bits, a view of 1,374 tokens and 16 heads took 18 us instead of 12.
template <int N>
__device__ __forceinline__ void store_turned(uint8_t* row, int o1, int o2, float (&a)[N], float (&b)[N], float inv, const RopeTable& tb,
                                             const int32_t* pos, int pair0, const Segment<uint16_t, N>& u,
                                             const Segment<uint16_t, N>& w) {
  bool border = false;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float lo[4], hi[4], lo2[4], hi2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float ea = (fabsf(a[i + j]) + fabsf(tb.interleaved ? a[(i + j) ^ 1] : b[i + j])) * 4.76837158203125e-07f;
      const float eb = tb.interleaved ? (fabsf(b[i + j]) + fabsf(b[(i + j) ^ 1])) * 4.76837158203125e-07f : ea;
      lo[j] = a[i + j] - ea;
      hi[j] = a[i + j] + ea;
      lo2[j] = b[i + j] - eb;
      hi2[j] = b[i + j] + eb;
    }
    border |= codes4(lo, inv) != codes4(hi, inv) || codes4(lo2, inv) != codes4(hi2, inv);
  }
  if (border) {
    spread(u, w, a, b);
    double s[N], c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) rope_sincos(tb, pair0 + i, pos[tb.axis[(pair0 + i) >> 2]], s[i], c[i]);
    turn(a, b, s, c, tb.interleaved);
  }
  store_codes(row + o1, a, inv);
  store_codes(row + o2, b, inv);
}

// Exponent of the scale that turned values of largest magnitude m need.  In fp32 they are off by 2^-21 of |a| + |b|, which is at
// most twice the larger turned value: where 2^-19 of m could change the exponent, they are turned again in 64 bits (pair0 < 0: these
// are not turned).  Found for a warp's rows at once: for each thread's it cost 2 us of 15.
__device__ __forceinline__ bool scale_in_doubt(float m) {
  return scale_exp(m * (1.f - 1.9073486328125e-06f)) != scale_exp(m * (1.f + 1.9073486328125e-06f));
}
template <int N>
__device__ __noinline__ int exact_scale_exp(const RopeTable& tb, const int32_t* pos, int pair0, const uint16_t* at1, const uint16_t* at2) {
  Segment<uint16_t, N> u, w;
  u.load(at1);
  w.load(at2);
  double a[N], b[N], s[N], c[N];
  spread(u, w, a, b);
  if (pair0 >= 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) rope_sincos(tb, pair0 + i, pos[tb.axis[(pair0 + i) >> 2]], s[i], c[i]);
    turn(a, b, s, c, tb.interleaved);
  }
  double m = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) {  // infinities and NaN do not count
    m = fmax(m, fabs(a[i]) <= kFltMax ? fabs(a[i]) : 0.0);
    m = fmax(m, fabs(b[i]) <= kFltMax ? fabs(b[i]) : 0.0);
  }
  return scale_exp(m);
}

// Dims of a thread's two segments: those of the rotation, or 2 kSeg neighbours.
template <int kSeg>
__device__ __forceinline__ void segments(const RopeTable& tb, bool rope, int g, int& o1, int& o2) {
  o1 = 2 * kSeg * g;
  o2 = o1 + kSeg;
  if (rope) {
    o1 = kSeg == 8 ? tb.wide1[g] : tb.o1[g];
    o2 = kSeg == 8 ? tb.wide2[g] : tb.o2[g];
  }
}

// A thread's rows of one task as they come from memory.
template <int kSeg>
struct RawRows {
  Segment<uint16_t, kSeg> u[16 / kSeg], w[16 / kSeg];
};

template <bool kE4m3, int kSeg>
__global__ void __launch_bounds__(32 * kWarps, 3) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = 32 / kSeg, kSteps = 16 / kSeg;  // threads of a row; rows of a step are kSeg
  __shared__ Chunk s_chunk;
  __shared__ int s_exp[2][kWarps];
  extern __shared__ float2 s_sc[];  // [rows of the page][32] (sine, cosine), with a rope
  const KvView& kv = p.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const Chunk c = find_chunk(kv, blockIdx.x, lane);
    if (lane == 0) s_chunk = c;
  }
  __syncthreads();
  const Chunk c = s_chunk;
  if (c.page < 0) return;
  const RopeTable& tb = p.rope;
  const int team_warps = kv.page >> 4, teams = kWarps / team_warps;
  const int team = warp / team_warps, wt = warp - team * team_warps;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int tasks = 2 * (min(h0 + p.heads_per_block, kv.n_heads) - h0);  // a head's keys, its values, the next head's keys, ..
  const int g = lane % kLanes, r0 = wt * 16 + lane / kLanes - c.row0;    // rows r0, r0 + kSeg, .. of the new ones
  auto load = [&](int task, RawRows<kSeg>& x) {
    if (task >= tasks) return;
    const bool is_k = (task & 1) == 0;
    int o1, o2;
    segments<kSeg>(tb, is_k && p.has_rope, g, o1, o2);
    const int head = h0 + (task >> 1);
    const uint16_t* src = is_k ? p.k_rows + head * p.k_hs : p.v_rows + head * p.v_hs;
    const long long ts = is_k ? p.k_ts : p.v_ts;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const int r = r0 + st * kSeg;
      if (r < 0 || r >= c.n) continue;
      const uint16_t* row = src + (c.token + r) * ts;
      x.u[st].load(row + o1);
      x.w[st].load(row + o2);
    }
  };
  RawRows<kSeg> now, next;
  load(team, now);  // on their way while the angles are worked out
  if (p.has_rope) {
    const int np = 4 * tb.n_groups;
    for (int i = threadIdx.x; i < c.n * 32; i += 32 * kWarps) {
      const int r = i >> 5, j = i & 31;
      if (j < np) {
        const int pos = p.pos[static_cast<long long>(c.token + r) * tb.n_axes + tb.axis[j >> 2]];
        float s, co;
        rope_sincos(tb, j, pos, s, co);
        s_sc[i] = make_float2(s, co);
      }
    }
    __syncthreads();
  }
  for (int i0 = 0, par = 0; i0 < tasks; i0 += teams, par ^= 1) {
    const int task = i0 + team;
    const bool live = task < tasks;
    const int head = h0 + (task >> 1);
    const bool is_k = (task & 1) == 0;
    const bool turns = is_k && p.has_rope && g * kSeg < 4 * tb.n_groups;
    int o1, o2;
    segments<kSeg>(tb, is_k && p.has_rope, g, o1, o2);
    const long long block = (static_cast<long long>(c.page) * kv.n_heads + head) << kv.page_log2;  // first row
    load(task + teams, next);
    // step st's values, turned (8-bit: twice, once for the largest and once to store; it costs less than keeping them)
    auto values = [&](int st, float(&a)[kSeg], float(&b)[kSeg]) {
      spread(now.u[st], now.w[st], a, b);
      if (!turns) return;
      const float4* sc = reinterpret_cast<const float4*>(s_sc + (r0 + st * kSeg) * 32 + kSeg * g);
      float s[kSeg], co[kSeg];
#pragma unroll
      for (int i = 0; i < kSeg / 2; ++i) {
        const float4 x = sc[i];
        s[2 * i] = x.x; co[2 * i] = x.y; s[2 * i + 1] = x.z; co[2 * i + 1] = x.w;
      }
      turn(a, b, s, co, tb.interleaved);
    };
    auto in = [&](int st) { return live && r0 + st * kSeg >= 0 && r0 + st * kSeg < c.n; };
    if constexpr (!kE4m3) {
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        if (!in(st)) continue;
        float a[kSeg], b[kSeg];
        values(st, a, b);
        store_rows(reinterpret_cast<uint16_t*>(is_k ? kv.k : kv.v) + (block + c.row0 + r0 + st * kSeg) * kD, o1, o2, a, b);
      }
    } else {
      float* scale = (is_k ? kv.k_scale : kv.v_scale) + static_cast<long long>(c.page) * kv.n_heads + head;
      const bool older = live && c.row0 > 0;
      const float was = older ? *scale : 0.f;
      float amax = 0.f;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        if (!in(st)) continue;
        float a[kSeg], b[kSeg];
        values(st, a, b);
        amax = largest(b, largest(a, amax));
      }
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // magnitudes order as their bits
      int e = scale_exp(amax);
      if (live && is_k && p.has_rope && scale_in_doubt(amax)) {  // the warp's rows once more
        e = kMinExp;
        const uint16_t* src = p.k_rows + head * p.k_hs;
        for (int r = r0; r < r0 + 16; r += kSeg) {
          if (r < 0 || r >= c.n) continue;
          const uint16_t* row = src + (c.token + r) * p.k_ts;
          e = max(e, exact_scale_exp<kSeg>(tb, p.pos + static_cast<long long>(c.token + r) * tb.n_axes, turns ? g * kSeg : -1, row + o1, row + o2));
        }
        e = __reduce_max_sync(0xffffffffu, e);
      }
      if (lane == 0) s_exp[par][warp] = e;
      __syncthreads();  // also: every thread has read the old scale
      if (live) {
        for (int x = 0; x < team_warps; ++x) e = max(e, s_exp[par][team * team_warps + x]);
        float to = power_of_two(e), inv = power_of_two(-e);
        uint8_t* dst = (is_k ? kv.k : kv.v) + block * kD;
        if (older) {
          if (to > was) {
            rescale_rows(dst, c.row0, was * inv, wt * 32 + lane, team_warps * 32);
          } else {
            to = was;
            inv = 1.f / was;  // a power of two: exact
          }
        }
        if (wt == 0 && lane == 0) *scale = to;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          if (!in(st)) continue;
          float a[kSeg], b[kSeg];
          values(st, a, b);
          uint8_t* row = dst + (c.row0 + r0 + st * kSeg) * kD;
          if (turns) {
            store_turned(row, o1, o2, a, b, inv, tb, p.pos + static_cast<long long>(c.token + r0 + st * kSeg) * tb.n_axes, g * kSeg,
                         now.u[st], now.w[st]);
          } else {
            store_codes(row + o1, a, inv);
            store_codes(row + o2, b, inv);
          }
        }
      }
    }
    now = next;
  }
}

// Steps of single tokens: a few threads of a warp have a key or value row of one token and head, so that one wave of blocks
// takes the whole step.
template <bool kE4m3, int kSeg>
__global__ void __launch_bounds__(32 * kWarps) append_token_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = 32 / kSeg;
  const KvView& kv = p.kv;
  const int lane = threadIdx.x & 31, g = lane % kLanes, rows = 2 * kv.n_heads;
  const long long i = (static_cast<long long>(blockIdx.x) * (32 * kWarps) + threadIdx.x) / kLanes;
  const int b = static_cast<int>(i / rows), task = static_cast<int>(i - static_cast<long long>(b) * rows);
  const bool is_k = task < kv.n_heads;
  const int head = is_k ? task : task - kv.n_heads;
  const RopeTable& tb = p.rope;
  int o1, o2;
  segments<kSeg>(tb, is_k && p.has_rope, g, o1, o2);
  SeqInfo s{0, 0, 0, false};
  if (b < kv.n_seqs) s = seq_info(kv, b);
  bool live = s.n_new > 0;
  const int at = s.len - 1, r = at & (kv.page - 1);
  int page = 0;
  float x[kSeg], y[kSeg];
  Segment<uint16_t, kSeg> u, w;
  const bool turns = is_k && p.has_rope && g * kSeg < 4 * tb.n_groups;
  const int32_t* pos = p.pos + static_cast<long long>(s.row0) * tb.n_axes;
  if (live) {
    page = kv.table[static_cast<long long>(b) * kv.max_pages + (at >> kv.page_log2)];
    const uint16_t* row = is_k ? p.k_rows + s.row0 * p.k_ts + head * p.k_hs : p.v_rows + s.row0 * p.v_ts + head * p.v_hs;
    u.load(row + o1);
    w.load(row + o2);
    if (turns) {
      float sn[kSeg], cs[kSeg];
#pragma unroll
      for (int j = 0; j < kSeg; ++j)
        rope_sincos(tb, g * kSeg + j, pos[tb.axis[(g * kSeg + j) >> 2]], sn[j], cs[j]);
      spread(u, w, x, y);
      turn(x, y, sn, cs, tb.interleaved);
    } else {
      spread(u, w, x, y);
    }
    if (page < 0 || page >= kv.n_pages) {
      atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
      live = false;
    }
  }
  const long long block = live ? (static_cast<long long>(page) * kv.n_heads + head) << kv.page_log2 : 0;  // first row
  if constexpr (!kE4m3) {
    if (live) store_rows(reinterpret_cast<uint16_t*>(is_k ? kv.k : kv.v) + (block + r) * kD, o1, o2, x, y);
  } else {
    float* scale = (is_k ? kv.k_scale : kv.v_scale) + (block >> kv.page_log2);
    const bool older = live && r > 0;
    const float was = older ? *scale : 0.f;
    const float m = live ? largest(y, largest(x, 0.f)) : 0.f;
    int e = scale_exp(m);
    if (turns && live && scale_in_doubt(m)) {
      const uint16_t* row = p.k_rows + s.row0 * p.k_ts + head * p.k_hs;
      e = exact_scale_exp<kSeg>(tb, pos, g * kSeg, row + o1, row + o2);
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, d));
    float now = power_of_two(e), inv = power_of_two(-e);
    const bool grows = older && now > was;
    if (older && !grows) {
      now = was;
      inv = 1.f / was;  // a power of two: exact
    }
    uint8_t* dst = (is_k ? kv.k : kv.v) + block * kD;
    // the whole warp rescales, row by row of those that need it
    uint32_t todo = __ballot_sync(0xffffffffu, grows && g == 0);
    while (todo) {
      const int q = __ffs(todo) - 1;
      todo &= todo - 1;
      const long long to = __shfl_sync(0xffffffffu, block, q);
      const bool k = __shfl_sync(0xffffffffu, static_cast<int>(is_k), q) != 0;
      rescale_rows((k ? kv.k : kv.v) + to * kD, __shfl_sync(0xffffffffu, r, q), __shfl_sync(0xffffffffu, was * inv, q), lane, 32);
    }
    if (!live) return;
    if (g == 0) *scale = now;
    if (turns) {
      store_turned(dst + r * kD, o1, o2, x, y, inv, tb, pos, g * kSeg, u, w);
    } else {
      store_codes(dst + r * kD + o1, x, inv);
      store_codes(dst + r * kD + o2, y, inv);
    }
  }
}

template <int kSeg>
void launch_append_seg(const AppendParams& p, bool e4m3, dim3 grid, size_t smem, cudaStream_t stream) {
  if (p.kv.max_new == 1) {
    if (e4m3)
      append_token_kernel<true, kSeg><<<grid, 32 * kWarps, 0, stream>>>(p);
    else
      append_token_kernel<false, kSeg><<<grid, 32 * kWarps, 0, stream>>>(p);
  } else if (e4m3) {
    append_kernel<true, kSeg><<<grid, 32 * kWarps, smem, stream>>>(p);
  } else {
    append_kernel<false, kSeg><<<grid, 32 * kWarps, smem, stream>>>(p);
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p0, bool e4m3, int num_sms, cudaStream_t stream, int* n_launch) {
  AppendParams p = p0;
  const KvView& kv = p.kv;
  if (kv.n_seqs == 0 || kv.n_tokens == 0 || kv.max_new == 0) return cudaSuccess;
  const bool wide = !p.has_rope || p.rope.wide;
  dim3 grid;
  size_t smem = 0;
  if (kv.max_new == 1) {
    const long long threads = static_cast<long long>(kv.n_seqs) * 2 * kv.n_heads * (wide ? 4 : 8);
    grid = dim3(static_cast<unsigned>((threads + 32 * kWarps - 1) / (32 * kWarps)));
  } else {
    // the pages that can take new rows: new rows of a sequence touch at most (new - 2) / page + 2 pages
    long long chunks = static_cast<long long>(kv.n_tokens) / kv.page + 2LL * kv.n_seqs;
    const long long each = (kv.max_new - 2) / kv.page + 2;
    chunks = chunks < each * kv.n_seqs ? chunks : each * kv.n_seqs;
    chunks = chunks < kv.n_tokens ? chunks : kv.n_tokens;
    // heads of a block share its sines: as many as leave 4 blocks for each SM, and at least what the teams take at once
    const int teams = kWarps / (kv.page >> 4);
    const int least = teams >= 2 ? teams / 2 : 1;
    int hpb = kv.n_heads;
    while (hpb > least && chunks * ((kv.n_heads + hpb - 1) / hpb) < 4LL * num_sms) hpb = (hpb + 1) / 2;
    p.heads_per_block = hpb;
    grid = dim3(static_cast<unsigned>(chunks), (kv.n_heads + hpb - 1) / hpb);
    smem = p.has_rope ? static_cast<size_t>(kv.page) * 32 * sizeof(float2) : 0;
  }
  if (wide)
    launch_append_seg<8>(p, e4m3, grid, smem, stream);
  else
    launch_append_seg<4>(p, e4m3, grid, smem, stream);
  ++*n_launch;
  return cudaGetLastError();
}

}  // namespace saf3r
