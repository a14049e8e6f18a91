// One query row's attention, key by key in fp32: the slow exact path for rows next to which a masked
// value row is not finite (0 * infinity in a tile product would reach rows that do not see it).
#pragma once
#include "stream.h"

namespace saf3r {

// Page of row j (of sequence b), -1: none (views held at once have none).
__device__ __forceinline__ int page_of(const KvAttnParams& p, int b, int j) {
  return p.ck ? 0 : p.kv.table[static_cast<long long>(b) * p.kv.max_pages + (j >> p.kv.page_log2)];
}
// Element index of row j (of kv head hk, on page id) in its pool, and the index of its scale; -1: none.
__device__ __forceinline__ long long kv_row(const KvAttnParams& p, int id, int hk, int j, long long* scale) {
  const KvView& kv = p.kv;
  if (p.ck) return (static_cast<long long>(hk) * kv.n_tokens + j) * kD;
  if (id < 0 || id >= kv.n_pages) {
    atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
    return -1;
  }
  *scale = static_cast<long long>(id) * kv.n_heads + hk;
  return ((*scale << kv.page_log2) + (j & (kv.page - 1))) * kD;
}

// The answer of a row whose weights add up to 0.  Every row sees itself at least, so all its logits are minus infinity, and
// the softmax of those is not a number.
__device__ __forceinline__ float no_weight() { return __uint_as_float(0x7fffffffu); }

// Two neighbouring values (bits of bf16, or codes) as fp32.
template <bool kCodes>
__device__ __forceinline__ float2 pair_of(uint32_t bits) {
  if constexpr (!kCodes) return make_float2(__uint_as_float(bits << 16), __uint_as_float(bits & 0xffff0000u));
  return f32x2_of_f16x2(f16x2_of_e4m3(bits));
}

// Run by one warp: token `row` of the step's tensors, at position pos of sequence b.  Writes columns c0..c1-1.  32 keys at a
// time, a lane each: its logit from 16-byte loads of the key, then the values of 4 keys on their way at a time (8 take more
// registers than the callers have to spare), two columns a lane; page entries a step ahead.  kCodes: the cache holds 8-bit
// codes.  About 800 instructions that wait for one another for 32 keys, 0.11 us a key (0.46 when every value was loaded by itself, which for the 32 rows of a warp of the tensor-core kernel
// was longer than the other warps wait from 140,000 keys on; now it is from 550,000 on).  Prefetches change nothing.
template <bool kCodes>
static __device__ __noinline__ void exact_row(const KvAttnParams& p, int b, int len, int row, int pos, int head, int lane, int c0,
                                              int c1) {
  constexpr int kSize = kCodes ? 1 : 2;  // bytes of a value
  const int hk = p.by_group.div(head);
  const Span sp = span_of(p.win, pos, len);
  const uint4* q = reinterpret_cast<const uint4*>(p.q + row * p.q_ts + head * p.q_hs);
  const uint8_t* keys = p.ck ? reinterpret_cast<const uint8_t*>(p.ck) : p.kv.k;
  const uint8_t* values = (p.ck ? reinterpret_cast<const uint8_t*>(p.cv) : p.kv.v) + 2 * lane * kSize;
  float m = -INFINITY, l = 0.f, a0 = 0.f, a1 = 0.f;
  const Runs runs = runs_of(sp.lo, sp.hi, sp.sink);
  for (int part = 0; part < 2; ++part) {
    const int end = part ? runs.b_end : runs.a_end;
    int j = (part ? runs.b_begin : 0) + lane;
    int id = j < end ? page_of(p, b, j) : 0;
    for (; j - lane < end; j += 32) {
      long long at = -1, sc = 0;
      if (j < end) at = kv_row(p, id, hk, j, &sc);
      if (j + 32 < end) id = page_of(p, b, j + 32);
      float s = -INFINITY, vs = 1.f;
      if (at >= 0) {
        const uint4* key = reinterpret_cast<const uint4*>(keys + at * kSize);
        constexpr int kLoads = kCodes ? 4 : 8;
        uint4 k[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) k[i] = key[i];
        float ks = 1.f;
        if (kCodes) {
          ks = p.kv.k_scale[sc];
          vs = p.kv.v_scale[sc];
        }
        float dot[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // 8 dims
          const uint4 qv = q[i], y = k[kCodes ? i >> 1 : i];
          uint32_t kw[4] = {y.x, y.y, y.z, y.w};
          if (kCodes) {
            const uint32_t lo = (i & 1) ? y.z : y.x, hi = (i & 1) ? y.w : y.y;
            kw[0] = lo; kw[1] = lo >> 16; kw[2] = hi; kw[3] = hi >> 16;
          }
          const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = pair_of<false>(qw[e]), w = pair_of<kCodes>(kw[e]);
            dot[0] += u.x * w.x;
            dot[1] += u.y * w.y;
          }
        }
        s = (dot[0] + dot[1]) * ks * 0.125f;
      }
      float mx = s;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(m, mx);
      const float f = m == -INFINITY ? 0.f : expf(m - mn);
      const float w = at >= 0 ? expf(s - (mn == -INFINITY ? 0.f : mn)) : 0.f;
      float ws = w;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, d);
      // (a0, a1) stays the mean of the values so far: a sum of large ones would leave fp32's range
      const float before = l * f;
      l = before + ws;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      a0 *= before * inv;
      a1 *= before * inv;
      m = mn;
      const float wv = w * inv * vs;
#pragma unroll 1
      for (int i0 = 0; i0 < 32; i0 += 4) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long vi = __shfl_sync(0xffffffffu, at, i0 + i);
          // (a key that is not there: some row, its bits left out)
          const uint8_t* v = vi >= 0 ? values + vi * kSize : reinterpret_cast<const uint8_t*>(q) + 2 * lane * kSize;
          x[i] = kCodes ? *reinterpret_cast<const uint16_t*>(v) : *reinterpret_cast<const uint32_t*>(v);
          if (vi < 0) x[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float wi = __shfl_sync(0xffffffffu, wv, i0 + i);
          const float2 v = pair_of<kCodes>(x[i]);
          a0 += wi * v.x;
          a1 += wi * v.y;
        }
      }
    }
  }
  if (l == 0.f) a0 = a1 = no_weight();
  if (2 * lane < c0 || 2 * lane >= c1) return;
  const long long o = row * p.out_ts + head * p.out_hs + 2 * lane;
  if (p.out_fp32) {
    static_cast<float*>(p.out)[o] = a0;
    static_cast<float*>(p.out)[o + 1] = a1;
  } else {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(a1), "f"(a0));
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + o) = r;
  }
}

}  // namespace saf3r
