// One query row's attention, key by key in fp32: the slow exact path for rows next to which a masked
// value row is not finite (0 * infinity in a tile product would reach rows that do not see it).
#pragma once
#include "stream.h"

namespace saf3r {

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float e4m3_at(const uint8_t* p) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(*p)));
  float v;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(v) : "r"(h));
  return v;
}

// Element index of row j (of kv head hk of sequence b) in its pool, and the index of its scale; -1: none.
__device__ __forceinline__ long long kv_row(const KvAttnParams& p, int b, int hk, int j, long long* scale) {
  const KvView& kv = p.kv;
  if (p.ck) return (static_cast<long long>(hk) * kv.n_tokens + j) * kD;
  const int id = kv.table[static_cast<long long>(b) * kv.max_pages + (j >> kv.page_log2)];
  if (id < 0 || id >= kv.n_pages) {
    atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
    return -1;
  }
  *scale = static_cast<long long>(id) * kv.n_heads + hk;
  return ((*scale << kv.page_log2) + (j & (kv.page - 1))) * kD;
}

// Run by one warp: token `row` of the step's tensors, at position pos of sequence b.  Writes columns c0..c1-1.
static __device__ __noinline__ void exact_row(const KvAttnParams& p, int b, int len, int row, int pos, int head, int lane, int c0,
                                       int c1) {
  const int hk = p.by_group.div(head);
  const Span sp = span_of(p.win, pos, len);
  const uint16_t* q = p.q + row * p.q_ts + head * p.q_hs;
  float m = -INFINITY, l = 0.f, a0 = 0.f, a1 = 0.f;
  const Runs runs = runs_of(sp.lo, sp.hi, sp.sink);
  for (int part = 0; part < 2; ++part) {
    const int end = part ? runs.b_end : runs.a_end;
    for (int j0 = part ? runs.b_begin : 0; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      long long at = -1, sc = 0;
      if (j < end) at = kv_row(p, b, hk, j, &sc);
      float s = -INFINITY, vs = 1.f;
      if (at >= 0) {
        float dot = 0.f;
        if (p.ck) {
          for (int d = 0; d < kD; ++d) dot += bf16_at(q + d) * bf16_at(p.ck + at + d);
        } else if (!p.e4m3) {
          for (int d = 0; d < kD; ++d) dot += bf16_at(q + d) * bf16_at(reinterpret_cast<const uint16_t*>(p.kv.k) + at + d);
        } else {
          for (int d = 0; d < kD; ++d) dot += bf16_at(q + d) * e4m3_at(p.kv.k + at + d);
          dot *= p.kv.k_scale[sc];
          vs = p.kv.v_scale[sc];
        }
        s = dot * 0.125f;
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
      l = l * f + ws;
      a0 *= f;
      a1 *= f;
      m = mn;
      for (int i = 0; i < 32; ++i) {
        const long long vi = __shfl_sync(0xffffffffu, at, i);
        if (vi < 0) continue;
        const float wi = __shfl_sync(0xffffffffu, w * vs, i);
        float v0, v1;
        if (p.ck || !p.e4m3) {
          const uint16_t* v = (p.ck ? p.cv : reinterpret_cast<const uint16_t*>(p.kv.v)) + vi + 2 * lane;
          v0 = bf16_at(v);
          v1 = bf16_at(v + 1);
        } else {
          v0 = e4m3_at(p.kv.v + vi + 2 * lane);
          v1 = e4m3_at(p.kv.v + vi + 2 * lane + 1);
        }
        a0 += wi * v0;
        a1 += wi * v1;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  a0 *= inv;
  a1 *= inv;
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
