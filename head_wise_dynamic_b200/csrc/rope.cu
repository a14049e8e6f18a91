// Rotary positions with several axes: (a, b) -> (a cos x - b sin x, a sin x + b cos x) for every
// pair of a head's rotated dims, x = pos[axis] * base^(-2i/D).
//
// Bound by memory: x is read once and out written once.  A thread owns one token's group of four
// pairs (8 of the 64 dims), computes their sines and cosines once and walks a chunk of the heads
// with them, four heads' loads in flight.  32 tokens per block: a warp moves four whole rows per step.
#include <cmath>
#include <cstring>

#include "stream.h"

namespace saf3r {

static bool compute_rope_table(const saf3r_rope_cfg* cfg, RopeTable* t) {
  if (cfg->n_axes < 1 || cfg->n_axes > 4) return false;
  if (cfg->pairing != SAF3R_ROPE_HALF && cfg->pairing != SAF3R_ROPE_PAIRS && cfg->pairing != SAF3R_ROPE_SECTIONS)
    return false;
  if (!(cfg->base >= 1.0 && cfg->base <= 1e12)) return false;
  int width = 0;
  for (int a = 0; a < cfg->n_axes; ++a) {
    if (cfg->dims[a] < 8 || cfg->dims[a] > kD || (cfg->dims[a] & 7)) return false;
    width += cfg->dims[a];
  }
  if (width > kD) return false;
  const long double turn = 18446744073709551616.0L / 6.283185307179586476925286766559L;  // 2^64 / (2 pi)
  auto freq = [&](int i, int d) {
    return static_cast<uint64_t>(std::llroundl(turn * std::pow(static_cast<long double>(cfg->base), -2.0L * i / d)));
  };
  for (int i = 0; i < 32; ++i) t->freq[i] = 0;
  t->n_axes = cfg->n_axes;
  t->interleaved = cfg->pairing == SAF3R_ROPE_PAIRS;
  t->n_groups = width / 8;
  int at = 0;
  for (int a = 0; a < cfg->n_axes; ++a) {
    const int d = cfg->dims[a];
    for (int i = 0; i < d / 2; ++i)
      t->freq[at / 2 + i] = cfg->pairing == SAF3R_ROPE_SECTIONS ? freq(at / 2 + i, width) : freq(i, d);
    for (int i = 0; i < d / 8; ++i) {
      const int g = at / 8 + i;
      t->axis[g] = static_cast<int8_t>(a);
      if (cfg->pairing == SAF3R_ROPE_HALF) {
        t->o1[g] = static_cast<int8_t>(at + 4 * i);
        t->o2[g] = static_cast<int8_t>(at + d / 2 + 4 * i);
      } else if (cfg->pairing == SAF3R_ROPE_PAIRS) {
        t->o1[g] = static_cast<int8_t>(8 * g);
        t->o2[g] = static_cast<int8_t>(8 * g + 4);
      } else {
        t->o1[g] = static_cast<int8_t>(4 * g);
        t->o2[g] = static_cast<int8_t>(width / 2 + 4 * g);
      }
    }
    at += d;
  }
  for (int g = t->n_groups; g < 8; ++g) {
    t->axis[g] = 0;
    t->o1[g] = static_cast<int8_t>(8 * g);
    t->o2[g] = static_cast<int8_t>(8 * g + 4);
  }
  return true;
}

// The 32 frequencies take 10 us of the host's time, more than a small call's kernel: the table of this host thread's
// last configuration is kept, by the configuration's values.
bool build_rope_table(const saf3r_rope_cfg* cfg, RopeTable* t) {
  thread_local saf3r_rope_cfg last{};
  thread_local RopeTable table;
  thread_local bool have = false;
  if (!cfg) return false;
  if (have && std::memcmp(cfg, &last, sizeof(last)) == 0) {
    *t = table;
    return true;
  }
  if (!compute_rope_table(cfg, t)) return false;
  last = *cfg;
  table = *t;
  have = true;
  return true;
}

namespace {

constexpr int kTokens = 32;  // tokens of a block, 8 threads each

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}

template <typename In, typename Out>
__global__ void __launch_bounds__(8 * kTokens) rope_kernel(const __grid_constant__ RopeParams p) {
  const int g = threadIdx.x & 7;
  const long long t = static_cast<long long>(blockIdx.x) * kTokens + (threadIdx.x >> 3);
  if (t >= p.n_tokens) return;
  const RopeTable& tb = p.table;
  float s[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {1.f, 1.f, 1.f, 1.f};
  const int h0 = blockIdx.y * p.heads_per_block;
  const int h1 = min(h0 + p.heads_per_block, p.n_heads);
  const bool turns = g < tb.n_groups;
  if (turns && h0 < p.n_rot) {
    const int pos = p.pos[t * tb.n_axes + tb.axis[g]];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rope_sincos(tb, 4 * g + i, pos, s[i], c[i]);
      if (p.inverse) s[i] = -s[i];
    }
  }
  const int o1 = tb.o1[g], o2 = tb.o2[g];
  const In* x = static_cast<const In*>(p.x) + t * p.x_ts;
  Out* out = static_cast<Out*>(p.out) + t * p.out_ts;
  for (int h = h0; h < h1; h += 4) {
    float u[4][4], w[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (h + j < h1) {
        load4(x + (h + j) * p.x_hs + o1, u[j]);
        load4(x + (h + j) * p.x_hs + o2, w[j]);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (h + j >= h1) continue;
      if (turns && h + j < p.n_rot) {
        if (tb.interleaved) {
          const float a0 = u[j][0], a1 = u[j][2], a2 = w[j][0], a3 = w[j][2];
          const float b0 = u[j][1], b1 = u[j][3], b2 = w[j][1], b3 = w[j][3];
          u[j][0] = a0 * c[0] - b0 * s[0]; u[j][1] = a0 * s[0] + b0 * c[0];
          u[j][2] = a1 * c[1] - b1 * s[1]; u[j][3] = a1 * s[1] + b1 * c[1];
          w[j][0] = a2 * c[2] - b2 * s[2]; w[j][1] = a2 * s[2] + b2 * c[2];
          w[j][2] = a3 * c[3] - b3 * s[3]; w[j][3] = a3 * s[3] + b3 * c[3];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = u[j][i], b = w[j][i];
            u[j][i] = a * c[i] - b * s[i];
            w[j][i] = a * s[i] + b * c[i];
          }
        }
      }
      store4(out + (h + j) * p.out_hs + o1, u[j]);
      store4(out + (h + j) * p.out_hs + o2, w[j]);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p0, bool in_fp32, bool out_fp32, cudaStream_t stream, int* n_launch) {
  RopeParams p = p0;
  if (p.n_tokens == 0 || p.n_heads == 0) return cudaSuccess;
  const long long bx = (p.n_tokens + kTokens - 1) / kTokens;
  // heads of a block: as many as still leave a few blocks per SM (they share the sines), a multiple of 4
  int hpb = 16;
  while (hpb > 4 && bx * ((p.n_heads + hpb - 1) / hpb) < 1184) hpb -= 4;
  p.heads_per_block = hpb;
  const dim3 grid(static_cast<unsigned>(bx), (p.n_heads + hpb - 1) / hpb);
  if (in_fp32 && out_fp32)
    rope_kernel<float, float><<<grid, 8 * kTokens, 0, stream>>>(p);
  else if (in_fp32)
    rope_kernel<float, uint16_t><<<grid, 8 * kTokens, 0, stream>>>(p);
  else if (out_fp32)
    rope_kernel<uint16_t, float><<<grid, 8 * kTokens, 0, stream>>>(p);
  else
    rope_kernel<uint16_t, uint16_t><<<grid, 8 * kTokens, 0, stream>>>(p);
  ++*n_launch;
  return cudaGetLastError();
}

}  // namespace saf3r
