// Rotary positions with several axes: (a, b) -> (a cos x - b sin x, a sin x + b cos x) for every
// pair of a head's rotated dims, x = pos[axis] * base^(-2i/D).
//
// Bound by memory: x is read once and out written once.  A thread owns four or eight pairs of one token, computes
// their sines and cosines once and walks some of the heads with them.
#include <cmath>
#include <cstring>

#include "rope.cuh"
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
  // two groups as one of two 8-value segments, where both halves are contiguous and aligned
  t->wide = t->n_groups % 2 == 0;
  for (int q = 0; q < 4; ++q) {
    const bool copied = t->interleaved || 2 * q >= t->n_groups;
    t->wide1[q] = copied ? static_cast<int8_t>(16 * q) : t->o1[2 * q];
    t->wide2[q] = copied ? static_cast<int8_t>(16 * q + 8) : t->o2[2 * q];
    if (!copied && (t->o1[2 * q] % 8 || t->o2[2 * q] % 8 || t->o1[2 * q + 1] != t->o1[2 * q] + 4 || t->o2[2 * q + 1] != t->o2[2 * q] + 4))
      t->wide = 0;
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

constexpr int kThreads = 256;

// A thread owns two segments of kSeg values of one token's rows (kSeg pairs): 8 where the pairing's halves are
// aligned to 8 values, else 4.  It asks for its first heads' rows before it works out the angles, and has
// 128 bytes of rows on their way at a time.  Measured (43,968 tokens, 48 heads, bf16): 89 us, 93% of a plain
// copy's rate; with 4-value segments and 64 bytes on their way 136 us.
template <typename In, typename Out, int kSeg>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = 32 / kSeg;  // threads of a row
  constexpr int kFly = 64 / (kSeg * static_cast<int>(sizeof(In)));
  const int g = threadIdx.x % kLanes;
  const long long t = static_cast<long long>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (t >= p.n_tokens) return;
  const RopeTable& tb = p.table;
  const int o1 = kSeg == 8 ? tb.wide1[g] : tb.o1[g], o2 = kSeg == 8 ? tb.wide2[g] : tb.o2[g];
  const int h0 = blockIdx.y * p.heads_per_block, h1 = min(h0 + p.heads_per_block, p.n_heads);
  const In* x = static_cast<const In*>(p.x) + t * p.x_ts;
  Out* out = static_cast<Out*>(p.out) + t * p.out_ts;
  Segment<In, kSeg> u[kFly], w[kFly];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < kFly; ++j)
      if (h + j < h1) {
        u[j].load(x + (h + j) * p.x_hs + o1);
        w[j].load(x + (h + j) * p.x_hs + o2);
      }
  };
  load(h0);
  float s[kSeg], c[kSeg];
  const bool turns = g * kSeg < 4 * tb.n_groups && h0 < p.n_rot;
  if (turns) {
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
      const int pos = p.pos[t * tb.n_axes + tb.axis[(g * kSeg + i) >> 2]];
      rope_sincos(tb, g * kSeg + i, pos, s[i], c[i]);
      if (p.inverse) s[i] = -s[i];
    }
  }
  for (int h = h0;;) {
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      if (h + j >= h1) break;
      float a[kSeg], b[kSeg];
      spread(u[j], w[j], a, b);
      if (turns && h + j < p.n_rot) turn(a, b, s, c, tb.interleaved);
      Segment<Out, kSeg> ra, rb;
#pragma unroll
      for (int i = 0; i < kSeg; i += 2) {
        ra.set2(i, a[i], a[i + 1]);
        rb.set2(i, b[i], b[i + 1]);
      }
      ra.store(out + (h + j) * p.out_hs + o1);
      rb.store(out + (h + j) * p.out_hs + o2);
    }
    h += kFly;
    if (h >= h1) break;
    load(h);
  }
}

template <int kSeg>
void launch_rope_seg(const RopeParams& p, bool in_fp32, bool out_fp32, dim3 grid, cudaStream_t stream) {
  if (in_fp32 && out_fp32)
    rope_kernel<float, float, kSeg><<<grid, kThreads, 0, stream>>>(p);
  else if (in_fp32)
    rope_kernel<float, uint16_t, kSeg><<<grid, kThreads, 0, stream>>>(p);
  else if (out_fp32)
    rope_kernel<uint16_t, float, kSeg><<<grid, kThreads, 0, stream>>>(p);
  else
    rope_kernel<uint16_t, uint16_t, kSeg><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p0, bool in_fp32, bool out_fp32, int num_sms, cudaStream_t stream, int* n_launch) {
  RopeParams p = p0;
  if (p.n_tokens == 0 || p.n_heads == 0) return cudaSuccess;
  const int seg = p.table.wide ? 8 : 4, tokens = kThreads * seg / 32;
  const long long bx = (p.n_tokens + tokens - 1) / tokens;
  // heads of a block share its sines: as many as leave at least 16 blocks for each SM, and no fewer than are in flight
  const int fly = 64 / (seg * (in_fp32 ? 4 : 2));
  int hpb = 4 * fly;
  while (hpb > fly && bx * ((p.n_heads + hpb - 1) / hpb) < 16LL * num_sms) hpb /= 2;
  p.heads_per_block = hpb;
  const dim3 grid(static_cast<unsigned>(bx), (p.n_heads + hpb - 1) / hpb);
  if (seg == 8)
    launch_rope_seg<8>(p, in_fp32, out_fp32, grid, stream);
  else
    launch_rope_seg<4>(p, in_fp32, out_fp32, grid, stream);
  ++*n_launch;
  return cudaGetLastError();
}

}  // namespace saf3r
