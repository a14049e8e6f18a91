// Appends a step's keys and values to the paged cache, the keys rotated on the way.
//
// A block owns one page of one sequence that takes new rows, for some of the kv heads: 8 warps in
// teams of page / 16, each team one head's keys or values, a warp 16 rows of the page.  A team
// holds its rows in registers in fp32 between the largest magnitude (8-bit caches: it fixes the
// page's scale) and the store, so every row is read once.  Sines and cosines are computed once per block
// and row and shared by its heads.  Because one block owns a (page, head), growing a scale and
// re-rounding the older rows needs no atomics.  Bound by memory for whole views, by launch and
// latency for single tokens.
//
// Scales are powers of two: x / scale is exact, and re-rounding older codes when a scale grows is too
// unless they become subnormal.
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
  if (kv.max_new == 1) {
    b = x;
    s = seq_info(kv, b);
  } else {
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

__device__ __forceinline__ void unpack(uint2 x, float (&v)[8], int at) {
  v[at] = __uint_as_float(x.x << 16); v[at + 1] = __uint_as_float(x.x & 0xffff0000u);
  v[at + 2] = __uint_as_float(x.y << 16); v[at + 3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes >> (16 * i))));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1]) : "r"(h));
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

template <bool kE4m3>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ Chunk s_chunk;
  __shared__ float s_amax[2][kWarps];
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
  const int team_warps = kv.page >> 4, teams = kWarps / team_warps;
  const int team = warp / team_warps, wt = warp - team * team_warps;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int tasks = 2 * (min(h0 + p.heads_per_block, kv.n_heads) - h0);
  const int g = lane & 7;
  for (int i0 = 0, par = 0; i0 < tasks; i0 += teams, par ^= 1) {
    const int task = i0 + team;
    const bool live = task < tasks;
    const int head = h0 + (task >> 1);
    const bool is_k = (task & 1) == 0;
    const bool turns = is_k && p.has_rope && g < tb.n_groups;
    const int o1 = is_k && p.has_rope ? tb.o1[g] : 8 * g;
    const int o2 = is_k && p.has_rope ? tb.o2[g] : 8 * g + 4;
    const uint16_t* src = (is_k ? p.k_rows : p.v_rows) + head * (is_k ? p.k_hs : p.v_hs);
    const long long ts = is_k ? p.k_ts : p.v_ts;
    const long long block = (static_cast<long long>(c.page) * kv.n_heads + head) << kv.page_log2;  // first row
    float x[4][8];
    uint2 raw[4][2];
    bool in[4];
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      const int r = wt * 16 + st * 4 + (lane >> 3) - c.row0;
      in[st] = live && r >= 0 && r < c.n;
      if (in[st]) {
        const uint16_t* row = src + (c.token + r) * ts;
        raw[st][0] = *reinterpret_cast<const uint2*>(row + o1);
        raw[st][1] = *reinterpret_cast<const uint2*>(row + o2);
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      if (!in[st]) continue;
      unpack(raw[st][0], x[st], 0);
      unpack(raw[st][1], x[st], 4);
      if (turns) {
        const int r = wt * 16 + st * 4 + (lane >> 3) - c.row0;
        const float4* sc = reinterpret_cast<const float4*>(s_sc + r * 32 + 4 * g);
        const float4 t0 = sc[0], t1 = sc[1];
        const float s[4] = {t0.x, t0.z, t1.x, t1.z}, co[4] = {t0.y, t0.w, t1.y, t1.w};
        if (tb.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[st][2 * i], b = x[st][2 * i + 1];
            x[st][2 * i] = a * co[i] - b * s[i];
            x[st][2 * i + 1] = a * s[i] + b * co[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[st][i], b = x[st][4 + i];
            x[st][i] = a * co[i] - b * s[i];
            x[st][4 + i] = a * s[i] + b * co[i];
          }
        }
      }
      if (kE4m3) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = fabsf(x[st][i]);
          amax = fmaxf(amax, a <= kFltMax ? a : 0.f);  // infinities and NaN do not count
        }
      }
    }
    if constexpr (!kE4m3) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(is_k ? kv.k : kv.v) + block * kD;
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (!in[st]) continue;
        uint16_t* row = dst + (wt * 16 + st * 4 + (lane >> 3)) * kD;
        *reinterpret_cast<uint2*>(row + o1) = make_uint2(pack2(x[st][0], x[st][1]), pack2(x[st][2], x[st][3]));
        *reinterpret_cast<uint2*>(row + o2) = make_uint2(pack2(x[st][4], x[st][5]), pack2(x[st][6], x[st][7]));
      }
      continue;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (lane == 0) s_amax[par][warp] = amax;
    float* scale = (is_k ? kv.k_scale : kv.v_scale) + static_cast<long long>(c.page) * kv.n_heads + head;
    const bool older = live && c.row0 > 0;
    const float was = older ? *scale : 0.f;
    __syncthreads();  // also: every thread has read the old scale
    if (!live) continue;
    float m = 0.f;
    for (int w = 0; w < team_warps; ++w) m = fmaxf(m, s_amax[par][team * team_warps + w]);
    const int e = scale_exp(m);
    float now = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint8_t* dst = (is_k ? kv.k : kv.v) + block * kD;
    if (older) {
      if (now > was) {
        const float f = was * inv;
        uint4* old = reinterpret_cast<uint4*>(dst);
        for (int i = wt * 32 + lane; i < c.row0 * 4; i += team_warps * 32) {
          uint4 v = old[i];
          v.x = rescale4(v.x, f);
          v.y = rescale4(v.y, f);
          v.z = rescale4(v.z, f);
          v.w = rescale4(v.w, f);
          old[i] = v;
        }
      } else {
        now = was;
        inv = 1.f / was;  // a power of two: exact
      }
    }
    if (wt == 0 && lane == 0) *scale = now;
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      if (!in[st]) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = x[st][i];
        x[st][i] = fabsf(a) <= kFltMax ? a * inv : __uint_as_float(0x7fffffffu);
      }
      uint8_t* row = dst + (wt * 16 + st * 4 + (lane >> 3)) * kD;
      *reinterpret_cast<uint32_t*>(row + o1) = e4m3x4(x[st][0], x[st][1], x[st][2], x[st][3]);
      *reinterpret_cast<uint32_t*>(row + o2) = e4m3x4(x[st][4], x[st][5], x[st][6], x[st][7]);
    }
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p0, bool e4m3, int num_sms, cudaStream_t stream, int* n_launch) {
  AppendParams p = p0;
  const KvView& kv = p.kv;
  if (kv.n_seqs == 0 || kv.n_tokens == 0 || kv.max_new == 0) return cudaSuccess;
  // the pages that can take new rows: new rows of a sequence touch at most (new - 2) / page + 2 pages
  long long chunks = kv.n_seqs;
  if (kv.max_new > 1) {
    chunks = static_cast<long long>(kv.n_tokens) / kv.page + 2LL * kv.n_seqs;
    const long long each = (kv.max_new - 2) / kv.page + 2;
    chunks = chunks < each * kv.n_seqs ? chunks : each * kv.n_seqs;
    chunks = chunks < kv.n_tokens ? chunks : kv.n_tokens;
  }
  // heads of a block share its sines: as many as leave a few blocks per SM, and at least what the teams take at once
  const int teams = kWarps / (kv.page >> 4);
  const int least = teams >= 2 ? teams / 2 : 1;
  int hpb = kv.n_heads;
  while (hpb > least && chunks * ((kv.n_heads + hpb - 1) / hpb) < 4LL * num_sms) hpb = (hpb + 1) / 2;
  p.heads_per_block = hpb;
  const dim3 grid(static_cast<unsigned>(chunks), (kv.n_heads + hpb - 1) / hpb);
  const size_t smem = p.has_rope ? static_cast<size_t>(kv.page) * 32 * sizeof(float2) : 0;
  if (e4m3)
    append_kernel<true><<<grid, 32 * kWarps, smem, stream>>>(p);
  else
    append_kernel<false><<<grid, 32 * kWarps, smem, stream>>>(p);
  ++*n_launch;
  return cudaGetLastError();
}

}  // namespace saf3r
