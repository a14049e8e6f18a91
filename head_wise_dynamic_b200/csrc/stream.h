// Plans of the streaming operators (rotary positions, paged key/value append, attention over the
// cache), shared by their kernels and the host side.  Not part of the C ABI.
#pragma once
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace saf3r {

// Rotation table of a head's 64 dims in 8 groups of 8 values: group g holds dims o1[g]..+3 and
// o2[g]..+3.  Groups below n_groups turn four pairs each (pairs 4g..4g+3), the others are copied.
// freq is the turn per position in units of 2^-64 turns, so pos * freq modulo 2^64 is the angle's
// fraction of a turn with no reduction error at any int32 position.
struct RopeTable {
  uint64_t freq[32];
  int8_t axis[8], o1[8], o2[8];
  int32_t n_groups;
  int32_t interleaved;  // pairs (0,1),(2,3) of each half of a group, and o2 = o1 + 4; else (o1 + i, o2 + i)
  int32_t n_axes;
  int32_t wide;         // groups 2q and 2q + 1 join to dims wide1[q]..+7 and wide2[q]..+7
  int8_t wide1[4], wide2[4];
};

struct RopeParams {
  RopeTable table;
  const void* x;
  void* out;
  const int32_t* pos;
  long long n_tokens, x_ts, x_hs, out_ts, out_hs;
  int32_t n_heads, n_rot, inverse, heads_per_block;
};

// A batch's device arrays and the cache, as the kernels see them.
struct KvView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* cu;
  const int32_t* kv_lens;
  const int32_t* table;
  int* err;
  int32_t n_pages, n_heads, page, page_log2;
  int32_t n_seqs, n_tokens, max_new, max_pages;
};

struct AppendParams {
  KvView kv;
  RopeTable rope;
  int32_t has_rope, heads_per_block;
  const uint16_t* k_rows;
  const uint16_t* v_rows;
  long long k_ts, k_hs, v_ts, v_hs;
  const int32_t* pos;
};

// n / d for 0 <= n < 2^31 by a multiplication: with 2^l >= d > 2^(l-1), q = (t + ((n - t) >> s1)) >> s2, t the upper half
// of n * mul, mul = floor(2^32 (2^l - d) / d) + 1 (Granlund and Montgomery, "Division by invariant integers using
// multiplication").  The attention kernels divide by two numbers of the call, and a division waits 10 times as long.
struct FastDiv {
  uint32_t mul, s1, s2;
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const {
    const uint32_t t = __umulhi(mul, static_cast<uint32_t>(n));
    return static_cast<int>((t + ((static_cast<uint32_t>(n) - t) >> s1)) >> s2);
  }
#endif
};
inline FastDiv make_div(int32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < static_cast<uint64_t>(d)) ++l;
  FastDiv f;
  f.mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - static_cast<uint64_t>(d))) / static_cast<uint64_t>(d) + 1);
  f.s1 = l > 1 ? 1 : l;
  f.s2 = l > 1 ? l - 1 : 0;
  return f;
}

struct WindowMask {
  int32_t view, window, sink, causal;
  FastDiv by_view;
};

struct KvAttnParams {
  KvView kv;          // contiguous mode (ck != NULL): n_heads, n_seqs = 1, n_tokens, err only
  WindowMask win;
  const uint16_t* ck;  // keys and values held at once, bf16 [heads][n_tokens][64] (NULL: the paged cache)
  const uint16_t* cv;
  const uint16_t* q;
  void* out;
  long long q_ts, q_hs, out_ts, out_hs;
  int32_t n_heads, group, out_fp32;
  FastDiv by_group;
  int32_t e4m3;
  uint8_t* ws;
  int32_t num_sms;
  long long wait_budget;
  int32_t withhold;
  int32_t least_share; // few rows: chunks that are worth a warp
  int32_t box_log2;    // keys of one TMA box
  int32_t q_tma;       // tensor cores: the queries come by TMA
};

#ifdef __CUDACC__

// Two codes (the lower 16 bits) as fp16, exactly; two fp16 values as fp32; two fp32 values rounded to fp16.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ float2 f32x2_of_f16x2(uint32_t h) {
  float2 v;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(v.x), "=f"(v.y) : "r"(h));
  return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^e, e in -126 .. 127
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Sequence b of a batch: its rows, cached length and whether the numbers fit.
struct SeqInfo {
  int row0, n_new, len;
  bool ok;
};
__device__ __forceinline__ SeqInfo seq_info(const KvView& kv, int b) {
  SeqInfo s;
  if (kv.cu == nullptr) return SeqInfo{0, kv.n_tokens, kv.n_tokens, true};  // views held at once
  s.row0 = kv.cu[b];
  const int end = kv.cu[b + 1];
  s.len = kv.kv_lens[b];
  s.n_new = end - s.row0;
  s.ok = s.row0 >= 0 && end >= s.row0 && end <= kv.n_tokens && s.n_new <= kv.max_new && s.len >= s.n_new &&
         s.len <= (static_cast<long long>(kv.max_pages) << kv.page_log2);
  if (!s.ok) {
    atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
    s.row0 = s.n_new = s.len = 0;
  }
  return s;
}

// The keys a query at position p of a sequence of len tokens sees: [lo, hi) and [0, sink).
struct Span {
  int lo, hi, sink;
};
__device__ __forceinline__ Span span_of(const WindowMask& w, int p, int len) {
  const long long f = w.by_view.div(p);
  Span s;
  s.lo = 0;
  if (w.window > 0 && f - w.window + 1 > 0) s.lo = static_cast<int>((f - w.window + 1) * w.view);
  const long long end = w.causal ? (f + 1) * w.view : (w.window > 0 ? (f + w.window) * w.view : len);
  s.hi = end < len ? static_cast<int>(end) : len;
  s.sink = min(w.sink, w.causal ? s.hi : len);
  return s;
}

// The same as two runs of keys in order: [0, a_end) and [b_begin, b_end).  For a tile of queries at positions
// first..last: lo of the first, hi and sink of the last.
struct Runs {
  int a_end, b_begin, b_end;
};
__device__ __forceinline__ Runs runs_of(int lo, int hi, int sink) {
  if (sink >= lo) return Runs{0, 0, max(hi, sink)};
  return Runs{sink, lo, hi};
}

// The chunks (64 keys, from multiples of 64) that two runs touch, in order.
struct Chunks {
  int na, b0, total;
  __device__ __forceinline__ int key(int i) const { return (i < na ? i : i - na + b0) << 6; }
};
__device__ __forceinline__ Chunks chunks_of(const Runs& r) {
  Chunks c;
  c.na = (r.a_end + 63) >> 6;
  c.b0 = r.b_begin >> 6;
  if (c.b0 < c.na) c.na = 0, c.b0 = 0;  // the runs share a chunk
  c.total = c.na + (r.b_end > r.b_begin ? ((r.b_end + 63) >> 6) - c.b0 : 0);
  return c;
}

// The angle pos * freq as a signed part of a quarter turn from the nearest one: r * 2^-64, and which quarter.
__device__ __forceinline__ int64_t rope_angle(const RopeTable& t, int pair, int pos, uint32_t& quarter) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * t.freq[pair];
  quarter = static_cast<uint32_t>((turn + (1ull << 61)) >> 62);
  return static_cast<int64_t>(turn << 2);
}
template <typename T>
__device__ __forceinline__ void to_quarter(uint32_t quarter, T& s, T& c) {
  if (quarter & 1) {
    const T x = s;
    s = c;
    c = -x;
  }
  if (quarter & 2) {
    s = -s;
    c = -c;
  }
}
__device__ __forceinline__ void rope_sincos(const RopeTable& t, int pair, int pos, float& s, float& c) {
  uint32_t quarter;
  const int64_t r = rope_angle(t, pair, pos, quarter);
  // the upper 32 bits, in half turns: [-1/4, 1/4)
  sincospif(static_cast<float>(static_cast<int32_t>(r >> 32)) * 1.1641532182693481e-10f, &s, &c);
  to_quarter(quarter, s, c);
}
// The same in 64 bits, by the sine's and cosine's series: |x| <= pi / 4, so the terms left out are below 1e-15.
__device__ __forceinline__ void rope_sincos(const RopeTable& t, int pair, int pos, double& s, double& c) {
  uint32_t quarter;
  const double x = static_cast<double>(rope_angle(t, pair, pos, quarter)) * (1.5707963267948966 / 18446744073709551616.0);
  const double y = x * x;
  double a = -1.0 / 1307674368000.0, b = -1.0 / 87178291200.0;
  a = fma(a, y, 1.0 / 6227020800.0);
  b = fma(b, y, 1.0 / 479001600.0);
  a = fma(a, y, -1.0 / 39916800.0);
  b = fma(b, y, -1.0 / 3628800.0);
  a = fma(a, y, 1.0 / 362880.0);
  b = fma(b, y, 1.0 / 40320.0);
  a = fma(a, y, -1.0 / 5040.0);
  b = fma(b, y, -1.0 / 720.0);
  a = fma(a, y, 1.0 / 120.0);
  b = fma(b, y, 1.0 / 24.0);
  a = fma(a, y, -1.0 / 6.0);
  b = fma(b, y, -0.5);
  s = fma(a * y, x, x);
  c = fma(b, y, 1.0);
  to_quarter(quarter, s, c);
}

#endif

// Launches a kernel whose blocks are set up while the one before it in the stream still runs, and which waits for that one's end
// on the device (griddepcontrol.wait) before it reads what it wrote.
template <typename Kernel, typename Params>
cudaError_t launch_behind(Kernel kernel, dim3 grid, dim3 block, cudaStream_t stream, const Params& p) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

bool build_rope_table(const saf3r_rope_cfg* cfg, RopeTable* t);
cudaError_t launch_rope(const RopeParams& p, bool in_fp32, bool out_fp32, int num_sms, cudaStream_t stream, int* n_launch);
cudaError_t launch_append(const AppendParams& p, bool e4m3, int num_sms, cudaStream_t stream, int* n_launch);

// few query rows per sequence and kv head (kv_decode.cu)
bool decode_takes(int max_new, int group);
size_t decode_workspace_bytes(const KvView& kv, int group);
saf3r_status launch_decode(const KvAttnParams& p, cudaStream_t stream, int* n_launch);

// the tensor-core kernel (kv_attn_sm100.cu)
size_t attn_workspace_bytes();
saf3r_status launch_attn(const KvAttnParams& p, cudaStream_t stream, int* n_launch);

// host side of api.cu that the streaming entry points share
bool call_device(int* sms, int* major, int** err);
saf3r_status validate_layout(const saf3r_layout* L);
void set_launch_count(int n);
long long call_wait_budget();
bool take_withhold_arrive();
bool make_map_rows(CUtensorMap* m, const void* base, long long rows, long long row_stride, int heads,
                   long long head_stride, int box_rows);
bool make_map_queries(CUtensorMap* m, const void* q, int group, int n_tokens, int kv_heads, long long token_stride,
                      long long head_stride, int box_tokens);
bool make_map_codes(CUtensorMap* m, const void* base, long long rows, int box_rows, bool swizzle);

}  // namespace saf3r
