// Attention of a few query rows per sequence over the paged cache (single tokens and short chunks).
//
// Bound by memory: every visible key and value row is read once per kv head and 8 or 16 query rows (the heads of a
// group times the new tokens).  An item is those rows of one sequence and kv head; the items' chunks of 64
// keys, laid end to end, are cut into equal shares, one for each warp, so that unequal lengths and few
// streams keep every SM reading alike.  An item cut by a share's border is finished by a second small kernel.
//
// A warp streams its keys 8 KB at a time (64 keys of 8 bits, 32 of bf16) through two TMA buffers of its own: one is
// in flight while the other is worked on.  The products are transposed, S^T = K Q^T and O^T = V^T P^T: the keys
// are the 16 rows of m16n8k16 and 8 query rows its columns, which halves the work against 16 rows when
// there are 8 or fewer.  The 64 dims may be contracted in any order, and the rows of O^T may be any dims: lane (g, t)
// takes the 16 dims 16t.. of its keys and the 8 dims 8g.. of its values.  Keys g of a group of 16 stand for its keys
// sigma(g), which with the tensor map's swizzle makes every shared load free of bank conflicts.
//
// 8-bit caches: codes become fp16 exactly (one conversion for two) and Q is scaled by a power of
// two per row so that it fits fp16 (its 8 significant bits do, down to 2^-24 of the row's largest).  The page's key
// scale multiplies the fp32 logits.  Its value scale goes into the exponent: with x = s + log2(vs), P = 2^(x - reference)
// is the weight times vs, and the row's sum takes P / vs.
//
// bf16 caches use bf16 products throughout, with the weights in two terms (16 bits): one term alone leaves up to 2^-8 of a row with
// few weights that count, and one token's 16 rows were 0.0023 to 0.0028 off in all, 0.0017 with two, which is the output's
// rounding.  It costs nothing at one token (14.4 us), 0.8% at 4 rows per kv head (64 streams of up to 22,000 keys, 4 kv heads:
// 125 us), 6% at 16 (137 us) and 7% at 64 (276 us).
// The reference is the largest x of the first step; it moves when a later one exceeds it by 2^15
// (fp16 P, which ends 2^-24 below it) or 2^24.
//
// Measured, 64 8-bit streams of 1 to 22,000 keys, 4 kv heads of 4 query heads: 79 us with the join, 70% of the measured copy
// rate.  In its stride a warp's step of 8 KB takes 3,660 cycles with 12 warps an SM, more than that rate;
// the first step ends 12,000 cycles after the start (lengths, page, scales and codes are four loads that wait for one another).  16-row
// products straight from global memory, without the transposition, took 216 us.
#include <cuda.h>

#include "ptx.cuh"
#include "stream.h"
#include "stream_exact.cuh"

namespace saf3r {

namespace {

constexpr int kWarps = 4;              // of a block
constexpr int kBlocksPerSm = 3;        // 64 KB of shared memory and at most 168 registers a thread
constexpr int kMaxRows = 16;
constexpr int kStepBytes = 8192;       // of keys and values
constexpr int kMaxShares = 160 * kBlocksPerSm * kWarps;
constexpr int kCostItem = 1;           // an item's start and end, in chunks
constexpr int kWild = 64;              // largest spread of value scales (in exponents) that a row's fp32 sum is sure to bear
// Exponent of the value scale of a page of zeros (or of values below 2^-91): beside pages of scales 2^kWild larger and more it
// would spread the scales, while its values are less than any weight in fp16 can tell.  There it takes part with a weight of
// zero: its keys count in a row's sum of weights as if its scale were the largest so far.  (Such a page sent its rows key by
// key: one token over 16,384 keys with one such page took 7,520 us instead of 17.)
constexpr int kZeros = -100, kNone = 1000;
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
// an 8 x 8 matrix of 16-bit values across the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// A warp's part of an item that a border cuts: per row the part's answer, log2 of the sum of its weights, and flags.
struct Slot {
  float o[kMaxRows][kD];
  float w[kMaxRows];
  int32_t flags[kMaxRows];  // 1: some streamed key is out of the row's sight, 2: value scales too far apart
};
// The shares that hold an item's first and last chunk (written by those warps).
struct ItemRec {
  int32_t first, last;
};

// Row group rg of a sequence: rows rg * R.. of its (token, group head) rows.
struct Item {
  int b, hk, rg, rows;
  SeqInfo s;
  Runs runs;
  Chunks ch;
  Span first, last;  // what the first and the last row see
};
__device__ __forceinline__ int row_groups(const KvAttnParams& p, const SeqInfo& s, int R) {
  return s.n_new <= 0 ? 0 : (s.n_new * p.group + R - 1) / R;
}
__device__ __forceinline__ Item item_of(const KvAttnParams& p, const SeqInfo& s, int b, int hk, int rg, int R) {
  Item it;
  it.b = b;
  it.hk = hk;
  it.rg = rg;
  it.s = s;
  it.rows = min(R, s.n_new * p.group - rg * R);
  const int pos0 = s.len - s.n_new;
  it.first = span_of(p.win, pos0 + p.by_group.div(rg * R), s.len);
  it.last = span_of(p.win, pos0 + p.by_group.div(rg * R + it.rows - 1), s.len);
  it.runs = runs_of(it.first.lo, it.last.hi, it.last.sink);
  it.ch = chunks_of(it.runs);
  return it;
}
__device__ __forceinline__ long long seq_head_cost(const KvAttnParams& p, const SeqInfo& s, int R) {
  const int n = row_groups(p, s, R);
  long long c = 0;
  for (int rg = 0; rg < n; ++rg) c += item_of(p, s, 0, 0, rg, R).ch.total + kCostItem;
  return c;
}

__device__ __forceinline__ long long item_index(const KvAttnParams& p, int b, int hk, int rg, int R) {
  const int groups = (p.kv.max_new * p.group + R - 1) / R;
  return (static_cast<long long>(b) * p.kv.n_heads + hk) * groups + rg;
}
__device__ __forceinline__ Slot* slots(const KvAttnParams& p) { return reinterpret_cast<Slot*>(p.ws); }
__device__ __forceinline__ ItemRec* recs(const KvAttnParams& p) { return reinterpret_cast<ItemRec*>(p.ws + kMaxShares * 2 * sizeof(Slot)); }

// Walks the pieces of a warp's share.
struct Walk {
  long long x, xs, xe;
  int b, hk, rg;
  SeqInfo s;

  // the next piece: chunks c0 .. c1 - 1 of the item
  __device__ __forceinline__ bool next(const KvAttnParams& p, int R, Item& it, int& c0, int& c1) {
    while (x < xe) {
      while (rg >= row_groups(p, s, R)) {
        rg = 0;
        if (++hk >= p.kv.n_heads || s.n_new <= 0) {
          hk = 0;
          if (++b >= p.kv.n_seqs) return false;
          s = seq_info(p.kv, b);
        }
      }
      it = item_of(p, s, b, hk, rg, R);
      const long long d0 = xs - x, d1 = xe - x;
      c0 = d0 <= 0 ? 0 : (d0 < it.ch.total ? static_cast<int>(d0) : it.ch.total);
      c1 = d1 < it.ch.total ? static_cast<int>(d1) : it.ch.total;
      x += it.ch.total + kCostItem;
      ++rg;
      if (c0 < c1) return true;
    }
    return false;
  }
};

// Finds every warp's share (run by the whole block; each warp gets its own walk).
__device__ __forceinline__ Walk make_walk(const KvAttnParams& p, int R, long long* entries) {
  constexpr int kThreads = 32 * kWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = p.kv.n_seqs;
  const int per = (n + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int b = threadIdx.x * per; b < min(static_cast<int>(threadIdx.x + 1) * per, n); ++b)
    mine += seq_head_cost(p, seq_info(p.kv, b), R);  // of one kv head
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  entries[threadIdx.x] = incl;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += entries[32 * w + 31];
  total *= p.kv.n_heads;
  const int most = gridDim.x * kWarps;
  const int shares = total >= static_cast<long long>(most) * p.least_share ? most : max(1, static_cast<int>(total) / p.least_share);
  // (a 64-bit division takes several times as long)
  const long long each = total >> 31 ? total / shares : static_cast<long long>(static_cast<uint32_t>(total) / static_cast<uint32_t>(shares));
  const int extra = static_cast<int>(total - each * shares);
  auto share_start = [&](int i) { return each * i + min(i, extra); };
  // neighbouring shares go to different SMs: few streams spread over all of them
  const int me = warp * gridDim.x + blockIdx.x;
  Walk w;
  w.b = w.hk = w.rg = 0;
  w.s = SeqInfo{0, 0, 0, false};
  w.xs = me < shares ? share_start(me) : total;
  w.xe = me < shares ? share_start(me + 1) : total;
  w.x = w.xs;
  if (w.xs >= w.xe) return w;
  long long rest = w.xs, head = 0;  // head: cost of the sequence for one kv head
  for (int q = 0; q < kWarps; ++q) {
    const long long in = entries[32 * q + lane];
    const uint32_t hit = __ballot_sync(0xffffffffu, rest < in * p.kv.n_heads);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const long long before = src > 0 ? entries[32 * q + src - 1] : 0;
      w.b = (32 * q + src) * per;
      head = entries[32 * q + src] - before;
      rest -= before * p.kv.n_heads;
      break;
    }
    rest -= entries[32 * q + 31] * p.kv.n_heads;
  }
  w.s = seq_info(p.kv, w.b);
  for (; per > 1; w.s = seq_info(p.kv, ++w.b)) {
    head = seq_head_cost(p, w.s, R);
    if (w.b + 1 >= n || rest < head * p.kv.n_heads) break;
    rest -= head * p.kv.n_heads;
  }
  while (rest >= head && w.hk + 1 < p.kv.n_heads) {
    rest -= head;
    ++w.hk;
  }
  const int groups = row_groups(p, w.s, R);
  while (w.rg + 1 < groups) {
    const int c = item_of(p, w.s, w.b, w.hk, w.rg, R).ch.total + kCostItem;
    if (rest < c) break;
    rest -= c;
    ++w.rg;
  }
  w.x = w.xs - rest;
  return w;
}

__device__ __forceinline__ void store8(const KvAttnParams& p, const Item& it, int row, int R, int col, const float* o) {
  const int i = it.rg * R + row, tok = p.by_group.div(i), head = it.hk * p.group + i - tok * p.group;
  const long long at = (it.s.row0 + tok) * p.out_ts + head * p.out_hs + col;
  if (p.out_fp32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
    d[0] = make_float4(o[0], o[1], o[2], o[3]);
    d[1] = make_float4(o[4], o[5], o[6], o[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) =
        make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
  }
}
template <bool kE4m3>
__device__ __forceinline__ void exact_item_row(const KvAttnParams& p, const Item& it, int row, int R, int lane) {
  const int i = it.rg * R + row, tok = p.by_group.div(i);
  exact_row<kE4m3>(p, it.b, it.s.len, it.s.row0 + tok, it.s.len - it.s.n_new + tok, it.hk * p.group + i - tok * p.group, lane, 0, kD);
}

struct DecodeSmem {
  uint8_t buf[kWarps][2][kStepBytes];
  uint64_t full[kWarps][2];
  long long entries[32 * kWarps];
  int abort;
};

// kB: tiles of 8 query rows.
template <bool kE4m3, int kB>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm)
    decode_kernel(const __grid_constant__ KvAttnParams p, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  constexpr int R = 8 * kB;
  constexpr int kT = kE4m3 ? 64 : 32;     // keys of a step
  constexpr int kG = kT / 16;             // groups of 16 keys
  constexpr int kRowBytes = kE4m3 ? 64 : 128;
  constexpr int kSteps = 64 / kT;         // steps of a chunk
  constexpr float kRaise = kE4m3 ? 15.f : 24.f;
  extern __shared__ uint8_t smem_raw[];
  DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const KvView& kv = p.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kWarps; ++w) {
      mbar_init(&sm.full[w][0], 1);
      mbar_init(&sm.full[w][1], 1);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  Walk walk = make_walk(p, R, sm.entries);  // (syncs the block)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  uint64_t* full = sm.full[warp];
  uint32_t issued = 0, used = 0;
  bool ok = true;
  // sigma(m): the key of its group of 16 that row m of the products stands for
  auto sigma = [](int m) { return m ^ ((m >> 1) & 1); };
  Item it;
  int c0, c1;
  const int me = warp * gridDim.x + blockIdx.x;
  while (ok && walk.next(p, R, it, c0, c1)) {
    if (lane == 0) {
      ItemRec* rec = recs(p) + item_index(p, it.b, it.hk, it.rg, R);
      if (c0 == 0) rec->first = me;
      if (c1 == it.ch.total) rec->last = me;
    }
    const int n_steps = (c1 - c0) * kSteps;
    const int32_t* table = kv.table + static_cast<long long>(it.b) * kv.max_pages;
    auto step_key = [&](int i) { return it.ch.key(c0 + i / kSteps) + (i % kSteps) * kT; };
    auto seen = [&](int j) { return j < it.runs.b_end && (j >= it.runs.b_begin || j < it.runs.a_end); };
    // this lane's box of step i: its first key, -1 where there is none to read
    auto box_key = [&](int i) {
      if (lane >= (kT >> p.box_log2) || i >= n_steps) return -1;
      const int j = step_key(i) + (lane << p.box_log2);
      return j < it.runs.b_end && (j + (1 << p.box_log2) > it.runs.b_begin || j < it.runs.a_end) ? j : -1;
    };
    auto box_entry = [&](int i) {
      const int j = box_key(i);
      return j >= 0 ? table[j >> kv.page_log2] : 0;
    };
    // copies step i, whose page entry is `entry`; returns the scales of this lane's box
    auto issue = [&](int i, int entry) {
      const int j = box_key(i);
      int row = -1;
      float2 scale = make_float2(1.f, 0.f);  // a box that is not read has no value scale
      if (j >= 0) {
        if (entry < 0 || entry >= kv.n_pages) {
          atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
        } else {
          const int at = entry * kv.n_heads + it.hk;
          row = (at << kv.page_log2) + (j & (kv.page - 1));
          if (kE4m3) scale = make_float2(kv.k_scale[at], kv.v_scale[at]);
        }
      }
      if (i < n_steps) {
        uint64_t* bar = &full[issued & 1];
        uint8_t* dst = sm.buf[warp][issued & 1];
        const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
        if (lane == 0) mbar_arrive_expect_tx(bar, ((2 * __popc(have)) << p.box_log2) * kRowBytes);
        __syncwarp();
        if (row >= 0) {
          uint8_t* d = dst + (lane << p.box_log2) * kRowBytes;
          tma_load_3d(d, &map_k, 0, row, 0, bar);
          tma_load_3d(d + kStepBytes / 2, &map_v, 0, row, 0, bar);
        }
        __syncwarp();
        ++issued;
      }
      return scale;
    };
    float2 sc0 = issue(0, box_entry(0));
    float2 sc1 = issue(1, box_entry(1));
    int entry = box_entry(2);

    // Q^T fragments: query row g of each tile, dims 16t..16t+15
    uint32_t qb[kB][4][2];
    float qs[kB][2];  // of rows 2t and 2t + 1: what a logit is multiplied by
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int r = 8 * b + g;
      uint4 u = make_uint4(0, 0, 0, 0), w = u;
      if (r < it.rows) {
        const int a = it.rg * R + r, tok = p.by_group.div(a);
        const uint4* q = reinterpret_cast<const uint4*>(p.q + (it.s.row0 + tok) * p.q_ts +
                                                        (it.hk * p.group + a - tok * p.group) * p.q_hs + 16 * t);
        u = q[0];
        w = q[1];
      }
      uint32_t v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
      float mine = kLog2Scale;
      if (kE4m3) {
        // the row's largest exponent; then every value times 2^-e, as fp16
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = max(mx, max((v[j] >> 7) & 0xffu, (v[j] >> 23) & 0xffu));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = mx == 0xff ? 0 : min(max(static_cast<int>(mx) - 127, -120), 120);  // an infinity or NaN stays one
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        mine = kLog2Scale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = pack_f16x2(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xffff0000u) * f);
      }
      qs[b][0] = __shfl_sync(0xffffffffu, mine, 8 * t);
      qs[b][1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        qb[b][kk][0] = v[2 * kk];
        qb[b][kk][1] = v[2 * kk + 1];
      }
    }

    float o[kB][4][4];
    float ref[kB][2], l[kB][2];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      ref[b][0] = ref[b][1] = -INFINITY;
      l[b][0] = l[b][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.f;
    }
    // bf16: a weight's second term may be 0 or negative, which an infinite value in sight does not bear
    bool part = !kE4m3, unset = true;
    int lv_lo = kNone, lv_hi = -kNone;  // exponents of the value scales so far, those of pages of zeros left out

    bool zeros_first = false;  // pages of zeros came before any other
    // What was summed over pages of zeros, as if their scale were 2^e: the references grow by e - kZeros.
    auto to_scale = [&](int e) {
      const float f = power_of_two(-e), f0 = power_of_two(kZeros);  // one factor alone could leave fp32's range
#pragma unroll
      for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          ref[b][c] += static_cast<float>(e - kZeros);
          l[b][c] = l[b][c] * f0 * f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[b][i][c] = o[b][i][c] * f0 * f;
            o[b][i][2 + c] = o[b][i][2 + c] * f0 * f;
          }
        }
    };

    for (int st = 0; st < n_steps; ++st) {
      const int j0 = step_key(st);
      const uint32_t slot = used & 1;
      // the scales of the groups of 16 keys
      float ks[kG], lv[kG], vi[kG];
      uint32_t drop = 0;  // groups whose values are nothing beside the others'
      if constexpr (kE4m3) {
        int e[kG];
        const int hi0 = lv_hi;
        bool zeros = false;
#pragma unroll
        for (int i = 0; i < kG; ++i) {
          const int src = (16 * i) >> p.box_log2;
          ks[i] = __shfl_sync(0xffffffffu, sc0.x, src);
          e[i] = static_cast<int>((__float_as_uint(__shfl_sync(0xffffffffu, sc0.y, src)) >> 23) & 0xffu) - 127;
          zeros |= e[i] == kZeros;
          if (e[i] > kZeros) {
            lv_lo = min(lv_lo, e[i]);
            lv_hi = max(lv_hi, e[i]);
          }
        }
        if (hi0 == -kNone && zeros_first && lv_hi > kZeros + kWild) to_scale(lv_hi);
        zeros_first |= zeros && lv_hi == -kNone;
#pragma unroll
        for (int i = 0; i < kG; ++i) {
          if (e[i] == kZeros && lv_hi > kZeros + kWild) {
            e[i] = lv_hi;
            drop |= 1u << i;
          }
          if (e[i] < kZeros) e[i] = 0;  // not read
          lv[i] = static_cast<float>(e[i]);
          vi[i] = power_of_two(-e[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kG; ++i) {
          ks[i] = vi[i] = 1.f;
          lv[i] = 0.f;
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], (used >> 1) & 1, &sm.abort, kv.err, p.wait_budget, SAF3R_ERR_TIMEOUT));
      if (!ok) break;
      const uint8_t* kb = sm.buf[warp][slot];
      const uint8_t* vb = kb + kStepBytes / 2;
      const bool whole = (j0 >= it.last.lo && j0 + kT <= it.first.hi) || j0 + kT <= it.first.sink;  // every row sees every key
      part |= !whole;

      // S^T: keys sigma(g), sigma(g + 8) of each group; query rows 2t, 2t + 1 of each tile
      float s[kB][kG][4];
#pragma unroll
      for (int i = 0; i < kG; ++i) {
#pragma unroll
        for (int b = 0; b < kB; ++b) s[b][i][0] = s[b][i][1] = s[b][i][2] = s[b][i][3] = 0.f;
        const int r0 = 16 * i + sigma(g), r1 = r0 + 8;
        if (kE4m3) {
          const uint4 x = *reinterpret_cast<const uint4*>(kb + r0 * 64 + ((t ^ ((r0 >> 1) & 3)) << 4));
          const uint4 y = *reinterpret_cast<const uint4*>(kb + r1 * 64 + ((t ^ ((r1 >> 1) & 3)) << 4));
          const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t a[4] = {f16x2_of_e4m3(wx[kk]), f16x2_of_e4m3(wy[kk]), f16x2_of_e4m3(wx[kk] >> 16), f16x2_of_e4m3(wy[kk] >> 16)};
#pragma unroll
            for (int b = 0; b < kB; ++b) mma_f16(s[b][i], a, qb[b][kk][0], qb[b][kk][1]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(kb + r0 * 128 + (((2 * t + c) ^ (r0 & 7)) << 4));
            const uint4 y = *reinterpret_cast<const uint4*>(kb + r1 * 128 + (((2 * t + c) ^ (r1 & 7)) << 4));
            const uint32_t a[4] = {x.x, y.x, x.y, y.y}, a2[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
            for (int b = 0; b < kB; ++b) {
              mma_bf16(s[b][i], a, qb[b][2 * c][0], qb[b][2 * c][1]);
              mma_bf16(s[b][i], a2, qb[b][2 * c + 1][0], qb[b][2 * c + 1][1]);
            }
          }
        }
      }
      // to logits in units of log2 (times the value scale)
#pragma unroll
      for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int i = 0; i < kG; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[b][i][c] = fmaf(s[b][i][c], qs[b][c & 1] * ks[i], lv[i]);
      if (!whole) {
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = it.rg * R + min(8 * b + 2 * t + c, it.rows - 1);
            const Span sp = span_of(p.win, it.s.len - it.s.n_new + p.by_group.div(r), it.s.len);
#pragma unroll
            for (int i = 0; i < kG; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int j = j0 + 16 * i + sigma(g) + 8 * h;
                if (!((j >= sp.lo && j < sp.hi) || j < sp.sink)) s[b][i][2 * h + c] = -INFINITY;
              }
          }
      }
      // the reference moves on the first step, and where a logit is far above it
      bool raise = unset;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < kG; ++i) mx[c] = max3f(mx[c], s[b][i][c], s[b][i][2 + c]);
        raise |= mx[0] > ref[b][0] + kRaise || mx[1] > ref[b][1] + kRaise;
      }
      if (__any_sync(0xffffffffu, raise)) {
        unset = false;
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = ref[b][c];
#pragma unroll
            for (int i = 0; i < kG; ++i) mx = max3f(mx, s[b][i][c], s[b][i][2 + c]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float f = mx == ref[b][c] ? 1.f : fast_exp2(ref[b][c] - mx);  // from -inf: 0
            ref[b][c] = mx;
            unset |= mx == -INFINITY;
            l[b][c] *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[b][i][c] *= f;
              o[b][i][2 + c] *= f;
            }
          }
        unset = __any_sync(0xffffffffu, unset);
      }
      // P^T fragments; bf16: what the rounding left, as a second term
      uint32_t pb[kB][kG][2], pl[kE4m3 ? 1 : kB][kE4m3 ? 1 : kG][2];
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const float u0 = ref[b][0] == -INFINITY ? 0.f : ref[b][0], u1 = ref[b][1] == -INFINITY ? 0.f : ref[b][1];
#pragma unroll
        for (int i = 0; i < kG; ++i) {
          const float e0 = fast_exp2(s[b][i][0] - u0), e1 = fast_exp2(s[b][i][1] - u1);
          const float e2 = fast_exp2(s[b][i][2] - u0), e3 = fast_exp2(s[b][i][3] - u1);
          l[b][0] = fmaf(e0 + e2, vi[i], l[b][0]);
          l[b][1] = fmaf(e1 + e3, vi[i], l[b][1]);
          uint32_t x = kE4m3 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
          uint32_t y = kE4m3 ? pack_f16x2(e2, e3) : pack_bf16x2(e2, e3);
          if (kE4m3 && ((drop >> i) & 1u)) x = y = 0u;  // not the values: one that is not a number stays one
          pb[b][i][0] = transpose8(x);
          pb[b][i][1] = transpose8(y);
          if constexpr (!kE4m3) {
            pl[b][i][0] = transpose8(pack_bf16x2(e0 - bf16_lo(x), e1 - bf16_hi(x)));
            pl[b][i][1] = transpose8(pack_bf16x2(e2 - bf16_lo(y), e3 - bf16_hi(y)));
          }
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        // value rows of the keys 2t, 2t + 1, 2t + 8, 2t + 9 of the group's order
        uint32_t v[4][kE4m3 ? 2 : 4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = 16 * i + sigma(2 * t + (c & 1)) + 8 * (c >> 1);
          if (kE4m3) {
            const uint2 x = *reinterpret_cast<const uint2*>(vb + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
            v[c][0] = x.x;
            v[c][1] = x.y;
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(vb + r * 128 + ((g ^ (r & 7)) << 4));
            v[c][0] = x.x;
            v[c][1] = x.y;
            v[c][kE4m3 ? 0 : 2] = x.z;
            v[c][kE4m3 ? 1 : 3] = x.w;
          }
          if (!whole && !seen(j0 + r)) {  // what no row sees need not be finite
#pragma unroll
            for (int w = 0; w < (kE4m3 ? 2 : 4); ++w) v[c][w] = 0u;
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {  // dims 8g + 2m and 8g + 2m + 1
          uint32_t a[4];
          if (kE4m3) {
            const uint32_t sel = (m & 1) ? 0x7362 : 0x5140;
            const uint32_t x = __byte_perm(v[0][m >> 1], v[1][m >> 1], sel), y = __byte_perm(v[2][m >> 1], v[3][m >> 1], sel);
            a[0] = f16x2_of_e4m3(x);
            a[1] = f16x2_of_e4m3(x >> 16);
            a[2] = f16x2_of_e4m3(y);
            a[3] = f16x2_of_e4m3(y >> 16);
          } else {
            const int w = kE4m3 ? 0 : m;
            a[0] = __byte_perm(v[0][w], v[1][w], 0x5410);
            a[1] = __byte_perm(v[0][w], v[1][w], 0x7632);
            a[2] = __byte_perm(v[2][w], v[3][w], 0x5410);
            a[3] = __byte_perm(v[2][w], v[3][w], 0x7632);
          }
#pragma unroll
          for (int b = 0; b < kB; ++b) {
            if constexpr (kE4m3) {
              mma_f16(o[b][m], a, pb[b][i][0], pb[b][i][1]);
            } else {
              mma_bf16(o[b][m], a, pb[b][i][0], pb[b][i][1]);
              mma_bf16(o[b][m], a, pl[b][i][0], pl[b][i][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the buffer
      ++used;
      sc0 = sc1;
      sc1 = issue(st + 2, entry);
      entry = box_entry(st + 3);
    }
    if (!ok) break;

    const bool wild = kE4m3 && lv_hi - lv_lo > kWild;
    const bool only = c0 == 0 && c1 == it.ch.total;
    Slot* sl = nullptr;
    if (!only) sl = slots(p) + 2LL * me + (c0 > 0 ? 0 : 1);
#pragma unroll
    for (int b = 0; b < kB; ++b)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[b][c];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float inv = sum == 0.f ? (only ? no_weight() : 0.f) : 1.f / sum;
        float x[8];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = o[b][i >> 1][c + 2 * (i & 1)] * inv;
          bad |= !(fabsf(x[i]) <= 3.402823466e+38f);
        }
        const int row = 8 * b + 2 * t + c;
        const bool live = row < it.rows;
        if (only) {
          const uint32_t todo = __ballot_sync(0xffffffffu, live && ((bad && part) || wild));
          if (live && !(todo & (0x11111111u << t))) store8(p, it, row, R, 8 * g, x);
          for (int q = 0; q < 4; ++q)
            if (todo & (0x11111111u << q)) exact_item_row<kE4m3>(p, it, 8 * b + 2 * q + c, R, lane);
        } else if (live) {
          float4* d = reinterpret_cast<float4*>(&sl->o[row][8 * g]);
          d[0] = make_float4(x[0], x[1], x[2], x[3]);
          d[1] = make_float4(x[4], x[5], x[6], x[7]);
          if (g == 0) {
            sl->w[row] = sum == 0.f ? -INFINITY : ref[b][c] + log2f(sum);
            sl->flags[row] = (part ? 1 : 0) | (wild ? 2 : 0);
          }
        }
      }
  }
  // copies that a wait gave up on land before the block exits
  for (; used < issued; ++used) mbar_wait_drain(&full[used & 1], (used >> 1) & 1, kDrainBudget);
}

// Joins the parts of one item (block x: its kv head and row group, y: its sequence).  Few rows get several warps each, which
// take parts in turn: their weights first, then 2 columns a lane, in a fixed order.
constexpr int kJoinWarps = 8;
template <bool kE4m3, int kB>
__global__ void __launch_bounds__(32 * kJoinWarps) decode_join_kernel(const __grid_constant__ KvAttnParams p) {
  constexpr int R = 8 * kB;
  __shared__ float s_a[kJoinWarps][kD], s_big[kJoinWarps], s_sum[kJoinWarps];
  __shared__ int s_flags[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = gridDim.x / p.kv.n_heads, hk = blockIdx.x / groups, rg = blockIdx.x - hk * groups;
  const SeqInfo s = seq_info(p.kv, blockIdx.y);  // the call's input: the first kernel does not write it
  const int rows = min(R, s.n_new * p.group - rg * R);
  if (rows <= 0) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const ItemRec rec = recs(p)[item_index(p, blockIdx.y, hk, rg, R)];
  const int i0 = rec.first, i1 = rec.last;
  if (i0 == i1 || i0 < 0 || i1 >= kMaxShares) return;  // one warp had the whole item (or, after a wait that gave up, none)
  const int turn = rows > 4 ? 1 : rows > 2 ? 2 : rows > 1 ? 4 : 8;  // warps of a row
  const int at0 = warp & (turn - 1);
  const Slot* base = slots(p);
  auto slot = [&](int i) -> const Slot& { return base[2LL * i + (i == i0 ? 1 : 0)]; };
  for (int row = warp / turn; row < rows; row += kJoinWarps / turn) {
    float big = -INFINITY, sum = 0.f, a0 = 0.f, a1 = 0.f;
    int flags = 0;
    for (int i = i0 + at0; i <= i1; i += 32 * turn) {  // 32 parts at a time
      float w = -INFINITY;
      const int mine = i + lane * turn;
      if (mine <= i1) {
        w = slot(mine).w[row];
        flags |= slot(mine).flags[row];
      }
      float now = w;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
      now = fmaxf(now, big);
      const float f = big == now ? 1.f : fast_exp2(big - now);  // from -inf: 0
      big = now;
      sum *= f;
      a0 *= f;
      a1 *= f;
      w = w == -INFINITY ? 0.f : fast_exp2(w - big);
      const int n = min(32, (i1 - i) / turn + 1);
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const float2 x = reinterpret_cast<const float2*>(slot(i + k * turn).o[row])[lane];
        sum += wk;
        a0 += wk * x.x;
        a1 += wk * x.y;
      }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (turn > 1) {  // every warp of the block has one row then
      s_a[warp][2 * lane] = a0;
      s_a[warp][2 * lane + 1] = a1;
      if (lane == 0) {
        s_big[warp] = big;
        s_sum[warp] = sum;
        s_flags[warp] = flags;
      }
    }
    if (turn > 1) {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / turn), "r"(32 * turn) : "memory");  // the row's warps
      if (at0 > 0) return;
      for (int q = 1; q < turn; ++q) big = fmaxf(big, s_big[warp + q]);
      sum = a0 = a1 = 0.f;
      for (int q = 0; q < turn; ++q) {
        const float f = s_big[warp + q] == -INFINITY ? 0.f : fast_exp2(s_big[warp + q] - big);
        sum += f * s_sum[warp + q];
        a0 += f * s_a[warp + q][2 * lane];
        a1 += f * s_a[warp + q][2 * lane + 1];
        flags |= s_flags[warp + q];
      }
    }
    const float inv = sum == 0.f ? no_weight() : 1.f / sum;
    a0 *= inv;
    a1 *= inv;
    const bool bad = !(fabsf(a0) <= 3.402823466e+38f && fabsf(a1) <= 3.402823466e+38f);
    const int at_row = rg * R + row, tok = p.by_group.div(at_row), head = hk * p.group + at_row - tok * p.group;
    bool exact = (flags & 2) != 0;
    if (!exact && __any_sync(0xffffffffu, bad)) {
      // a value out of sight is not finite; or no part holds a NaN: the sum left fp32's range
      bool nan = false;
      for (int i = i0; i <= i1; ++i) {
        const float2 x = reinterpret_cast<const float2*>(slot(i).o[row])[lane];
        nan |= x.x != x.x || x.y != x.y;
      }
      exact = (flags & 1) || !__any_sync(0xffffffffu, nan);
    }
    if (exact) {
      exact_row<kE4m3>(p, blockIdx.y, s.len, s.row0 + tok, s.len - s.n_new + tok, head, lane, 0, kD);
      continue;
    }
    const long long at = (s.row0 + tok) * p.out_ts + head * p.out_hs + 2 * lane;
    if (p.out_fp32)
      *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(a0, a1);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at) = pack_bf16x2(a0, a1);
  }
}

int tile_rows(int max_new, int group) { return static_cast<long long>(max_new) * group <= 8 ? 8 : 16; }

}  // namespace

// Rows per sequence and kv head that this kernel takes.  It streams the keys once for every 16 rows, the tensor-core kernel once
// for 256.  Measured, us, here and there:
//   rows                                        17           32           48           64
//   8-bit, 4 sequences, 12,000 keys, 16 heads   76 / 79      79 / 79      99 / 79      121 / 79
//   8-bit, 8 sequences, 4,096 keys, 4 heads     34 / 33      35 / 33      40 / 33      42 / 33
//   bf16, 4 sequences, 12,000 keys, 16 heads    83 / 66      87 / 66      91 / 66      115 / 66
//   bf16, 8 sequences, 4,096 keys, 4 heads      31 / 29      32 / 29      34 / 29      36 / 29
// Up to 16 rows the other one has a tile of 128 rows for them.  From 17 to 64 rows bf16 stays here for its 16 bits of a weight
// against 8, which callers of short chunks rely on; 8-bit rows stay with it, up to 32 at no cost.  The rule goes by the step's
// longest sequence: a chunk among single tokens takes all of them there (64 sequences of 1,400 to 23,000 keys, 4 heads of 4, one
// with 1,374 new tokens: 8-bit 121 us against 41 for the chunk and 35 for the others alone, bf16 87 against 32 and 49).
bool decode_takes(int max_new, int group) { return static_cast<long long>(max_new) * group <= 64; }

size_t decode_workspace_bytes(const KvView& kv, int group) {
  const int R = tile_rows(kv.max_new, group);
  const size_t items = static_cast<size_t>(kv.n_seqs) * kv.n_heads * ((static_cast<size_t>(kv.max_new) * group + R - 1) / R);
  return kMaxShares * 2 * sizeof(Slot) + items * sizeof(ItemRec);
}

saf3r_status launch_decode(const KvAttnParams& p0, cudaStream_t stream, int* n_launch) {
  KvAttnParams p = p0;
  const KvView& kv = p.kv;
  const int keys = p.e4m3 ? 64 : 32, box = kv.page < keys ? kv.page : keys;
  p.box_log2 = box == 16 ? 4 : box == 32 ? 5 : 6;
  p.least_share = p.e4m3 ? 2 : 1;  // two steps: both of a warp's buffers
  const long long rows = static_cast<long long>(kv.n_pages) * kv.n_heads * kv.page;
  CUtensorMap mk, mv;
  if (!(p.e4m3 ? make_map_codes(&mk, kv.k, rows, box, true) && make_map_codes(&mv, kv.v, rows, box, true)
               : make_map_rows(&mk, kv.k, rows, kD, 1, rows * kD, box) && make_map_rows(&mv, kv.v, rows, kD, 1, rows * kD, box)))
    return SAF3R_ERR_CUDA;
  const bool wide = tile_rows(kv.max_new, p.group) == 16;
  const auto kernel = p.e4m3 ? (wide ? decode_kernel<true, 2> : decode_kernel<true, 1>) : (wide ? decode_kernel<false, 2> : decode_kernel<false, 1>);
  const int smem = static_cast<int>(sizeof(DecodeSmem) + 1024);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return SAF3R_ERR_CUDA;
  const int grid = (p.num_sms < 160 ? p.num_sms : 160) * kBlocksPerSm;
  kernel<<<grid, 32 * kWarps, smem, stream>>>(p, mk, mv);
  ++*n_launch;
  if (cudaGetLastError() != cudaSuccess) return SAF3R_ERR_CUDA;
  const int R = wide ? 16 : 8;
  const auto join = p.e4m3 ? (wide ? decode_join_kernel<true, 2> : decode_join_kernel<true, 1>)
                           : (wide ? decode_join_kernel<false, 2> : decode_join_kernel<false, 1>);
  const dim3 items(kv.n_heads * ((kv.max_new * p.group + R - 1) / R), kv.n_seqs);
  if (launch_behind(join, items, dim3(32 * kJoinWarps), stream, p) != cudaSuccess) return SAF3R_ERR_CUDA;
  ++*n_launch;
  return SAF3R_OK;
}

}  // namespace saf3r
