// Attention over the paged cache, or over keys and values held at once, for many query rows: the
// tensor-core kernel of the streaming operators (tcgen05, sm_100a).
//
// An item is 256 rows of one kv head (its group's heads times new tokens, token after token) of one sequence: two
// 128-row tiles.  The keys that some row of the item sees (Runs) are streamed 128 at a time, as two
// chunks of 64.  The items' key blocks, laid end to end, are cut into equal shares, one CTA each: an item
// cut by a share's border is finished by the join kernel from its pieces' unnormalised sums.  Equal shares
// keep every SM busy with few items (one view of one stream: 96 items of unequal length on 148 SMs).
//
// Warps (20):
//   0-2    loaders: copy (bf16) or convert (8-bit) each block's K and V rows into a ring of kStages stages, in the
//          128-byte-swizzled layout that the tensor core reads.  Rows that no row of the item sees are zero, so
//          what lies behind a sequence's end or in another's page never enters.  An 8-bit code times its page's
//          power-of-two scale is a bf16 value exactly (4 significant bits, the exponent within bf16's), so the products
//          are the bf16 ones in both cases.
//   4-19   softmax: four warpgroups, one for each tile and key half; a thread has one row's 64 keys of a block.
//          Sixteen warps, four for each scheduler in different steps of two tiles, hide each other's waits.
//   3      issues the products.
// Tensor memory (512 columns): for each tile S (128 fp32 columns; each half's bf16 P goes over the first 32 columns of
// its half once read) and an accumulator O for each key half (64 columns).  The halves have a running
// maximum and sum of their own and meet when the piece ends.
//
// A row's reference maximum moves only when a block exceeds it by 2^8: bf16 P and the fp32 sums
// keep their relative precision at any reference, so the answer does not depend on it.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ptx.cuh"
#include "stream.h"
#include "stream_exact.cuh"

namespace saf3r {

namespace {

constexpr int kLoaders = 3;            // warps
constexpr int kThreads = 640;
constexpr int kStages = 3;
constexpr int kRaw = 3;
constexpr int kItem = 256;             // rows of an item
constexpr int kRowBytes = 128;
constexpr int kBlockBytes = 128 * kRowBytes;  // 128 rows x 64 bf16
constexpr float kScaleLog2 = 0.18033688011112042f;  // log2(e) / sqrt(64)
constexpr float kGrow = 8.0f;
constexpr int kMaxShares = 160;        // CTAs of a launch at most (one for each SM)
constexpr int kPlanEntries = 1024;
// Cost of a key block and of an item's start and end, in eighths of a two-tile block.
constexpr int kCost2 = 8, kCost1 = 5, kCostItem = 8;
constexpr int kLeastShare = 4 * kCost2;  // shares smaller than this are not worth a CTA

// Pairs (of the 32 of a row's 64 keys) whose exponentials run on the FMA pipe.
constexpr uint32_t kPolyPairs = 0x88888888u;
// p(f) = 1 + f (c1 + f (c2 + f c3)), fitted to 2^f on [0, 1) for least maximum relative error (8.6e-5)
constexpr float kExpC1 = 0.6951168179512024f, kExpC2 = 0.22764486074447632f, kExpC3 = 0.07706713676452637f;

// A share's unfinished item: per row the sum of weights times values, their sum and reference maximum.
struct Slot {
  float o[kItem][kD];
  float m[kItem], l[kItem];
  int32_t part[kItem];  // nonzero: some streamed key is out of the row's sight
};
static_assert(sizeof(Slot) % 16 == 0, "slots stay aligned");

// An item whose first cut is the start of share i.
struct Cut {
  int32_t valid, b, hk, row0, rows;
  int32_t first, n_new, len;  // the sequence
  int32_t nblk, unit, shares;
  int32_t pad;
  long long x0, total;
};

struct Work {
  Cut cuts[kMaxShares];
  Slot slots[kMaxShares][2];  // [0]: an item begun by an earlier share, [1]: one that a later share ends
};

struct Piece {
  int b, hk, row0, rows;  // rows row0 .. row0 + rows - 1 of the sequence's (token, group head) rows
  SeqInfo s;
  Runs runs;
  Chunks ch;
  int blk0, blk1;         // key blocks of 128
  int slot;               // -1: the whole item
};

struct Tile {
  int rows, nblk, unit;
  long long cost;
  Runs runs;
  Chunks ch;
};

__device__ __forceinline__ Tile tile_of(const KvAttnParams& p, const SeqInfo& s, int i) {
  Tile t;
  const int r0 = i * kItem;
  t.rows = min(kItem, s.n_new * p.group - r0);
  const int start = s.len - s.n_new;
  const Span a = span_of(p.win, start + r0 / p.group, s.len);
  const Span z = span_of(p.win, start + (r0 + t.rows - 1) / p.group, s.len);
  t.runs = runs_of(a.lo, z.hi, z.sink);
  t.ch = chunks_of(t.runs);
  t.nblk = (t.ch.total + 1) >> 1;
  t.unit = t.rows > 128 ? kCost2 : kCost1;
  t.cost = static_cast<long long>(t.nblk) * t.unit + kCostItem;
  return t;
}

__device__ __forceinline__ int tiles_of(const KvAttnParams& p, const SeqInfo& s) {
  return s.n_new <= 0 ? 0 : (s.n_new * p.group + kItem - 1) / kItem;
}

// Blocks of an item that lie before distance d from its start.
__device__ __forceinline__ int blocks_before(long long d, int nblk, int unit) {
  if (d <= 0) return 0;
  const long long n = (d + unit - 1) / unit;
  return n < nblk ? static_cast<int>(n) : nblk;
}

// This CTA's share: its range of the line of all items, and the item that holds its start.
struct Plan {
  long long xs, xe, x;  // range; start of the first item
  int hk, b, tile;
  int shares;
};

struct AttnSmem {
  uint8_t q[2][2][kBlockBytes];
  uint8_t kv[kStages][2 * kBlockBytes];  // 128 rows of K, then of V
  uint8_t raw[kRaw][kBlockBytes];        // 8-bit caches: 128 rows of 64 codes of K, then of V
  uint64_t full[kStages], empty[kStages];
  uint64_t q_empty[2];
  uint64_t s_full[2], o_done[2], p_full[2][2];
  uint64_t drain;
  uint64_t pair[2][4];                // the two warps of a tile's 32 rows meet here
  float stats[2][2][2][128][2];       // [piece parity][tile][half][row] = (maximum, sum)
  Plan plan;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Cost of a sequence's tiles for one kv head (run by a warp).
__device__ __forceinline__ long long seq_cost(const KvAttnParams& p, int b, int lane) {
  const SeqInfo s = seq_info(p.kv, b);
  const int n = tiles_of(p, s);
  long long c = 0;
  for (int i = lane; i < n; i += 32) c += tile_of(p, s, i).cost;
  return warp_sum(c);
}

// Finds this CTA's share (run by all threads; `entries` is scratch in shared memory).
__device__ void make_plan(const KvAttnParams& p, Plan& plan, long long* entries) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.kv.n_seqs + kPlanEntries - 1) / kPlanEntries;
  const int n = (p.kv.n_seqs + per - 1) / per;
  for (int e = warp; e < n; e += kThreads / 32) {
    long long c = 0;
    for (int b = e * per; b < min((e + 1) * per, p.kv.n_seqs); ++b) c += seq_cost(p, b, lane);
    if (lane == 0) entries[e] = c;
  }
  __syncthreads();
  if (warp != 0) return;
  long long mine = 0;
  for (int e = lane; e < n; e += 32) mine += entries[e];
  const long long head = warp_sum(mine);  // of one kv head
  const long long total = head * p.kv.n_heads;
  const long long most = total / kLeastShare;
  const int shares = most < 1 ? 1 : (most < gridDim.x ? static_cast<int>(most) : gridDim.x);
  const int me = blockIdx.x;
  Plan pl;
  pl.shares = shares;
  pl.xs = total * me / shares;
  pl.xe = me < shares ? total * (me + 1) / shares : pl.xs;
  pl.x = pl.xs;
  pl.hk = pl.b = pl.tile = 0;
  Cut cut{};
  if (pl.xs < pl.xe) {
    pl.hk = static_cast<int>(pl.xs / head);
    long long rest = pl.xs - pl.hk * head;  // inside the head
    int e = 0;
    for (int e0 = 0;; e0 += 32) {
      const long long c = e0 + lane < n ? entries[e0 + lane] : 0;
      long long incl = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, rest < incl);
      if (hit) {
        const int src = __ffs(hit) - 1;
        e = e0 + src;
        rest -= __shfl_sync(0xffffffffu, incl - c, src);
        break;
      }
      rest -= __shfl_sync(0xffffffffu, incl, 31);
      if (e0 + 32 >= n) break;  // not reached: rest < head
    }
    int b = e * per;
    for (; b + 1 < p.kv.n_seqs; ++b) {
      const long long c = seq_cost(p, b, lane);
      if (rest < c) break;
      rest -= c;
    }
    const SeqInfo s = seq_info(p.kv, b);
    const int nt = tiles_of(p, s);
    for (int t0 = 0; t0 < nt; t0 += 32) {
      const long long c = t0 + lane < nt ? tile_of(p, s, t0 + lane).cost : 0;
      long long incl = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, rest < incl);
      if (hit) {
        const int src = __ffs(hit) - 1;
        pl.tile = t0 + src;
        rest -= __shfl_sync(0xffffffffu, incl - c, src);
        break;
      }
      rest -= __shfl_sync(0xffffffffu, incl, 31);
    }
    pl.b = b;
    pl.x = pl.xs - rest;
    const Tile t = tile_of(p, s, pl.tile);
    const int cutblk = blocks_before(rest, t.nblk, t.unit);
    const long long before = me > 0 ? total * (me - 1) / shares : 0;
    cut.valid = me > 0 && cutblk > 0 && cutblk < t.nblk && blocks_before(before - pl.x, t.nblk, t.unit) == 0;
    cut.b = b;
    cut.hk = pl.hk;
    cut.row0 = pl.tile * kItem;
    cut.rows = t.rows;
    cut.first = s.row0;
    cut.n_new = s.n_new;
    cut.len = s.len;
    cut.nblk = t.nblk;
    cut.unit = t.unit;
    cut.shares = shares;
    cut.x0 = pl.x;
    cut.total = total;
  }
  if (lane == 0) {
    plan = pl;
    reinterpret_cast<Work*>(p.ws)->cuts[me] = cut;
  }
}

// Walks the pieces of this CTA's share; every role walks for itself.
struct Walk {
  long long x, xs, xe;
  int hk, b, tile;
  SeqInfo s;

  __device__ __forceinline__ Walk(const KvAttnParams& p, const Plan& pl)
      : x(pl.x), xs(pl.xs), xe(pl.xe), hk(pl.hk), b(pl.b), tile(pl.tile) {
    if (xs < xe) s = seq_info(p.kv, b);
  }
  __device__ __forceinline__ bool next(const KvAttnParams& p, Piece& pc) {
    while (x < xe) {
      while (tile >= tiles_of(p, s)) {
        tile = 0;
        if (++b == p.kv.n_seqs) {
          b = 0;
          if (++hk == p.kv.n_heads) return false;
        }
        s = seq_info(p.kv, b);
      }
      const Tile t = tile_of(p, s, tile);
      const int b0 = blocks_before(xs - x, t.nblk, t.unit), b1 = blocks_before(xe - x, t.nblk, t.unit);
      const int row0 = tile * kItem;
      x += t.cost;
      ++tile;
      if (b0 < b1) {
        pc.b = b;
        pc.hk = hk;
        pc.row0 = row0;
        pc.rows = t.rows;
        pc.s = s;
        pc.runs = t.runs;
        pc.ch = t.ch;
        pc.blk0 = b0;
        pc.blk1 = b1;
        pc.slot = b0 > 0 ? 0 : (b1 < t.nblk ? 1 : -1);
        return true;
      }
    }
    return false;
  }
};

__device__ __forceinline__ bool wait_all(const KvAttnParams& p, AttnSmem& sm, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, &sm.abort, p.kv.err, p.wait_budget, SAF3R_ERR_TIMEOUT));
}

// ------------------------------------------------------------------ loaders

// First row in the pools (or in ck, cv) of the 16 keys from key j of the piece, -1: none of them is read.
__device__ __forceinline__ int group_row(const KvAttnParams& p, const Piece& pc, int j) {
  if (!(j < pc.runs.b_end && (j + 16 > pc.runs.b_begin || j < pc.runs.a_end))) return -1;
  const KvView& kv = p.kv;
  if (p.ck) return pc.hk * kv.n_tokens + j;
  const int id = kv.table[static_cast<long long>(pc.b) * kv.max_pages + (j >> kv.page_log2)];
  if (id < 0 || id >= kv.n_pages) {
    atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
    return -1;
  }
  return ((id * kv.n_heads + pc.hk) << kv.page_log2) + (j & (kv.page - 1));
}

__device__ __forceinline__ bool seen_by_some(const Runs& r, int j) { return j < r.b_end && (j >= r.b_begin || j < r.a_end); }

// Key of group g (16 keys) of block `blk`, and whether the chunk exists.
__device__ __forceinline__ int group_key(const Piece& pc, int blk, int g) {
  const int i = 2 * blk + (g >> 2);
  return i < pc.ch.total ? pc.ch.key(i) + 16 * (g & 3) : -1;
}

// A block's copies are cut into units of one instruction of a warp, dealt to the kLoaders warps in turn.
__device__ __forceinline__ void load_q(const KvAttnParams& p, AttnSmem& sm, const Piece& pc, int buf, int warp, int lane) {
  const int col = lane & 7;
#pragma unroll 2
  for (int u = warp; u < kItem / 4; u += kLoaders) {
    const int r = 4 * u + (lane >> 3), a = pc.row0 + r;
    const bool have = r < pc.rows;
    const int tok = a / p.group, head = pc.hk * p.group + a - tok * p.group;
    const uint16_t* src = have ? p.q + (pc.s.row0 + tok) * p.q_ts + head * p.q_hs + col * 8 : p.q;
    cp_async16(smem_u32(sm.q[buf][r >> 7]) + (r & 127) * kRowBytes + ((col ^ (r & 7)) << 4), src, have ? 16u : 0u);
  }
}

__device__ __forceinline__ void loader_bf16(const KvAttnParams& p, AttnSmem& sm, int warp, int lane) {
  const int col = lane & 7, rr = lane >> 3;
  const uint16_t* kp = (p.ck ? p.ck : reinterpret_cast<const uint16_t*>(p.kv.k)) + col * 8;
  const uint16_t* vp = (p.ck ? p.cv : reinterpret_cast<const uint16_t*>(p.kv.v)) + col * 8;
  Walk w(p, sm.plan);
  Piece pc;
  uint32_t n = 0, pieces = 0;
  bool ok = true;
  while (ok && w.next(p, pc)) {
    const int buf = pieces & 1;
    if (pieces >= 2 && !wait_all(p, sm, &sm.q_empty[buf], ((pieces >> 1) - 1) & 1)) break;
    ++pieces;
    load_q(p, sm, pc, buf, warp, lane);
    auto rows_of = [&](int blk) {  // lane g < 8: the first row of the block's group g
      const int j = lane < 8 && blk < pc.blk1 ? group_key(pc, blk, lane) : -1;
      return j >= 0 ? group_row(p, pc, j) : -1;
    };
    int base = rows_of(pc.blk0);
    int pend = -1;
    for (int blk = pc.blk0; blk < pc.blk1; ++blk, ++n) {
      const int next = rows_of(blk + 1);
      const uint32_t st = n % kStages;
      if (n >= kStages && !wait_all(p, sm, &sm.empty[st], ((n / kStages) & 1) ^ 1)) {
        ok = false;
        break;
      }
      const uint32_t kd = smem_u32(sm.kv[st]);
      const int key0 = pc.ch.key(2 * blk), key1 = 2 * blk + 1 < pc.ch.total ? pc.ch.key(2 * blk + 1) : INT_MAX - 64;
#pragma unroll 4
      for (int u = warp; u < 32; u += kLoaders) {  // four rows of K and of V
        const int r = 4 * u + rr;
        const int row = __shfl_sync(0xffffffffu, base, u >> 2);
        const bool have = row >= 0 && seen_by_some(pc.runs, (r < 64 ? key0 : key1 - 64) + r);
        const long long at = have ? static_cast<long long>(row + (r & 15)) * kD : 0;
        const uint32_t dst = kd + r * kRowBytes + ((col ^ (r & 7)) << 4);
        cp_async16(dst, kp + at, have ? 16u : 0u);
        cp_async16(dst + kBlockBytes, vp + at, have ? 16u : 0u);
      }
      cp_async_commit();
      if (pend >= 0) {
        cp_async_wait<1>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[pend]);
      }
      pend = static_cast<int>(st);
      base = next;
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    __syncwarp();
    if (pend >= 0 && lane == 0) mbar_arrive(&sm.full[pend]);
  }
  cp_async_wait<0>();
}

// two codes as the bf16 values that they stand for
__device__ __forceinline__ uint32_t bf16x2_of_e4m3(uint32_t two, float scale) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  float a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(a), "=f"(b) : "r"(h));
  return pack_bf16x2(a * scale, b * scale);
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 8-bit caches: the codes go to a ring of raw blocks first, kRaw - 1 blocks ahead; each thread converts the
// 16-byte pieces that it copied itself, so that waiting for its own copies is enough.
__device__ __forceinline__ void loader_e4m3(const KvAttnParams& p, AttnSmem& sm, int warp, int lane) {
  const int c = lane & 3, rr = lane >> 2;
  const KvView& kv = p.kv;
  Walk w(p, sm.plan);
  Piece pc;
  uint32_t n = 0, pieces = 0;
  bool ok = true;
  while (ok && w.next(p, pc)) {
    const int buf = pieces & 1;
    if (pieces >= 2 && !wait_all(p, sm, &sm.q_empty[buf], ((pieces >> 1) - 1) & 1)) break;
    ++pieces;
    load_q(p, sm, pc, buf, warp, lane);
    float ks[kRaw], vs[kRaw];  // lane g < 8: the scales of group g, of the blocks in flight
    auto copy = [&](int blk, uint32_t slot, float& sk, float& sv) {
      sk = sv = 1.f;
      if (blk < pc.blk1) {
        const int j = lane < 8 ? group_key(pc, blk, lane) : -1;
        const int base = j >= 0 ? group_row(p, pc, j) : -1;
        if (base >= 0) {
          sk = kv.k_scale[base >> kv.page_log2];
          sv = kv.v_scale[base >> kv.page_log2];
        }
        const int key0 = pc.ch.key(2 * blk), key1 = 2 * blk + 1 < pc.ch.total ? pc.ch.key(2 * blk + 1) : INT_MAX - 64;
        const uint32_t dst = smem_u32(sm.raw[slot]) + lane * 16;
#pragma unroll 2
        for (int u = warp; u < 16; u += kLoaders) {  // eight rows of K and of V
          const int r = 8 * u + rr;
          const int row = __shfl_sync(0xffffffffu, base, u >> 1);
          const bool have = row >= 0 && seen_by_some(pc.runs, (r < 64 ? key0 : key1 - 64) + r);
          const long long at = have ? static_cast<long long>(row + (r & 15)) * kD + 16 * c : 0;
          cp_async16(dst + u * 512, kv.k + at, have ? 16u : 0u);
          cp_async16(dst + u * 512 + 8192, kv.v + at, have ? 16u : 0u);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i + 1 < kRaw; ++i) copy(pc.blk0 + i, (n + i) % kRaw, ks[i], vs[i]);
    for (int blk = pc.blk0; blk < pc.blk1; ++blk, ++n) {
      copy(blk + kRaw - 1, (n + kRaw - 1) % kRaw, ks[kRaw - 1], vs[kRaw - 1]);
      const uint32_t st = n % kStages;
      if (n >= kStages && !wait_all(p, sm, &sm.empty[st], ((n / kStages) & 1) ^ 1)) {
        ok = false;
        break;
      }
      cp_async_wait<kRaw - 1>();
      const uint32_t src = smem_u32(sm.raw[n % kRaw]) + lane * 16, kd = smem_u32(sm.kv[st]);
#pragma unroll 1
      for (int half = 0; half < 2; ++half)
#pragma unroll 2
        for (int u = warp; u < 16; u += kLoaders) {
          const float scale = __shfl_sync(0xffffffffu, half ? vs[0] : ks[0], u >> 1);
          uint32_t x[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(src + u * 512 + half * 8192)
                       : "memory");
          const uint32_t row = kd + half * kBlockBytes + (8 * u + rr) * kRowBytes;  // row & 7 is rr
#pragma unroll
          for (int i = 0; i < 2; ++i)
            st_shared16(row + (((2 * c + i) ^ rr) << 4), bf16x2_of_e4m3(x[2 * i], scale),
                        bf16x2_of_e4m3(x[2 * i] >> 16, scale), bf16x2_of_e4m3(x[2 * i + 1], scale),
                        bf16x2_of_e4m3(x[2 * i + 1] >> 16, scale));
        }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.full[st]);
#pragma unroll
      for (int i = 0; i + 1 < kRaw; ++i) {
        ks[i] = ks[i + 1];
        vs[i] = vs[i + 1];
      }
    }
    cp_async_wait<0>();
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ products

constexpr uint64_t kTileDesc = kBlockBytes >> 4, kStageDesc = 2 * kTileDesc;

// S_t = Q_t K^T for one block of 128 keys
__device__ __forceinline__ void issue_qk(uint64_t dq, uint64_t dk, uint32_t tmem, int t) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) mma_ss(tmem + t * 256, dq + 2 * kk, dk + 2 * kk, idesc, kk > 0 ? 1u : 0u);
}

// Run by the whole warp (which keeps the descriptors uniform); one elected lane issues.  For each block and tile:
// O += P V of each key half as soon as its warps have written P, then S = Q K^T of the next block, over P.
__device__ __forceinline__ void mma_role(const KvAttnParams& p, AttnSmem& sm, uint32_t tmem) {
  constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 64, 0, 1);
  const uint64_t q0 = smem_desc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
  const uint64_t k0 = smem_desc_sw128(smem_u32(sm.kv[0]), 16, 1024);
  const uint64_t v0 = smem_desc_sw128(smem_u32(sm.kv[0]) + kBlockBytes, 8192, 1024);
  Walk w(p, sm.plan);
  Piece pc;
  uint32_t n = 0, pieces = 0;
  uint32_t pfull[2] = {0, 0};
  while (w.next(p, pc)) {
    const int nblk = pc.blk1 - pc.blk0, tiles = pc.rows > 128 ? 2 : 1;
    const uint64_t dq = q0 + (pieces & 1) * 2 * kTileDesc;
    uint64_t* q_empty = &sm.q_empty[pieces & 1];
    ++pieces;
    {
      const uint32_t st = n % kStages;
      if (!wait_all(p, sm, &sm.full[st], (n / kStages) & 1)) return;
      tc_fence_after();
      if (elect_one()) {
        for (int t = 0; t < tiles; ++t) {
          issue_qk(dq + t * kTileDesc, k0 + st * kStageDesc, tmem, t);
          mma_commit(&sm.s_full[t]);
        }
        if (nblk == 1) mma_commit(q_empty);
      }
      __syncwarp();
    }
    for (int j = 0; j < nblk; ++j) {
      const uint32_t cs = (n + j) % kStages;
      const bool more = j + 1 < nblk;
      const uint32_t ns = (n + j + 1) % kStages;
      if (more && !wait_all(p, sm, &sm.full[ns], ((n + j + 1) / kStages) & 1)) return;
      tc_fence_after();
      const uint64_t dv = v0 + cs * kStageDesc;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t >= tiles) break;
        const uint32_t s_col = tmem + t * 256, o_col = s_col + 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait_all(p, sm, &sm.p_full[t][h], pfull[t] & 1)) return;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(o_col + 64 * h, s_col + 64 * h + kk * 8, dv + 128 * (4 * h + kk), idesc_pv, j > 0 || kk > 0 ? 1u : 0u);
          }
          __syncwarp();
        }
        ++pfull[t];
        if (elect_one()) {
          if (more) {
            issue_qk(dq + t * kTileDesc, k0 + ns * kStageDesc, tmem, t);
            mma_commit(&sm.s_full[t]);
          } else {
            mma_commit(&sm.o_done[t]);
          }
        }
        __syncwarp();
      }
      if (elect_one()) {
        mma_commit(&sm.empty[cs]);
        if (j + 2 == nblk) mma_commit(q_empty);
      }
      __syncwarp();
    }
    n += nblk;
  }
}

// ------------------------------------------------------------------ softmax

__device__ __forceinline__ uint64_t range_bits(int a, int b) {
  // bits [a, b) of a 64-bit word
  a = max(a, 0);
  b = min(b, 64);
  if (a >= b) return 0ull;
  return (~0ull >> (64 - (b - a))) << a;
}

// 2^x0, 2^x1 on the FMA pipe: 2^floor(x) p(x - floor(x)), the floor from one addition rounded down;
// x below -127 gives 0
__device__ __forceinline__ void exp2_poly2(float x0, float x1, float& e0, float& e1) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  x0 = fmaxf(x0, -127.f);
  x1 = fmaxf(x1, -127.f);
  uint64_t t, xi, f, pp;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(t) : "l"(f32x2(x0, x1)), "l"(f32x2(kMagic, kMagic)));
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(xi) : "l"(t), "l"(f32x2(kMagic, kMagic)));
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(f) : "l"(f32x2(x0, x1)), "l"(xi));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(pp) : "l"(f), "l"(f32x2(kExpC3, kExpC3)), "l"(f32x2(kExpC2, kExpC2)));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(pp) : "l"(pp), "l"(f), "l"(f32x2(kExpC1, kExpC1)));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(pp) : "l"(pp), "l"(f), "l"(f32x2(1.f, 1.f)));
  e0 = __uint_as_float(static_cast<uint32_t>(pp) + (static_cast<uint32_t>(t) << 23));
  e1 = __uint_as_float(static_cast<uint32_t>(pp >> 32) + (static_cast<uint32_t>(t >> 32) << 23));
}

// O of this warp's rows and key half times alpha
__device__ __forceinline__ void rescale_o(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    uint32_t o[16];
    tmem_ld16(tO + q * 16, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st16(tO + q * 16, o);
  }
}

__device__ __forceinline__ void softmax_role(const KvAttnParams& p, AttnSmem& sm, uint32_t tmem, int sw, int lane) {
  const int t = sw >> 3, h = (sw >> 2) & 1, wq = sw & 3;
  const int r = wq * 32 + lane;  // row of the tile
  const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t tS = tmem + lane_off + t * 256 + h * 64, tO = tmem + lane_off + t * 256 + 128;
  bool withhold = p.withhold != 0 && blockIdx.x == 0 && sw == 0;  // test hook
  Walk w(p, sm.plan);
  Piece pc;
  uint32_t sfull = 0, pieces = 0;
  while (w.next(p, pc)) {
    if (pc.rows <= t * 128) continue;  // the item has one tile
    const int a = pc.row0 + min(t * 128 + r, pc.rows - 1), tok = a / p.group;
    const Span sp = span_of(p.win, pc.s.len - pc.s.n_new + tok, pc.s.len);
    float m = -INFINITY, l = 0.f;
    bool part = false;  // some streamed key is out of this row's sight
    for (int blk = pc.blk0; blk < pc.blk1; ++blk) {
      const int i = 2 * blk + h, j0 = pc.ch.key(i);
      const bool have = i < pc.ch.total;
      const bool whole = have && ((j0 >= sp.lo && j0 + 64 <= sp.hi) || j0 + 64 <= sp.sink);
      const bool all = __all_sync(0xffffffffu, whole);
      uint64_t valid = ~0ull;
      if (!all) {
        valid = have ? range_bits(sp.lo - j0, sp.hi - j0) | range_bits(0, sp.sink - j0) : 0ull;
        part |= have && !whole;
      }
      if (!wait_all(p, sm, &sm.s_full[t], sfull & 1)) return;
      ++sfull;
      tc_fence_after();
      uint32_t pk[32];
      if (!all && __all_sync(0xffffffffu, valid == 0ull)) {
        // no row of this warp sees a key of the chunk
#pragma unroll
        for (int q = 0; q < 32; ++q) pk[q] = 0u;
      } else {
        float s[64];
        {
          uint32_t raw[64];
          tmem_ld64(tS, raw);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 64; ++q) s[q] = __uint_as_float(raw[q]);
        }
        if (!all) {
#pragma unroll
          for (int q = 0; q < 64; ++q)
            if (!((valid >> q) & 1ull)) s[q] = -INFINITY;
        }
        float mp[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mp[q] = s[q];
#pragma unroll
        for (int q = 2; q < 32; ++q) mp[q & 3] = max3f(mp[q & 3], s[2 * q], s[2 * q + 1]);
        const float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * kScaleLog2;
        if (blk == pc.blk0) {
          m = mx;
        } else {
          const bool grow = mx > m + kGrow;
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? fast_exp2(m - mx) : 1.f;  // m may be -inf: alpha = 0
            rescale_o(tO + h * 64, alpha);
            l *= alpha;
            if (grow) m = mx;
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float rp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          float x0 = s[2 * q], x1 = s[2 * q + 1];
          ffma2(x0, x1, kScaleLog2, -ref);
          if ((kPolyPairs >> q) & 1u) {
            exp2_poly2(x0, x1, x0, x1);
          } else {
            x0 = fast_exp2(x0);
            x1 = fast_exp2(x1);
          }
          fadd2(rp[2 * (q & 1)], rp[2 * (q & 1) + 1], x0, x1);
          pk[q] = pack_bf16x2(x0, x1);
        }
        l += (rp[0] + rp[1]) + (rp[2] + rp[3]);
      }
      tmem_st32(tS, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (withhold)
        withhold = false;
      else if (lane == 0)
        mbar_arrive(&sm.p_full[t][h]);
    }
    // join the two key halves; this thread finishes columns 32h..32h+31 of its row
    const uint32_t par = pieces & 1;
    ++pieces;
    float* mine = sm.stats[par][t][h][r];
    mine[0] = m;
    mine[1] = part ? -l - 1e-30f : l;  // the sign says that some keys are out of sight
    mbar_arrive(&sm.pair[t][wq]);
    if (!wait_all(p, sm, &sm.o_done[t], par)) return;
    if (!wait_all(p, sm, &sm.pair[t][wq], par)) return;
    tc_fence_after();
    const float* other = sm.stats[par][t][h ^ 1][r];
    const float mo = other[0], lo = fabsf(other[1]);
    part |= other[1] < 0.f;
    const float mm = fmaxf(m, mo);
    const float fm = m == -INFINITY ? 0.f : fast_exp2(m - mm), fo = mo == -INFINITY ? 0.f : fast_exp2(mo - mm);
    const float den = l * fm + lo * fo;
    const float scale = pc.slot >= 0 ? 1.f : (den == 0.f ? 0.f : 1.f / den);
    const float f0 = (h ? fo : fm) * scale, f1 = (h ? fm : fo) * scale;
    float o[32];
    {
      uint32_t oa[32], ob[32];
      tmem_ld32(tO + 32 * h, oa);
      tmem_ld32(tO + 64 + 32 * h, ob);
      tmem_wait_ld();
      tc_fence_before();
#pragma unroll
      for (int q = 0; q < 32; ++q) o[q] = __uint_as_float(oa[q]) * f0 + __uint_as_float(ob[q]) * f1;
    }
    const int row = t * 128 + r;
    if (pc.slot >= 0) {
      Slot& sl = reinterpret_cast<Work*>(p.ws)->slots[blockIdx.x][pc.slot];
      float4* d = reinterpret_cast<float4*>(&sl.o[row][32 * h]);
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      if (h == 0) {
        sl.m[row] = mm;
        sl.l[row] = den;
        sl.part[row] = part;
      }
      continue;
    }
    const int head = pc.hk * p.group + a - tok * p.group;
    const bool live = row < pc.rows;
    bool bad = false;
#pragma unroll
    for (int q = 0; q < 32; ++q) bad |= !(fabsf(o[q]) <= 3.402823466e+38f);
    bad &= part;
    if (live && !bad) {
      const long long at = (pc.s.row0 + tok) * p.out_ts + head * p.out_hs + 32 * h;
      if (p.out_fp32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
        for (int q = 0; q < 8; ++q) d[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      } else {
        uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          d[q] = make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                            pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
      }
    }
    // a value out of the row's sight is not finite (or one in sight is): key by key
    uint32_t todo = __ballot_sync(0xffffffffu, live && bad);
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int tk = __shfl_sync(0xffffffffu, tok, src), hd = __shfl_sync(0xffffffffu, head, src);
      exact_row(p, pc.b, pc.s.len, pc.s.row0 + tk, pc.s.len - pc.s.n_new + tk, hd, lane, 32 * h, 32 * h + 32);
    }
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_kernel(const __grid_constant__ KvAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  AttnSmem& sm = *reinterpret_cast<AttnSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], kLoaders);
      mbar_init(&sm.empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.q_empty[t], 1);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.o_done[t], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&sm.p_full[t][h], 4);
      for (int w = 0; w < 4; ++w) mbar_init(&sm.pair[t][w], 64);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  make_plan(p, sm.plan, reinterpret_cast<long long*>(sm.kv[0]));  // the ring is not in use yet
  if (warp == 3) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  // registers: launched with 96 x 640; 64 x 128 + 104 x 512 are as many
  if (warp < 4) {
    reg_dealloc_dec<64>();
    if (warp == 3) {
      mma_role(p, sm, tmem);
      // also after a wait that gave up: no product is in flight when the block lets its memory go
      if (elect_one()) mma_commit(&sm.drain);
      __syncwarp();
      mbar_wait_drain(&sm.drain, 0, kDrainBudget);
    } else if (kE4m3) {
      loader_e4m3(p, sm, warp, lane);
    } else {
      loader_bf16(p, sm, warp, lane);
    }
  } else {
    reg_alloc_inc<104>();
    softmax_role(p, sm, tmem, warp - 4, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Finishes the items that shares' borders cut: block (i, y) has rows 32y.. of the item first cut by share i's
// start.  8 threads a row, 8 columns each; pieces in their order.
__global__ void __launch_bounds__(256) kv_join_kernel(const __grid_constant__ KvAttnParams p) {
  const Work& wk = *reinterpret_cast<const Work*>(p.ws);
  const Cut& cut = wk.cuts[blockIdx.x + 1];
  const int r = blockIdx.y * 32 + (threadIdx.x >> 3), col = (threadIdx.x & 7) * 8, lane = threadIdx.x & 31;
  if (!cut.valid || blockIdx.y * 32 >= cut.rows) return;
  float mm = -INFINITY, l = 0.f, o[8];
  bool part = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  int b0 = 0;
  for (int c = blockIdx.x; b0 < cut.nblk; ++c) {
    const int b1 = blocks_before(cut.total * (c + 1) / cut.shares - cut.x0, cut.nblk, cut.unit);
    if (b1 > b0) {
      const Slot& sl = wk.slots[c][b0 > 0 ? 0 : 1];
      const float m = sl.m[r], nm = fmaxf(mm, m);
      const float f = mm == -INFINITY ? 0.f : fast_exp2(mm - nm), g = m == -INFINITY ? 0.f : fast_exp2(m - nm);
      const float4* src = reinterpret_cast<const float4*>(&sl.o[r][col]);
      const float4 x = src[0], y = src[1];
      o[0] = o[0] * f + x.x * g; o[1] = o[1] * f + x.y * g; o[2] = o[2] * f + x.z * g; o[3] = o[3] * f + x.w * g;
      o[4] = o[4] * f + y.x * g; o[5] = o[5] * f + y.y * g; o[6] = o[6] * f + y.z * g; o[7] = o[7] * f + y.w * g;
      l = l * f + sl.l[r] * g;
      part |= sl.part[r] != 0;
      mm = nm;
    }
    b0 = b1;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i] *= inv;
    bad |= !(fabsf(o[i]) <= 3.402823466e+38f);
  }
  // a row is exact as a whole: its 8 threads agree
  const bool live = r < cut.rows;
  uint32_t todo = __ballot_sync(0xffffffffu, live && bad && part);
  const bool mine = ((todo >> (lane & 24)) & 0xffu) != 0;
  const int a = cut.row0 + r, tok = a / p.group, head = cut.hk * p.group + a - tok * p.group;
  if (live && !mine) {
    const long long at = (cut.first + tok) * p.out_ts + head * p.out_hs + col;
    if (p.out_fp32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
      d[0] = make_float4(o[0], o[1], o[2], o[3]);
      d[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) =
          make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    }
  }
  for (int k = 0; k < 4; ++k) {
    if (!((todo >> (8 * k)) & 0xffu)) continue;
    const int tk = __shfl_sync(0xffffffffu, tok, 8 * k), hd = __shfl_sync(0xffffffffu, head, 8 * k);
    exact_row(p, cut.b, cut.len, cut.first + tk, cut.len - cut.n_new + tk, hd, lane, 0, kD);
  }
}

}  // namespace

size_t attn_workspace_bytes() { return sizeof(Work); }

cudaError_t launch_attn(const KvAttnParams& p, cudaStream_t stream, int* n_launch) {
  const int smem = static_cast<int>(sizeof(AttnSmem) + 1024);
  const auto kernel = p.e4m3 ? kv_attn_kernel<true> : kv_attn_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = p.num_sms < kMaxShares ? p.num_sms : kMaxShares;
  kernel<<<grid, kThreads, smem, stream>>>(p);
  ++*n_launch;
  if ((e = cudaGetLastError()) != cudaSuccess || grid == 1) return e;
  kv_join_kernel<<<dim3(grid - 1, kItem / 32), 256, 0, stream>>>(p);
  ++*n_launch;
  return cudaGetLastError();
}

}  // namespace saf3r
