// Attention over the paged cache, or over keys and values held at once, for many query rows: the
// tensor-core kernel of the streaming operators (tcgen05, sm_100a).
//
// An item is 256 rows of one kv head (its group's heads times new tokens, token after token) of one sequence: two
// 128-row tiles.  The keys that some row of the item sees (Runs) are streamed 128 at a time, as two
// chunks of 64.  The items' key blocks, laid end to end, are cut into equal shares, one CTA each: an item
// cut by a share's border is finished by the join kernel from its pieces' answers.  Equal shares
// keep every SM busy with few items (one view of one stream: 96 items of unequal length on 148 SMs).
//
// Warps (20, or 24 with 8-bit caches):
//   0-1    loaders: each block's K and V rows into a ring of stages, in the 128-byte-swizzled layout that the tensor
//          core reads, a TMA box for each page (or 64 rows of it).  Value rows that no row of the item sees are cleared:
//          what lies behind a sequence's end need not be finite.  bf16: TMA writes the stage itself.  8-bit: the
//          codes land beside it, and four more warps (4-7) turn them into fp16 times their page's scale over the
//          largest of the piece: exact where the scales are within 2^22 of one another; where the values' are not, or
//          the keys' and it would show, the piece's rows go key by key.  P is fp16 then: 2^-11 of a weight, and 2^-25 of the
//          row's first chunk's largest.
//   2-3    issue the products, a warp for each tile.
//   last 16 softmax: four warpgroups, one for each tile and key half; a thread has one row's 64 keys of a block.
//          Sixteen warps, four for each scheduler in different steps, hide each other's waits.
// Tensor memory (512 columns, 256 a tile).  bf16: three S buffers of 64 fp32 columns (P, bf16, goes over the first 32 columns
// of its S once read) and one accumulator O of 64 columns, whose halves share a reference.  8-bit: S and O for each key half.
//
// Weights are 2^(x - reference), the reference a row's largest logit of its first block: bf16 P and the fp32 sums
// keep their relative precision at any reference, so no maximum is taken of later blocks.  bf16 weights may grow to 2^64
// (a row beyond goes key by key); fp16 ones to 2^15, then the reference moves and what was summed so far is scaled.
// Key by key (stream_exact.cuh) go also rows whose answer is not finite while it may be: next to a masked value that is not, or
// where the sum of weights times values left fp32's range.  It costs 0.11 us a key and row: one 8-bit view of 1,374 tokens and 16
// heads over 5,496 keys 83 us, with all rows key by key 5.7 ms.
//
// What bounds it: at d = 64 each (query, key) pair is 256 tensor operations and one exponential, and the softmax warps' pipes
// set the pace: per block of 256 rows and 128 keys 1,792 cycles of the exponential unit (one pair in eight is computed on the
// FMA pipe: none took 604 us, one in four 571 us, one in eight 556 us) of about 2,350; products take 1,264.  Measured, 16 heads,
// bf16: 562 us for 10,992 rows and keys = 881 TFLOP/s with the GPU cool, 54% of the measured burst rate; long runs meet the power
// cap and end near 1.5 GHz and 690 TFLOP/s.  8-bit: 243 us for 2 x 1,374 rows over 12,366 keys = 573 TFLOP/s, where the
// converting warps take the schedulers' slots as well.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ptx.cuh"
#include "stream.h"
#include "stream_exact.cuh"

namespace saf3r {

namespace {

constexpr int kConverters = 4;         // warps that convert 8-bit codes
constexpr int kScales = 8;             // blocks whose scales are kept: 3 raw ones and the 4 stages'
constexpr int kMaxStages = 5;
constexpr int kPieces = 4;             // pieces that warp 0 may be ahead
constexpr int kItem = 256;             // rows of an item
constexpr int kRowBytes = 128;
constexpr int kBlockBytes = 128 * kRowBytes;  // 128 rows x 64 bf16
constexpr float kScaleLog2 = 0.18033688011112042f;  // log2(e) / sqrt(64)
constexpr float kGrowLog2 = 64.f, kGrow = 1.8446744073709552e19f;  // a row with weights beyond 2^64 goes key by key
constexpr float kGrowF16Log2 = 15.f, kGrowF16 = 32768.f;           // fp16 weights: 2^15
// Codes of a piece's largest scale are multiplied by 2^7 (448 * 2^7 is in fp16's range), those of scales down to 2^-22 of it
// by 2^-15 at least: exact in fp16, subnormal codes too.
constexpr int kCodeTop = 7, kWild = 22;
// Keys of scales below that lose up to 448 * 2^-25 (f16_power is 0 from 2^-32 on), queries are below 2: a sum of 64 products is
// off by 2^-9.2 at most, a logit by that times what the sum is multiplied by.  Up to 2^-3 it is 2^-12, within the exponentials'
// own error; above (the row's largest query times the largest key beyond about 2^15) the row goes key by key.
constexpr float kQuiet = 0.125f;
constexpr int kMaxShares = 160;        // CTAs of a launch at most (one for each SM)
constexpr int kPlanEntries = 1024;
// Cost of a key block of two tiles and of one (which waits more), and of an item's start and end, in sixteenths of the first.
constexpr int kCost2 = 16, kCost1 = 13, kCostItem = 56;
constexpr int kLeastShare = 2 * kCost2;  // shares smaller than this are not worth a CTA

// Pairs (of the 32 of a row's 64 keys) whose exponentials run on the FMA pipe.
constexpr uint32_t kPolyPairs = 0x10101010u;

// A share's part of an unfinished item: per row its answer, the sum of its weights and their reference.
struct Slot {
  float o[kItem][kD];  // the piece's own answer: divided by l
  float m[kItem], l[kItem];
  int32_t part[kItem];  // nonzero: some streamed key is out of the row's sight
};
static_assert(sizeof(Slot) % 16 == 0, "slots stay aligned");

// An item whose first cut is the start of share i.
struct Cut {
  int32_t valid, b, hk, row0, rows;
  int32_t first, n_new, len;  // the sequence
  int32_t nblk, unit, extra;
  int32_t pad;
  long long x0, each;  // where the item begins; share_start's
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
  const Span a = span_of(p.win, start + p.by_group.div(r0), s.len);
  const Span z = span_of(p.win, start + p.by_group.div(r0 + t.rows - 1), s.len);
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
  if (d >= static_cast<long long>(nblk) * unit) return nblk;
  return (static_cast<int>(d) + unit - 1) / unit;
}

// Where share i of the line starts: the first `extra` shares have one unit more than `each`.
__host__ __device__ __forceinline__ long long share_start(long long each, int extra, int i) { return each * i + (i < extra ? i : extra); }

// 8-bit: the scales of a block's groups of 16 keys: of the keys, then of the values.
struct alignas(16) BlockScale {
  float of[16];
};
// 8-bit: exponents of the largest scales of a piece's keys and values, and whether some scale is too small beside them (1: of
// the values, 2: of the keys).
struct PieceScale {
  int k, v, wild;
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

// Walks the pieces of this CTA's share: the range xs..xe of the line of all items (warp 0).
struct Walk {
  long long x, xs, xe;  // x: start of the item at (hk, b, tile)
  int hk, b, tile;
  SeqInfo s;

  __device__ __forceinline__ bool next(const KvAttnParams& p, Piece& pc) {
    while (x < xe) {
      while (tile >= tiles_of(p, s)) {
        tile = 0;
        if (++b == p.kv.n_seqs) {
          b = 0;
          if (++hk == p.kv.n_heads) break;
        }
        s = seq_info(p.kv, b);
      }
      if (hk == p.kv.n_heads) break;
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
    pc.blk1 = -1;
    return false;
  }
};

// The ring of key blocks (stages of 128 rows of K, then of V) and, for 8-bit caches, the raw blocks behind it.
template <bool kE4m3>
struct Ring {
  static constexpr int kWarps = kE4m3 ? 24 : 20, kSoftmax = kWarps - 16;  // warps, the first softmax warp
  static constexpr int kStages = kE4m3 ? 4 : 5, kRaw = kE4m3 ? 3 : 0;
  static constexpr int kBytes = (2 * kStages + kRaw) * kBlockBytes;
};
constexpr int kRingBytes = Ring<true>::kBytes > Ring<false>::kBytes ? Ring<true>::kBytes : Ring<false>::kBytes;

struct AttnSmem {
  uint8_t q[2][kBlockBytes];
  uint8_t ring[kRingBytes];
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t raw[kMaxStages], raw_empty[kMaxStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][3], o_done[2], p_full[2][3];
  uint64_t drain[2];
  uint64_t pair[2][4];                // the two warps of a tile's 32 rows meet here
  float2 stats[2][2][2][128];         // [parity][tile][half][row]: what the halves tell one another
  BlockScale scale[kScales];
  PieceScale piece_scale[kPieces];
  uint64_t scale_full[kPieces];
  int16_t q_exp[kPieces][kItem][2];   // 8-bit: exponent of a row's queries, for each half's threads
  Walk walk;
  Piece pieces[kPieces];              // warp 0's walk, for the other warps; blk1 < 0: the end
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint32_t tmem_base;
  int abort;
};

// Inclusive sums over a warp's lanes.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Finds this CTA's share and its first piece (run by all threads; `entries` is scratch in shared memory).  Nothing is
// planned ahead in a kernel of its own: the lengths are on the device, and a launch would cost more than this.
__device__ __forceinline__ void make_plan(const KvAttnParams& p, Walk& walk, Piece& first, long long* entries) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.kv.n_seqs + kPlanEntries - 1) / kPlanEntries;
  const int n = (p.kv.n_seqs + per - 1) / per;
  for (int e = warp; e < n; e += blockDim.x / 32) {
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
  const int shares = total >= static_cast<long long>(gridDim.x) * kLeastShare ? gridDim.x : max(1, static_cast<int>(total) / kLeastShare);
  const int me = blockIdx.x;
  const long long each = total / shares;
  const int extra = static_cast<int>(total - each * shares);
  Walk w;
  w.xs = me < shares ? share_start(each, extra, me) : total;
  w.xe = me < shares ? share_start(each, extra, me + 1) : total;
  w.x = w.xs;
  w.hk = w.b = w.tile = 0;
  w.s = SeqInfo{0, 0, 0, false};
  Cut cut{};
  if (w.xs < w.xe) {
    long long rest = w.xs;  // inside what is left
    while (rest >= head) {
      rest -= head;
      ++w.hk;
    }
    for (int e0 = 0; e0 < n; e0 += 32) {
      const long long c = e0 + lane < n ? entries[e0 + lane] : 0, incl = warp_scan(c, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, rest < incl);
      if (hit) {
        const int src = __ffs(hit) - 1;
        w.b = (e0 + src) * per;
        rest -= __shfl_sync(0xffffffffu, incl - c, src);
        break;
      }
      rest -= __shfl_sync(0xffffffffu, incl, 31);
    }
    for (; per > 1 && w.b + 1 < p.kv.n_seqs; ++w.b) {
      const long long c = seq_cost(p, w.b, lane);
      if (rest < c) break;
      rest -= c;
    }
    w.s = seq_info(p.kv, w.b);
    const int nt = tiles_of(p, w.s);
    for (int t0 = 0; t0 < nt; t0 += 32) {
      const long long c = t0 + lane < nt ? tile_of(p, w.s, t0 + lane).cost : 0, incl = warp_scan(c, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, rest < incl);
      if (hit) {
        const int src = __ffs(hit) - 1;
        w.tile = t0 + src;
        rest -= __shfl_sync(0xffffffffu, incl - c, src);
        break;
      }
      rest -= __shfl_sync(0xffffffffu, incl, 31);
    }
    w.x = w.xs - rest;
    const Tile t = tile_of(p, w.s, w.tile);
    const int cutblk = blocks_before(rest, t.nblk, t.unit);
    cut.valid = me > 0 && cutblk > 0 && cutblk < t.nblk && blocks_before(share_start(each, extra, me - 1) - w.x, t.nblk, t.unit) == 0;
    cut.b = w.b;
    cut.hk = w.hk;
    cut.row0 = w.tile * kItem;
    cut.rows = t.rows;
    cut.first = w.s.row0;
    cut.n_new = w.s.n_new;
    cut.len = w.s.len;
    cut.nblk = t.nblk;
    cut.unit = t.unit;
    cut.x0 = w.x;
    cut.each = each;
    cut.extra = extra;
  }
  Piece pc;
  w.next(p, pc);
  if (lane == 0) {
    walk = w;
    first = pc;
    reinterpret_cast<Work*>(p.ws)->cuts[me] = cut;
  }
}

__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ bool wait_all(const KvAttnParams& p, AttnSmem& sm, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, &sm.abort, p.kv.err, p.wait_budget, SAF3R_ERR_TIMEOUT));
}

// The other warps' view of the walk.
struct Feed {
  uint32_t i = 0;
  __device__ __forceinline__ const Piece* next(const KvAttnParams& p, AttnSmem& sm) const {
    if (!wait_all(p, sm, &sm.piece_full[i % kPieces], (i / kPieces) & 1)) return nullptr;
    const Piece* pc = &sm.pieces[i % kPieces];
    return pc->blk1 < 0 ? nullptr : pc;
  }
  __device__ __forceinline__ void done(AttnSmem& sm, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.piece_empty[i % kPieces]);
    ++i;
  }
};
// Warp 0 hands piece number i to the others (pc.blk1 < 0: there are no more).  The plan has handed over the first.
__device__ __forceinline__ bool publish(const KvAttnParams& p, AttnSmem& sm, uint32_t i, const Piece& pc, int lane) {
  if (i == 0) return true;
  if (i >= kPieces && !wait_all(p, sm, &sm.piece_empty[i % kPieces], ((i / kPieces) & 1) ^ 1)) return false;
  if (lane == 0) {
    sm.pieces[i % kPieces] = pc;
    mbar_arrive(&sm.piece_full[i % kPieces]);
  }
  __syncwarp();
  return true;
}

// ------------------------------------------------------------------ loaders

// First key of this lane's box (2^box_log2 keys) of a block, -1: there is none, or no row sees a key of it.
__device__ __forceinline__ int box_key(const KvAttnParams& p, const Piece& pc, int blk, int lane) {
  const int i = lane << p.box_log2, c = 2 * blk + (i >> 6);
  if (i >= 128 || c >= pc.ch.total || blk >= pc.blk1) return -1;
  const int j = pc.ch.key(c) + (i & 63);
  return j < pc.runs.b_end && (j + (1 << p.box_log2) > pc.runs.b_begin || j < pc.runs.a_end) ? j : -1;
}

// Its entry of the page table (used a block later, so that the load's latency is out of the way).
__device__ __forceinline__ int box_entry(const KvAttnParams& p, const Piece& pc, int blk, int lane) {
  const int j = box_key(p, pc, blk, lane);
  if (j < 0 || p.ck) return 0;
  return p.kv.table[static_cast<long long>(pc.b) * p.kv.max_pages + (j >> p.kv.page_log2)];
}

// Its first row in the pools (views held at once: in the head), -1: not read, or the page is not there.
__device__ __forceinline__ int box_row(const KvAttnParams& p, const Piece& pc, int blk, int lane, int id) {
  const KvView& kv = p.kv;
  const int j = box_key(p, pc, blk, lane);
  if (j < 0) return -1;
  if (p.ck) return j;
  if (id < 0 || id >= kv.n_pages) {
    atomicCAS(kv.err, 0, SAF3R_ERR_INDEX);
    return -1;
  }
  return ((id * kv.n_heads + pc.hk) << kv.page_log2) + (j & (kv.page - 1));
}

__device__ __forceinline__ bool seen_by_some(const Runs& r, int j) { return j < r.b_end && (j >= r.b_begin || j < r.a_end); }

// Whether some row of the item sees every key of the block.
__device__ __forceinline__ bool whole_block(const Piece& pc, int blk) {
  if (2 * blk + 1 >= pc.ch.total) return false;
  const int a = pc.ch.key(2 * blk), b = pc.ch.key(2 * blk + 1);
  return (a + 64 <= pc.runs.a_end || (a >= pc.runs.b_begin && a + 64 <= pc.runs.b_end)) &&
         (b + 64 <= pc.runs.a_end || (b >= pc.runs.b_begin && b + 64 <= pc.runs.b_end));
}

// A block's boxes of K and V into `dst` (64 rows of a chunk after the other, K then V); run by a warp, one lane a box.
__device__ __forceinline__ void issue_boxes(const KvAttnParams& p, const CUtensorMap* mk, const CUtensorMap* mv, const Piece& pc,
                                            int row, uint8_t* dst, uint64_t* bar, int row_bytes, int lane) {
  const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
  if (lane == 0) mbar_arrive_expect_tx(bar, ((2 * __popc(have)) << p.box_log2) * row_bytes);
  __syncwarp();
  if (row >= 0) {
    const int head = p.ck ? pc.hk : 0;
    uint8_t* d = dst + (lane << p.box_log2) * row_bytes;
    tma_load_3d(d, mk, 0, row, head, bar);
    tma_load_3d(d + 128 * row_bytes, mv, 0, row, head, bar);
  }
  __syncwarp();
}

// bf16, warp 0: every block's TMA boxes, straight into its stage.  Blocks that no row sees all of land on `raw` first,
// for warp 1 to clear the values out of sight.
__device__ __forceinline__ void load_role(const KvAttnParams& p, AttnSmem& sm, const CUtensorMap* mk, const CUtensorMap* mv, int lane) {
  constexpr int kStages = Ring<false>::kStages;
  Walk w = sm.walk;
  Piece pc = sm.pieces[0];
  uint32_t n = 0, raw = 0, last_raw = 0;  // bit st: parity of raw[st]; whether the stage's last block was a partial one
  uint32_t pieces = 0;
  bool ok = true;
  for (bool more = pc.blk1 >= 0; ok && more; more = w.next(p, pc)) {
    if (!publish(p, sm, pieces, pc, lane)) {
      ok = false;
      break;
    }
    ++pieces;
    int entry = box_entry(p, pc, pc.blk0, lane);
    for (int blk = pc.blk0; blk < pc.blk1; ++blk, ++n) {
      const int row = box_row(p, pc, blk, lane, entry);
      entry = box_entry(p, pc, blk + 1, lane);
      const uint32_t st = n % kStages;
      if (n >= kStages && !wait_all(p, sm, &sm.empty[st], ((n / kStages) & 1) ^ 1)) {
        ok = false;
        break;
      }
      const bool whole = whole_block(pc, blk);
      issue_boxes(p, mk, mv, pc, row, sm.ring + st * 2 * kBlockBytes, whole ? &sm.full[st] : &sm.raw[st], kRowBytes, lane);
      if (lane == 0) mbar_arrive(&sm.full[st]);
      raw ^= (whole ? 0u : 1u) << st;
      last_raw = (last_raw & ~(1u << st)) | ((whole ? 0u : 1u) << st);
    }
  }
  if (ok) publish(p, sm, pieces, pc, lane);
  // every copy has landed before the block exits
  for (uint32_t c = n > kStages ? n - kStages : 0; c < n; ++c) {
    const uint32_t st = c % kStages;
    if ((last_raw >> st) & 1u)
      mbar_wait_drain(&sm.raw[st], ((raw >> st) & 1u) ^ 1u, kDrainBudget);
    else
      mbar_wait_drain(&sm.full[st], (c / kStages) & 1, kDrainBudget);
  }
}

// bf16, warp 1: the pieces' queries where TMA takes them (p.q_tma), and zeros over the values of partial blocks that no row
// sees (what lies there need not be finite).
__device__ __forceinline__ void side_role(const KvAttnParams& p, AttnSmem& sm, const CUtensorMap* mq, int lane) {
  constexpr int kStages = Ring<false>::kStages;
  Feed feed;
  uint32_t n = 0, raw = 0, queries[2] = {0, 0};
  auto drain = [&]() {  // every copy has landed before the block exits
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (queries[t] > 0) mbar_wait_drain(&sm.q_full[t], (queries[t] & 1) ^ 1, kDrainBudget);
  };
  while (const Piece* next = feed.next(p, sm)) {
    const Piece& pc = *next;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (!p.q_tma || pc.rows <= t * 128) continue;
      if (queries[t] > 0 && !wait_all(p, sm, &sm.q_empty[t], (queries[t] & 1) ^ 1)) {
        drain();
        return;
      }
      ++queries[t];
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full[t], kBlockBytes);
#pragma unroll
        for (int i = 0; i < 2; ++i)  // 64 rows: the heads of the group, token after token
          tma_load_4d(sm.q[t] + i * kBlockBytes / 2, mq, 0, 0, pc.s.row0 + p.by_group.div(pc.row0 + t * 128 + i * 64), pc.hk, &sm.q_full[t]);
      }
      __syncwarp();
    }
    for (int blk = pc.blk0; blk < pc.blk1; ++blk, ++n) {
      if (whole_block(pc, blk)) continue;
      const uint32_t st = n % kStages;
      if (!wait_all(p, sm, &sm.raw[st], (raw >> st) & 1u)) {
        drain();
        return;
      }
      raw ^= 1u << st;
      const uint32_t v = smem_u32(sm.ring + st * 2 * kBlockBytes + kBlockBytes);
#pragma unroll 1
      for (int r = lane; r < 128; r += 32) {
        const int c = 2 * blk + (r >> 6);
        if (c < pc.ch.total && seen_by_some(pc.runs, pc.ch.key(c) + (r & 63))) continue;
        for (int i = 0; i < 8; ++i) st_shared16(v + r * kRowBytes + i * 16, 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.full[st]);
    }
    feed.done(sm, lane);
  }
  drain();
}

__device__ __forceinline__ int exponent(float scale) { return static_cast<int>((__float_as_uint(scale) >> 23) & 0xffu) - 127; }
// 2^(kCodeTop + d) twice as fp16 (d <= 0; 0 below fp16's range)
__device__ __forceinline__ uint32_t f16_power(int d) {
  const int e = kCodeTop + d + 15;
  const uint32_t h = e >= 1 && e < 31 ? static_cast<uint32_t>(e) << 10 : (e > -10 && e < 1 ? 1u << (e + 9) : 0u);
  return h | (h << 16);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 8-bit, warp 1: the largest scales of every piece, and whether some are too small beside them.  Values may lose no bits,
// as a row may see such a page alone.  Keys may where no row can tell (kQuiet).  A scale of 2^-100 is that of rows of zeros
// (or of numbers below 2^-91): it does not count as too small.
__device__ __forceinline__ void scan_role(const KvAttnParams& p, AttnSmem& sm, int lane) {
  const KvView& kv = p.kv;
  Feed feed;
  while (const Piece* next = feed.next(p, sm)) {
    const Piece& pc = *next;
    int k_hi = -127, k_lo = 127, v_hi = -127, v_lo = 127;
    const int per_log2 = 7 - p.box_log2;  // boxes of a block
    // eight boxes of a lane at a time: their entries, then their scales
    for (int i0 = (pc.blk0 << per_log2) + lane; i0 < (pc.blk1 << per_log2); i0 += 256) {
      int id[8];
      float ks[8], vs[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int i = i0 + 32 * c;
        id[c] = box_entry(p, pc, i >> per_log2, i & ((1 << per_log2) - 1));
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int i = i0 + 32 * c, row = box_row(p, pc, i >> per_log2, i & ((1 << per_log2) - 1), id[c]);
        ks[c] = vs[c] = 0.f;  // exponent -127: does not count
        if (row >= 0) {
          ks[c] = kv.k_scale[row >> kv.page_log2];
          vs[c] = kv.v_scale[row >> kv.page_log2];
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int k = exponent(ks[c]), v = exponent(vs[c]);
        k_hi = max(k_hi, k);
        v_hi = max(v_hi, v);
        if (k > -100) k_lo = min(k_lo, k);
        if (v > -100) v_lo = min(v_lo, v);
      }
    }
    k_hi = __reduce_max_sync(0xffffffffu, k_hi);
    k_lo = __reduce_min_sync(0xffffffffu, k_lo);
    v_hi = __reduce_max_sync(0xffffffffu, v_hi);
    v_lo = __reduce_min_sync(0xffffffffu, v_lo);
    if (lane == 0) {
      sm.piece_scale[feed.i % kPieces] = PieceScale{k_hi, v_hi, (v_lo < v_hi - kWild ? 1 : 0) | (k_lo < k_hi - kWild ? 2 : 0)};
      mbar_arrive(&sm.scale_full[feed.i % kPieces]);
    }
    feed.done(sm, lane);
  }
}

// The codes' loader looks up the pages and scales of 32 boxes at a time, a lane each (16 to 4 blocks).  A block at a time was
// 1 to 2% slower (11,000 keys of 18 sequences, 16 heads of 94 rows: 244 us against 239; chunks of 8 streams: 88 against 87).
// The bf16 rows' loader has one lookup for each block and stays with it (2 sequences of 12,000 keys, 16 heads of 1,280 rows:
// 164 us against 167 with batches).
struct Batch {
  int boxes_log2, blocks;  // boxes of a block; blocks of a batch
  int blk, box;            // this lane's
  __device__ __forceinline__ Batch(const KvAttnParams& p, int lane)
      : boxes_log2(7 - p.box_log2), blocks(32 >> boxes_log2), blk(lane >> boxes_log2), box(lane & ((1 << boxes_log2) - 1)) {}
  // What the batch has for box i of its block k (box i < boxes of a block; else -1 as a row).
  template <typename T>
  __device__ __forceinline__ T of_block(T v, int k, int i) const {
    const T x = __shfl_sync(0xffffffffu, v, ((k << boxes_log2) + i) & 31);
    return i < (1 << boxes_log2) ? x : T(-1);
  }
};

// 8-bit, warp 0: every block's TMA boxes of codes into the ring of raw blocks, and its scales.
__device__ __forceinline__ void load_codes_role(const KvAttnParams& p, AttnSmem& sm, const CUtensorMap* mk, const CUtensorMap* mv, int lane) {
  constexpr int kStages = Ring<true>::kStages, kRaw = Ring<true>::kRaw;
  const KvView& kv = p.kv;
  Walk w = sm.walk;
  Piece pc = sm.pieces[0];
  const Batch b(p, lane);
  uint32_t n = 0, pieces = 0;
  bool ok = true;
  for (bool more = pc.blk1 >= 0; ok && more; more = w.next(p, pc)) {
    if (!publish(p, sm, pieces, pc, lane)) {
      ok = false;
      break;
    }
    // page entries are loaded two batches ahead, scales one
    auto scales = [&](int row, float& k, float& v) {
      k = v = 1.f;
      if (row >= 0) {
        k = kv.k_scale[row >> kv.page_log2];
        v = kv.v_scale[row >> kv.page_log2];
      }
    };
    float sk, sv, nk = 1.f, nv = 1.f;
    int rows = box_row(p, pc, pc.blk0 + b.blk, b.box, box_entry(p, pc, pc.blk0 + b.blk, b.box)), next = -1;
    int entry = box_entry(p, pc, pc.blk0 + b.blocks + b.blk, b.box);
    scales(rows, sk, sv);
    for (int blk = pc.blk0; blk < pc.blk1; ++blk, ++n) {
      const int k = (blk - pc.blk0) & (b.blocks - 1);
      if (k == 0) {
        if (blk > pc.blk0) {
          rows = next;
          sk = nk;
          sv = nv;
        }
        next = box_row(p, pc, blk + b.blocks + b.blk, b.box, entry);
        scales(next, nk, nv);
        entry = box_entry(p, pc, blk + 2 * b.blocks + b.blk, b.box);
      }
      const int row = b.of_block(rows, k, lane);
      const uint32_t slot = n % kRaw;
      if (n >= kRaw && !wait_all(p, sm, &sm.raw_empty[slot], ((n / kRaw) & 1) ^ 1)) {
        ok = false;
        break;
      }
      const int g = lane & 7, box = (16 * g) >> p.box_log2;
      const float of = b.of_block(sk, k, box), ov = b.of_block(sv, k, box);
      if (lane < 8) {
        sm.scale[n % kScales].of[lane] = of;
        sm.scale[n % kScales].of[8 + lane] = ov;
      }
      __syncwarp();
      issue_boxes(p, mk, mv, pc, row, sm.ring + kStages * 2 * kBlockBytes + slot * kBlockBytes, &sm.raw[slot], kD, lane);
    }
    ++pieces;
  }
  if (ok) publish(p, sm, pieces, pc, lane);
  for (uint32_t c = n > kRaw ? n - kRaw : 0; c < n; ++c) mbar_wait_drain(&sm.raw[c % kRaw], (c / kRaw) & 1, kDrainBudget);
}

// 8-bit, warps 4 to 7: the raw codes to fp16 rows of the stage, eight rows of 64 codes at a time.
__device__ __forceinline__ void convert_role(const KvAttnParams& p, AttnSmem& sm, int warp, int lane) {
  constexpr int kStages = Ring<true>::kStages, kRaw = Ring<true>::kRaw;
  const int c = lane & 3, rr = lane >> 2;
  const uint32_t at0 = rr * kRowBytes + (((2 * c) ^ rr) << 4), at1 = rr * kRowBytes + (((2 * c + 1) ^ rr) << 4);
  Feed feed;
  uint32_t n = 0;
  while (const Piece* next = feed.next(p, sm)) {
    const int blk0 = next->blk0, blk1 = next->blk1;
    if (!wait_all(p, sm, &sm.scale_full[feed.i % kPieces], (feed.i / kPieces) & 1)) return;
    const int top = (lane & 8) ? sm.piece_scale[feed.i % kPieces].v : sm.piece_scale[feed.i % kPieces].k;
    for (int blk = blk0; blk < blk1; ++blk, ++n) {
      const uint32_t st = n % kStages, slot = n % kRaw;
      const bool whole = whole_block(*next, blk);
      if (!wait_all(p, sm, &sm.raw[slot], (n / kRaw) & 1)) return;
      if (n >= kStages && !wait_all(p, sm, &sm.empty[st], ((n / kStages) & 1) ^ 1)) return;
      // lane g: what the keys of group g are multiplied by, lane 8 + g: the values
      const uint32_t factors = f16_power(exponent(sm.scale[n % kScales].of[lane & 15]) - top);
      const uint8_t* src = sm.ring + kStages * 2 * kBlockBytes + slot * kBlockBytes + lane * 16;
      uint8_t* dst = sm.ring + st * 2 * kBlockBytes;
#pragma unroll 1
      for (int u0 = warp; u0 < 32; u0 += 4 * kConverters) {  // K is units 0 to 15, V 16 to 31
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(src + (u0 + i * kConverters) * 512);
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * ((u0 + i * kConverters) & 15) + rr, ch = 2 * blk + (r >> 6);
            if (ch >= next->ch.total || !seen_by_some(next->runs, next->ch.key(ch) + (r & 63))) x[i] = make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int u = u0 + i * kConverters;
          const uint32_t f = __shfl_sync(0xffffffffu, factors, u >> 1);  // two units a group
          const uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t h[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[2 * j] = mul_f16x2(f16x2_of_e4m3(y[j]), f);
            h[2 * j + 1] = mul_f16x2(f16x2_of_e4m3(y[j] >> 16), f);
          }
          uint8_t* to = dst + u * 8 * kRowBytes;
          *reinterpret_cast<uint4*>(to + at0) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(to + at1) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.raw_empty[slot]);
        mbar_arrive(&sm.full[st]);
      }
    }
    feed.done(sm, lane);
  }
}

// ------------------------------------------------------------------ products

constexpr uint64_t kTileDesc = kBlockBytes >> 4, kStageDesc = 2 * kTileDesc;

// M = 128, N = 64, fp32 accumulators; fp16 operands, or bf16 ones
template <bool kF16>
__device__ constexpr uint32_t idesc_of(int b_mn) {
  return idesc_bf16_f32(128, 64, 0, b_mn) & ~(kF16 ? (1u << 7) | (1u << 10) : 0u);
}

// S of key half h: Q K^T for 64 keys
template <bool kF16>
__device__ __forceinline__ void issue_qk(uint64_t dq, uint64_t dk, uint32_t s_col) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) mma_ss(s_col, dq + 2 * kk, dk + 2 * kk, idesc_of<kF16>(0), kk > 0 ? 1u : 0u);
}

// One warp for each tile; the whole warp runs (which keeps the descriptors uniform), one elected lane issues.  A key
// half goes its own way (8-bit): as soon as its warps have written P, its O += P V is issued and S = Q K^T of its next 64
// keys behind it, over P.  One product of 128 keys for both halves would read Q from shared memory half as often
// (tensor time 1024 cycles of a block of 256 rows against 1264), but ties the halves together.
__device__ __forceinline__ void mma_role(const KvAttnParams& p, AttnSmem& sm, uint32_t tmem_base, int t, int lane) {
  constexpr int kStages = Ring<true>::kStages;
  const uint32_t tmem = __reduce_max_sync(0xffffffffu, tmem_base) + t * 256;
  const uint64_t q0 = smem_desc_sw128(smem_u32(sm.q[t]), 16, 1024);
  const uint64_t k0 = smem_desc_sw128(smem_u32(sm.ring), 16, 1024);
  const uint64_t v0 = smem_desc_sw128(smem_u32(sm.ring) + kBlockBytes, 8192, 1024);
  Feed feed;
  uint32_t n = 0, pieces = 0, pfull = 0;
  while (const Piece* pc = feed.next(p, sm)) {
    // a warp reduction's result is known to be uniform, so that counters and descriptors stay in uniform registers
    const int nblk = __reduce_max_sync(0xffffffffu, pc->blk1 - pc->blk0);
    const int rows = __reduce_max_sync(0xffffffffu, pc->rows);
    feed.done(sm, lane);
    if (rows <= t * 128) {  // the item has one tile: this warp lets everything go
      for (int j = 0; j < nblk; ++j, ++n) {
        if (!wait_all(p, sm, &sm.full[n % kStages], (n / kStages) & 1)) return;
        if (lane == 0) mbar_arrive(&sm.empty[n % kStages]);
      }
      continue;
    }
    if (!wait_all(p, sm, &sm.q_full[t], pieces & 1)) return;
    ++pieces;
    if (!wait_all(p, sm, &sm.full[n % kStages], (n / kStages) & 1)) return;
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        issue_qk<true>(q0, k0 + (n % kStages) * kStageDesc + h * (kTileDesc / 2), tmem + h * 64);
        mma_commit(&sm.s_full[t][h]);
      }
      if (nblk == 1) mma_commit(&sm.q_empty[t]);
    }
    __syncwarp();
    for (int j = 0; j < nblk; ++j, ++n) {
      const uint32_t cs = n % kStages, ns = (n + 1) % kStages;
      const bool more = j + 1 < nblk;
      const uint64_t dv = v0 + cs * kStageDesc, dk = k0 + ns * kStageDesc;
      if (more && !wait_all(p, sm, &sm.full[ns], ((n + 1) / kStages) & 1)) return;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait_all(p, sm, &sm.p_full[t][h], pfull & 1)) return;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t s_col = tmem + h * 64, o_col = s_col + 128;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(o_col, s_col + kk * 8, dv + 128 * (4 * h + kk), idesc_of<true>(1), j > 0 || kk > 0 ? 1u : 0u);
          if (more) {
            issue_qk<true>(q0, dk + h * (kTileDesc / 2), s_col);
            mma_commit(&sm.s_full[t][h]);
          }
          if (h == 1) {
            if (!more) mma_commit(&sm.o_done[t]);
            mma_commit(&sm.empty[cs]);
            if (j + 2 == nblk) mma_commit(&sm.q_empty[t]);
          }
        }
        __syncwarp();
      }
      ++pfull;
    }
  }
}

// bf16: the same with one accumulator for both key halves of a tile and three S buffers: a step is one key half of
// one block, step n of the tile has buffer n % 3, and a buffer whose P V is issued takes the S of the third step after.
__device__ __forceinline__ void mma_role_joint(const KvAttnParams& p, AttnSmem& sm, uint32_t tmem_base, int t, int lane) {
  constexpr uint32_t kStages = Ring<false>::kStages;
  const uint32_t tmem = __reduce_max_sync(0xffffffffu, tmem_base) + t * 256, o_col = tmem + 192;
  const uint64_t q0 = smem_desc_sw128(smem_u32(sm.q[t]), 16, 1024);
  const uint64_t k0 = smem_desc_sw128(smem_u32(sm.ring), 16, 1024);
  const uint64_t v0 = smem_desc_sw128(smem_u32(sm.ring) + kBlockBytes, 8192, 1024);
  Feed feed;
  uint32_t n = 0, pieces = 0;  // key blocks of all pieces, pieces of this tile
  uint32_t buf = 0, par = 0;     // of the next P
  while (const Piece* pc = feed.next(p, sm)) {
    const int nblk = __reduce_max_sync(0xffffffffu, pc->blk1 - pc->blk0);
    const int rows = __reduce_max_sync(0xffffffffu, pc->rows);
    feed.done(sm, lane);
    if (rows <= t * 128) {  // the item has one tile: this warp lets everything go
      for (int j = 0; j < nblk; ++j, ++n) {
        if (!wait_all(p, sm, &sm.full[n % kStages], (n / kStages) & 1)) return;
        if (lane == 0) mbar_arrive(&sm.empty[n % kStages]);
      }
      continue;
    }
    if (!wait_all(p, sm, &sm.q_full[t], pieces & 1)) return;
    ++pieces;
    const int steps = 2 * nblk;
    // S of the piece's step i into buffer b
    auto scores = [&](int i, uint32_t b) {
      const uint32_t blk = n + (i >> 1);
      if (!(i & 1) && !wait_all(p, sm, &sm.full[blk % kStages], (blk / kStages) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        issue_qk<false>(q0, k0 + (blk % kStages) * kStageDesc + (i & 1) * (kTileDesc / 2), tmem + b * 64);
        mma_commit(&sm.s_full[t][b]);
        if (i == steps - 1) mma_commit(&sm.q_empty[t]);
      }
      __syncwarp();
      return true;
    };
    for (int i = 0; i < 3 && i < steps; ++i)
      if (!scores(i, buf + i >= 3 ? buf + i - 3 : buf + i)) return;
    for (int i = 0; i < steps; ++i) {
      if (!wait_all(p, sm, &sm.p_full[t][buf], par)) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t cs = (n + (i >> 1)) % kStages;
        const uint64_t dv = v0 + cs * kStageDesc + 512 * (i & 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(o_col, tmem + buf * 64 + kk * 8, dv + 128 * kk, idesc_of<false>(1), i > 0 || kk > 0 ? 1u : 0u);
        if (i & 1) mma_commit(&sm.empty[cs]);
        if (i == steps - 1) mma_commit(&sm.o_done[t]);
      }
      __syncwarp();
      if (i + 3 < steps && !scores(i + 3, buf)) return;
      if (++buf == 3) {
        buf = 0;
        par ^= 1;
      }
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

// Largest logit that a row sees of a chunk.
__device__ __forceinline__ float row_largest(uint32_t tS, uint64_t valid) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t s[16];
    tmem_ld16(tS + 16 * c, s);
    tmem_wait_ld();
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if ((valid >> (16 * c + q)) & 1ull) mx = fmaxf(mx, __uint_as_float(s[q]));
  }
  return mx;
}

// Raises the rows' references to the largest logit of the chunk at least, and scales what was summed so far.  Returns
// whether some row still has none (it has seen no key yet).
__device__ __forceinline__ bool new_reference(uint32_t tS, uint32_t tO, bool first, uint64_t valid, float qs, float& m,
                                              float& l) {
  const float now = fmaxf(m, row_largest(tS, valid) * qs);
  const float alpha = now == m ? 1.f : fast_exp2(m - now);  // m may be -inf: alpha = 0
  m = now;
  l *= alpha;
  if (!first) rescale_o(tO, alpha);
  return __any_sync(0xffffffffu, now == -INFINITY);
}

// The largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 logits against the reference: weights as bf16 pairs, their sums into rp, the largest x of the polynomial into top.
template <bool kF16, uint32_t kPoly, bool kMask>
__device__ __forceinline__ void weights16(const uint32_t (&s)[16], uint32_t valid, float scale, float add, uint32_t* pk, float (&rp)[4],
                                          float& top) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float x0 = __uint_as_float(s[2 * q]), x1 = __uint_as_float(s[2 * q + 1]);
    ffma2(x0, x1, scale, add);
    if ((kPoly >> q) & 1u) {
      top = max3_nan(top, x0, x1);
      exp2_poly2(x0, x1, x0, x1);
    } else {
      x0 = fast_exp2(x0);
      x1 = fast_exp2(x1);
    }
    if (kMask) {
      x0 = (valid >> (2 * q)) & 1u ? x0 : 0.f;
      x1 = (valid >> (2 * q + 1)) & 1u ? x1 : 0.f;
    }
    fadd2(rp[2 * (q & 1)], rp[2 * (q & 1) + 1], x0, x1);
    pk[q] = kF16 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
  }
}

// A row's 64 logits, 16 at a time, the next 16 on their way; the first 16 were asked for into `a`.  Returns the sum of the
// weights, which holds only where top, the largest x that the polynomial took (-infinity: none; NaN if one was), is
// below 128.
template <bool kF16, bool kMask>
__device__ __forceinline__ float weights(uint32_t tS, uint64_t valid, float m, float qs, uint32_t (&a)[16], uint32_t (&pk)[32],
                                         float& top) {
  const float add = m == -INFINITY ? 0.f : -m;
  constexpr uint32_t kPoly = kMask ? 0u : kPolyPairs;
  const uint32_t lo = static_cast<uint32_t>(valid), hi = static_cast<uint32_t>(valid >> 32);
  float rp[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t b[16];
  top = -INFINITY;
  tmem_wait_ld();
  tmem_ld16(tS + 16, b);
  weights16<kF16, (kPoly & 0xffu), kMask>(a, lo, qs, add, pk, rp, top);
  tmem_wait_ld();
  tmem_ld16(tS + 32, a);
  weights16<kF16, ((kPoly >> 8) & 0xffu), kMask>(b, lo >> 16, qs, add, pk + 8, rp, top);
  tmem_wait_ld();
  tmem_ld16(tS + 48, b);
  weights16<kF16, ((kPoly >> 16) & 0xffu), kMask>(a, hi, qs, add, pk + 16, rp, top);
  tmem_wait_ld();
  weights16<kF16, (kPoly >> 24), kMask>(b, hi >> 16, qs, add, pk + 24, rp, top);
  return (rp[0] + rp[1]) + (rp[2] + rp[3]);
}

__device__ __forceinline__ const uint16_t* query_row(const KvAttnParams& p, const Piece& pc, int row) {
  const int a = pc.row0 + row, tok = p.by_group.div(a), head = pc.hk * p.group + a - tok * p.group;
  return p.q + (pc.s.row0 + tok) * p.q_ts + head * p.q_hs;
}
__device__ __forceinline__ void prefetch_row(const void* src) { asm volatile("prefetch.global.L1 [%0];" ::"l"(src)); }

// Half h of query row t * 128 + r of a piece, the tile's number i (by its softmax thread; the whole warp runs).  8-bit: as
// fp16 times a power of two of the row (the row's largest has exponent 0; values below 2^-14 of it lose bits, 2^-25 of it
// at most).
template <bool kF16>
__device__ __forceinline__ bool load_query(const KvAttnParams& p, AttnSmem& sm, const Piece& pc, uint32_t i, uint32_t slot, int t,
                                           int h, int r, int lane) {
  if (pc.rows <= t * 128 || p.q_tma) return true;
  if (i >= 1 && !wait_all(p, sm, &sm.q_empty[t], (i & 1) ^ 1)) return false;
  const int row = t * 128 + r;
  {
    uint4 x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = make_uint4(0, 0, 0, 0);
    uint32_t mx = 0;
    if (row < pc.rows) {
      const uint4* src = reinterpret_cast<const uint4*>(query_row(p, pc, row));
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = src[4 * h + c];
      if (kF16) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 y = c < 4 ? x[c] : src[4 * (h ^ 1) + c - 4];
          const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) mx = max(mx, max((v[j] >> 7) & 0xffu, (v[j] >> 23) & 0xffu));
        }
      }
    }
    const int e = mx == 0xff ? 0 : min(max(static_cast<int>(mx) - 127, -120), 120);  // an infinity or NaN stays one
    const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const uint32_t at = smem_u32(sm.q[t]) + r * kRowBytes;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      if (kF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pack_f16x2(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xffff0000u) * f);
      }
      st_shared16(at + (((4 * h + c) ^ (r & 7)) << 4), v[0], v[1], v[2], v[3]);
    }
    if (kF16) sm.q_exp[slot][row][h] = static_cast<int16_t>(e);
    fence_proxy_async_smem();
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.q_full[t]);
  return true;
}

// Columns 32h..32h+31 of a piece's row: to the output, or to the share's slot.  (Run by a whole warp.)
template <bool kE4m3>
__device__ __forceinline__ void finish_row(const KvAttnParams& p, const Piece& pc, int row, int h, int tok, float mm, float den, bool part,
                                           bool wild, const float (&o)[32], int lane) {
  if (pc.slot >= 0) {
    Slot& sl = reinterpret_cast<Work*>(p.ws)->slots[blockIdx.x][pc.slot];
    float4* d = reinterpret_cast<float4*>(&sl.o[row][32 * h]);
#pragma unroll
    for (int q = 0; q < 8; ++q) d[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    if (h == 0) {
      sl.m[row] = mm;
      sl.l[row] = den;
      sl.part[row] = (part ? 1 : 0) | (wild ? 2 : 0);
    }
    return;
  }
  const int a = pc.row0 + min(row, pc.rows - 1), head = pc.hk * p.group + a - tok * p.group;
  const bool live = row < pc.rows;
  bool nan = false, inf = false;
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    nan |= o[q] != o[q];
    inf |= fabsf(o[q]) == INFINITY;
  }
  const bool bad = (nan && part) || inf || wild;
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
  // a value out of the row's sight is not finite, or a sum of weights times values left fp32's range: key by key
  uint32_t todo = __ballot_sync(0xffffffffu, live && bad);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    const int tk = __shfl_sync(0xffffffffu, tok, src), hd = __shfl_sync(0xffffffffu, head, src);
    exact_row<kE4m3>(p, pc.b, pc.s.len, pc.s.row0 + tk, pc.s.len - pc.s.n_new + tk, hd, lane, 32 * h, 32 * h + 32);
  }
}

// The softmax of a tile whose key halves share a reference and an accumulator.  The halves' warps of 32 rows meet at a block
// only while some of those rows have seen no key yet (a piece's first block, rows whose window begins later).  The
// reference never moves after that: bf16 weights hold 2^64 over it, and a row beyond is done key by key.
__device__ __forceinline__ void softmax_role_joint(const KvAttnParams& p, AttnSmem& sm, uint32_t tmem, int sw, int lane) {
  const int t = sw >> 3, h = (sw >> 2) & 1, wq = sw & 3;
  const int r = wq * 32 + lane;  // row of the tile
  const uint32_t base = tmem + (static_cast<uint32_t>(wq * 32) << 16) + t * 256;
  bool withhold = p.withhold != 0 && blockIdx.x == 0 && sw == 0;  // test hook
  Feed feed;
  uint32_t pieces = 0;
  uint32_t buf = h, par = 0;  // this warp's next step
  uint32_t meet = 0;
  // the other half's value of this row
  auto exchange = [&](float2 mine, float2& other) {
    sm.stats[meet & 1][t][h][r] = mine;
    mbar_arrive(&sm.pair[t][wq]);
    if (!wait_all(p, sm, &sm.pair[t][wq], meet & 1)) return false;
    other = sm.stats[meet & 1][t][h ^ 1][r];
    ++meet;
    return true;
  };
  const Piece* next = feed.next(p, sm);
  if (next && !load_query<false>(p, sm, *next, 0, 0, t, h, r, lane)) return;
  while (next) {
    const Piece& pc = *next;
    // the next piece's queries, before this one's end
    auto look_ahead = [&]() {
      Feed f = feed;
      ++f.i;
      next = f.next(p, sm);
      return !next || load_query<false>(p, sm, *next, pieces, f.i % kPieces, t, h, r, lane);
    };
    if (pc.rows <= t * 128) {  // the item has one tile
      if (!look_ahead()) return;
      feed.done(sm, lane);
      continue;
    }
    const int a = pc.row0 + min(t * 128 + r, pc.rows - 1), tok = p.by_group.div(a);
    const Span sp = span_of(p.win, pc.s.len - pc.s.n_new + tok, pc.s.len);
    float m = -INFINITY, l = 0.f;
    bool unset = true;  // some row of the two warps has no reference yet
    int flags = 0;      // 1: some streamed key is out of this row's sight, 2: weights beyond bf16's comfort
    const Chunks ch = pc.ch;
    const int blk0 = pc.blk0, blk1 = pc.blk1;
    // what every row of the warp sees
    const int all_lo = __reduce_max_sync(0xffffffffu, sp.lo), all_hi = __reduce_min_sync(0xffffffffu, sp.hi);
    const int all_sink = __reduce_min_sync(0xffffffffu, sp.sink);
    uint32_t first16[16];  // of the next S, on their way
    auto start = [&]() {
      if (!wait_all(p, sm, &sm.s_full[t][buf], par)) return false;
      tc_fence_after();
      tmem_ld16(base + buf * 64, first16);
      return true;
    };
    if (!start()) return;
    for (int blk = blk0;;) {
      const int i = 2 * blk + h, j0 = ch.key(i);
      const bool have = i < ch.total;
      const bool all = have && ((j0 >= all_lo && j0 + 64 <= all_hi) || j0 + 64 <= all_sink);
      uint64_t valid = ~0ull;
      if (!all) {
        valid = have ? range_bits(sp.lo - j0, sp.hi - j0) | range_bits(0, sp.sink - j0) : 0ull;
        if (have && valid != ~0ull) flags |= 1;
      }
      const uint32_t tS = base + buf * 64;
      const bool none = !all && __all_sync(0xffffffffu, valid == 0ull);
      if (unset) {
        tmem_wait_ld();
        const float2 mine = make_float2(none ? -INFINITY : row_largest(tS, valid) * kScaleLog2, 0.f);
        float2 other;
        if (!exchange(mine, other)) return;
        if (m == -INFINITY) m = fmaxf(mine.x, other.x);
        unset = __any_sync(0xffffffffu, m == -INFINITY);
      }
      uint32_t pk[32];
      if (none) {
        // no row of this warp sees a key of the chunk
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 32; ++q) pk[q] = 0u;
      } else {
        float top;
        const float sum = all ? weights<false, false>(tS, valid, m, kScaleLog2, first16, pk, top)
                              : weights<false, true>(tS, valid, m, kScaleLog2, first16, pk, top);
        if (sum > kGrow || top > kGrowLog2) flags |= 2;
        l += top == top ? sum : top;
      }
      tmem_st32(tS, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (withhold)
        withhold = false;
      else if (lane == 0)
        mbar_arrive(&sm.p_full[t][buf]);
      buf += 2;
      if (buf >= 3) {
        buf -= 3;
        par ^= 1;
      }
      if (++blk == blk1) break;
      if (!start()) return;
      if (blk + 1 == blk1 && !p.q_tma && mbar_try_wait(&sm.piece_full[(feed.i + 1) % kPieces], ((feed.i + 1) / kPieces) & 1)) {
        const Piece& nx = sm.pieces[(feed.i + 1) % kPieces];  // its queries, on their way to the caches
        if (nx.blk1 >= 0 && t * 128 + r < nx.rows) prefetch_row(query_row(p, nx, t * 128 + r));
      }
    }
    const uint32_t done = pieces & 1;
    ++pieces;
    if (!look_ahead()) return;
    float2 other;
    if (!exchange(make_float2(l, __int_as_float(flags)), other)) return;
    if (!wait_all(p, sm, &sm.o_done[t], done)) return;
    tc_fence_after();
    flags |= __float_as_int(other.y);
    const float den = l + other.x, scale = den == 0.f ? (pc.slot >= 0 ? 0.f : no_weight()) : 1.f / den;
    float o[32];
    {
      uint32_t x[32];
      tmem_ld32(base + 192 + 32 * h, x);
      tmem_wait_ld();
      tc_fence_before();
#pragma unroll
      for (int q = 0; q < 32; ++q) o[q] = __uint_as_float(x[q]) * scale;
    }
    finish_row<false>(p, pc, t * 128 + r, h, tok, m, den, (flags & 1) != 0, (flags & 2) != 0, o, lane);
    feed.done(sm, lane);
  }
}

// 8-bit: a reference and an accumulator for each key half.
__device__ __forceinline__ void softmax_role(const KvAttnParams& p, AttnSmem& sm, uint32_t tmem, int sw, int lane) {
  const int t = sw >> 3, h = (sw >> 2) & 1, wq = sw & 3;
  const int r = wq * 32 + lane;  // row of the tile
  const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t tS = tmem + lane_off + t * 256 + h * 64, tO = tmem + lane_off + t * 256 + 128;
  bool withhold = p.withhold != 0 && blockIdx.x == 0 && sw == 0;  // test hook
  Feed feed;
  uint32_t sfull = 0, pieces = 0, n = 0;  // pieces of this tile, key blocks of all
  const Piece* next = feed.next(p, sm);
  if (next && !load_query<true>(p, sm, *next, 0, 0, t, h, r, lane)) return;
  while (next) {
    const Piece& pc = *next;
    const uint32_t slot = feed.i % kPieces;
    // the next piece's queries, before this one's end
    auto look_ahead = [&]() {
      Feed f = feed;
      ++f.i;
      next = f.next(p, sm);
      return !next || load_query<true>(p, sm, *next, pieces, f.i % kPieces, t, h, r, lane);
    };
    if (pc.rows <= t * 128) {  // the item has one tile
      n += pc.blk1 - pc.blk0;
      if (!look_ahead()) return;
      feed.done(sm, lane);
      continue;
    }
    const int a = pc.row0 + min(t * 128 + r, pc.rows - 1), tok = p.by_group.div(a);
    const Span sp = span_of(p.win, pc.s.len - pc.s.n_new + tok, pc.s.len);
    float m = -INFINITY, l = 0.f;
    bool unset = false;  // some row of the warp has no reference yet
    bool part = false;  // some streamed key is out of this row's sight
    const Chunks ch = pc.ch;
    const int blk0 = pc.blk0, blk1 = pc.blk1;
    float qs = 0.f;  // what a product is multiplied by: known once the queries are there
    for (int blk = blk0; blk < blk1; ++blk, ++n) {
      const int i = 2 * blk + h, j0 = ch.key(i);
      const bool have = i < ch.total;
      const bool whole = have && ((j0 >= sp.lo && j0 + 64 <= sp.hi) || j0 + 64 <= sp.sink);
      const bool all = __all_sync(0xffffffffu, whole);
      uint64_t valid = ~0ull;
      if (!all) {
        valid = have ? range_bits(sp.lo - j0, sp.hi - j0) | range_bits(0, sp.sink - j0) : 0ull;
        part |= have && !whole;
      }
      if (blk + 2 == blk1 && mbar_try_wait(&sm.piece_full[(feed.i + 1) % kPieces], ((feed.i + 1) / kPieces) & 1)) {
        const Piece& nx = sm.pieces[(feed.i + 1) % kPieces];  // its queries, on their way to the caches
        if (nx.blk1 >= 0 && t * 128 + r < nx.rows) prefetch_row(query_row(p, nx, t * 128 + r));
      }
      if (!wait_all(p, sm, &sm.s_full[t][h], sfull & 1)) return;
      ++sfull;
      tc_fence_after();
      if (blk == blk0) {
        const int e = sm.q_exp[slot][t * 128 + r][h] + sm.piece_scale[slot].k - kCodeTop;
        qs = kScaleLog2 * __uint_as_float(static_cast<uint32_t>(127 + min(max(e, -126), 127)) << 23);
      }
      uint32_t pk[32];
      if (!all && __all_sync(0xffffffffu, valid == 0ull)) {
        // no row of this warp sees a key of the chunk
#pragma unroll
        for (int q = 0; q < 32; ++q) pk[q] = 0u;
        unset |= blk == blk0;
      } else {
        const bool first = blk == blk0;
        bool raise = first || unset;
        float sum, top;
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          if (raise) unset = new_reference(tS, tO + h * 64, first, valid, qs, m, l);
          uint32_t first16[16];
          tmem_ld16(tS, first16);
          sum = all ? weights<true, false>(tS, valid, m, qs, first16, pk, top) : weights<true, true>(tS, valid, m, qs, first16, pk, top);
          // far above the reference, or not a number
          raise = __any_sync(0xffffffffu, !(sum <= kGrowF16) || top > kGrowF16Log2);
          if (!raise || pass == 1) break;
        }
        l += top == top ? sum : top;
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
    const uint32_t par = pieces & 1;
    ++pieces;
    if (!look_ahead()) return;
    // join the two key halves; this thread finishes columns 32h..32h+31 of its row
    sm.stats[par][t][h][r] = make_float2(m, part ? -l - 1e-30f : l);  // the sign says that some keys are out of sight
    mbar_arrive(&sm.pair[t][wq]);
    if (!wait_all(p, sm, &sm.o_done[t], par)) return;
    if (!wait_all(p, sm, &sm.pair[t][wq], par)) return;
    tc_fence_after();
    const float2 other = sm.stats[par][t][h ^ 1][r];
    const float mo = other.x, lo = fabsf(other.y);
    part |= other.y < 0.f;
    const int wild_scales = sm.piece_scale[slot].wild;
    const bool wild = (wild_scales & 1) || ((wild_scales & 2) && qs > kQuiet);
    const float mm = fmaxf(m, mo);
    const float fm = m == -INFINITY ? 0.f : fast_exp2(m - mm), fo = mo == -INFINITY ? 0.f : fast_exp2(mo - mm);
    const float den = l * fm + lo * fo;
    float scale = den == 0.f ? (pc.slot >= 0 ? 0.f : no_weight()) : 1.f / den;
    scale *= __uint_as_float(static_cast<uint32_t>(127 + max(sm.piece_scale[slot].v - kCodeTop, -126)) << 23);
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
    finish_row<true>(p, pc, t * 128 + r, h, tok, mm, den, part, wild, o, lane);
    feed.done(sm, lane);
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(32 * Ring<kE4m3>::kWarps, 1)
    kv_attn_kernel(const __grid_constant__ KvAttnParams p, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q) {
  extern __shared__ uint8_t smem_raw[];
  AttnSmem& sm = *reinterpret_cast<AttnSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 96) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sm.full[s], kE4m3 ? kConverters : 2);
      mbar_init(&sm.empty[s], 2);
      mbar_init(&sm.raw[s], 1);
      mbar_init(&sm.raw_empty[s], kConverters);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < kPieces / 2; ++i) {
        mbar_init(&sm.piece_full[2 * i + t], 1);
        mbar_init(&sm.piece_empty[2 * i + t], Ring<kE4m3>::kWarps - 1);
        mbar_init(&sm.scale_full[2 * i + t], 1);
      }
      mbar_init(&sm.q_full[t], p.q_tma ? 1 : 8);
      mbar_init(&sm.q_empty[t], 1);
      mbar_init(&sm.drain[t], 1);
      mbar_init(&sm.o_done[t], 1);
      for (int h = 0; h < 3; ++h) {
        mbar_init(&sm.s_full[t][h], 1);
        mbar_init(&sm.p_full[t][h], 4);
      }
      for (int w = 0; w < 4; ++w) mbar_init(&sm.pair[t][w], 64);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    __syncwarp();
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  make_plan(p, sm.walk, sm.pieces[0], reinterpret_cast<long long*>(sm.ring));  // the ring is not in use yet
  if (threadIdx.x == 0) mbar_arrive(&sm.piece_full[0]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // registers: launched with 96 x 640 or 80 x 768; 64 x 128 + 104 x 512 and 64 x 256 + 88 x 512 are as many
  if (warp < Ring<kE4m3>::kSoftmax) {
    reg_dealloc_dec<64>();
    if (kE4m3 && warp >= 4) {
      convert_role(p, sm, warp - 4, lane);
    } else if (warp >= 2) {
      if constexpr (kE4m3)
        mma_role(p, sm, tmem, warp - 2, lane);
      else
        mma_role_joint(p, sm, tmem, warp - 2, lane);
      // also after a wait that gave up: no product is in flight when the block lets its memory go
      if (elect_one()) mma_commit(&sm.drain[warp - 2]);
      __syncwarp();
      mbar_wait_drain(&sm.drain[warp - 2], 0, kDrainBudget);
    } else if (kE4m3 && warp == 0) {
      load_codes_role(p, sm, &map_k, &map_v, lane);
    } else if (!kE4m3 && warp == 0) {
      load_role(p, sm, &map_k, &map_v, lane);
    } else if (kE4m3) {
      scan_role(p, sm, lane);
    } else {
      side_role(p, sm, &map_q, lane);
    }
  } else {
    if (kE4m3)
      reg_alloc_inc<88>();
    else
      reg_alloc_inc<104>();
    if constexpr (kE4m3)
      softmax_role(p, sm, tmem, warp - Ring<kE4m3>::kSoftmax, lane);
    else
      softmax_role_joint(p, sm, tmem, warp - Ring<kE4m3>::kSoftmax, lane);
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
template <bool kE4m3>
__global__ void __launch_bounds__(256) kv_join_kernel(const __grid_constant__ KvAttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Work& wk = *reinterpret_cast<const Work*>(p.ws);
  const Cut& cut = wk.cuts[blockIdx.x + 1];
  const int r = blockIdx.y * 32 + (threadIdx.x >> 3), col = (threadIdx.x & 7) * 8, lane = threadIdx.x & 31;
  if (!cut.valid || blockIdx.y * 32 >= cut.rows) return;
  float mm = -INFINITY, l = 0.f, o[8];
  bool part = false, wild = false, nan = false;  // nan: in a piece's answer
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  int b0 = 0;
  for (int c = blockIdx.x; b0 < cut.nblk; ++c) {
    const int b1 = blocks_before(share_start(cut.each, cut.extra, c + 1) - cut.x0, cut.nblk, cut.unit);
    if (b1 > b0) {
      const Slot& sl = wk.slots[c][b0 > 0 ? 0 : 1];
      const float m = sl.m[r], nm = fmaxf(mm, m);
      const float f = mm == -INFINITY ? 0.f : fast_exp2(mm - nm), g = m == -INFINITY ? 0.f : fast_exp2(m - nm) * sl.l[r];
      const float4* src = reinterpret_cast<const float4*>(&sl.o[r][col]);
      const float4 x = src[0], y = src[1];
      o[0] = o[0] * f + x.x * g; o[1] = o[1] * f + x.y * g; o[2] = o[2] * f + x.z * g; o[3] = o[3] * f + x.w * g;
      nan |= x.x != x.x || x.y != x.y || x.z != x.z || x.w != x.w || y.x != y.x || y.y != y.y || y.z != y.z || y.w != y.w;
      o[4] = o[4] * f + y.x * g; o[5] = o[5] * f + y.y * g; o[6] = o[6] * f + y.z * g; o[7] = o[7] * f + y.w * g;
      l = l * f + g;
      part |= (sl.part[r] & 1) != 0;
      wild |= (sl.part[r] & 2) != 0;
      mm = nm;
    }
    b0 = b1;
  }
  const float inv = l == 0.f ? no_weight() : 1.f / l;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i] *= inv;
    bad |= !(fabsf(o[i]) <= 3.402823466e+38f);
  }
  // a row is exact as a whole: its 8 threads agree.  (Not finite though no piece holds a NaN: the sum left fp32's range.)
  const bool live = r < cut.rows;
  uint32_t todo = __ballot_sync(0xffffffffu, live && ((bad && (part || !nan)) || wild));
  const bool mine = ((todo >> (lane & 24)) & 0xffu) != 0;
  const int a = cut.row0 + r, tok = p.by_group.div(a), head = cut.hk * p.group + a - tok * p.group;
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
    exact_row<kE4m3>(p, cut.b, cut.len, cut.first + tk, cut.len - cut.n_new + tk, hd, lane, 0, kD);
  }
}

}  // namespace

size_t attn_workspace_bytes() { return sizeof(Work); }

saf3r_status launch_attn(const KvAttnParams& p0, cudaStream_t stream, int* n_launch) {
  KvAttnParams p = p0;
  const KvView& kv = p.kv;
  CUtensorMap mk, mv;
  bool ok;
  if (p.ck) {
    p.box_log2 = 6;
    const long long head = static_cast<long long>(kv.n_tokens) * kD;
    ok = make_map_rows(&mk, p.ck, kv.n_tokens, kD, kv.n_heads, head, 64) &&
         make_map_rows(&mv, p.cv, kv.n_tokens, kD, kv.n_heads, head, 64);
  } else {
    p.box_log2 = kv.page_log2 < 6 ? kv.page_log2 : 6;
    const int box = 1 << p.box_log2;
    const long long rows = static_cast<long long>(kv.n_pages) * kv.n_heads * kv.page;
    ok = p.e4m3 ? make_map_codes(&mk, kv.k, rows, box, false) && make_map_codes(&mv, kv.v, rows, box, false)
                : make_map_rows(&mk, kv.k, rows, kD, 1, rows * kD, box) && make_map_rows(&mv, kv.v, rows, kD, 1, rows * kD, box);
  }
  // queries by TMA: 64 rows are whole tokens of a group (bf16 products only: 8-bit caches want them as fp16)
  CUtensorMap mq = mk;
  p.q_tma = !p.e4m3 && p.group <= 64 && (p.group & (p.group - 1)) == 0 &&
            make_map_queries(&mq, p.q, p.group, kv.n_tokens, kv.n_heads, p.q_ts, p.q_hs, 64 / p.group);
  if (!ok) return SAF3R_ERR_CUDA;
  const int smem = static_cast<int>(sizeof(AttnSmem) + 1024);
  const auto kernel = p.e4m3 ? kv_attn_kernel<true> : kv_attn_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return SAF3R_ERR_CUDA;
  const int grid = p.num_sms < kMaxShares ? p.num_sms : kMaxShares;
  kernel<<<grid, 32 * (p.e4m3 ? Ring<true>::kWarps : Ring<false>::kWarps), smem, stream>>>(p, mk, mv, mq);
  ++*n_launch;
  if (cudaGetLastError() != cudaSuccess) return SAF3R_ERR_CUDA;
  if (grid > 1) {
    if (launch_behind(p.e4m3 ? kv_join_kernel<true> : kv_join_kernel<false>, dim3(grid - 1, kItem / 32), dim3(256), stream, p) != cudaSuccess)
      return SAF3R_ERR_CUDA;
    ++*n_launch;
  }
  return SAF3R_OK;
}

}  // namespace saf3r
