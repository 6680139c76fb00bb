// Absorbed-MLA decode over INT4 pages: for every new token and head s_j = scale (q~ . c_j + q^R . k^R_j) over
// the keys it may see, out = sum_j softmax(s)_j c_j, lse = ln sum_j exp(s_j), where the latent c_j is
// held as 512 four-bit codes n and 16 scales, c = (n - 8) scale  ("MLA inference: two computation paths and
// FlashMLA", section "Decode attention becomes a compute problem").
//
// What bounds it: a key is 416 bytes and 2176 FLOP for each row (token and head) that reads it, so up to ~50 rows a key
// HBM, beyond that the tensor cores; and a key's 512 values have to become bf16 in every SM that reads it.
//
// Work split.  The keys are the M dimension: S^T = K Q^T and O^T = C^T P^T.  A tile is a page, 64 keys, expanded once
// by a CTA that needs no other's help: up to 64 rows are its N = 16, 32, 48 or 64 columns, O^T is 4 x [128 dims x N] in tensor
// memory.  A unit of the plan is one CTA, or two for 65 to 128 heads, which read the same pages at the same time (the
// second from L2).  With several new tokens a sequence, groups of them of up to 64 rows share every
// key; a group's number of tokens divides s_q.
//
// That one copy is both products' A operand: blocks [64 keys][64 dims] of shared memory with the 128-byte swizzle, K-major for the
// scores (M = 64), MN-major for the output (M = 128 dims).  MMAs of K = 16 take 32 / 32 / 37 cycles for the scores, 44 / 44 / 50
// for the output (N = 16 / 32 / 64).  What bounds a tile is the way to shared memory: for N = 16 / 48 / 64 the tensor cores read their
// operands in 1306 / 1725 / 1928 passes of 128 bytes (A's are ~1095 of them), the warps load and store in 1279 / 1549 / 1649, together 2585 / 3274 /
// 3577 of the 2690 / 3870 / 3790 cycles that a tile takes (counters of a launch; the tile's time from its growth with the length, at
// 2070 MHz).  (The scores' A in tensor
// memory is read without it, at 12 to 32 cycles an MMA, but beside the expanding warps' stores there they took 53, and the output's
// MMAs 70: 64 streams x 16 heads 87 us instead of 83, 128 heads ragged 218 instead of 153.)
// Beyond its tiles a call takes 11 / 14 / 18 us (launch, the first page and queries, the last tile's way out, the merge's launch), and a
// unit's every further piece 5.6 / 8.0 / 12.6 us, four to seven tiles: the plan's price of a piece is six.
//
// Pages come by bulk copies into shared memory, as they are.  (Loads into registers, 64 bytes of a row at a time, kept the load
// units busy for ~1500 cycles a page.  A second page ahead changed nothing.)  The four quarters of a tile (128 dims each) are
// expanded by four warps each into a ring of quarters of 16 KB, eight up to 32 rows, seven for 48, six for 64: there the next tile's first ones are
// expanded and multiplied with the queries while the softmax works (with four: 178 us instead of 153).
//
// The scores' 64 rows are lanes 0..15 of each of tensor memory's four quadrants; the 16-lane loads deal a row of columns out to
// four lanes in turn: lane j of a quad has rows 4 b + j of the block, and its weights are neighbours in P, so that row 4 b + j of a
// warpgroup is column j NC / 4 + b of P and O^T.
//
// Roles (warps): softmax (a warpgroup for 16 columns, for N = 64 for 32; a row's maximum lies across lanes and
// warps, so scores are taken against the maximum so far, and only where one exceeds it by 2^8 are the new maxima found and O
// rescaled); 16 warps expand; one copies pages and queries and writes the tiles' records; a thread of the last issues the MMAs.
//
// Measured: 64 streams x 16 heads, 190 MB of cache, 82 us; 128 heads, 64 ragged sequences up to 32,768 keys (142 MB) 151 us, 4 up to
// 131,072 (94 MB) 114 us; 24 sequences of 4 tokens x 20 heads (36 MB) 55 us (with
// 64 columns 59).  64 x 8192 keys, 218 MB: 16 heads 90 us, 32 99, 40 127, 64 130, 128 235.  At 65 to 128 heads the decode of the same
// lengths over bf16 pages is the faster one (148 us), and so is that over FP8 pages (193 us): each of the two CTAs here expands all
// 512 dims of a page, each of a pair's there has its own half of them.  Up to 64 heads this one is (16 heads: 138 and 184 us).
// Registers: n48 spills 20 bytes (44 loaded back), n64 8 (44); n16 and n32 none.
#pragma once
#include "common.cuh"
#include "decode_kernel.cuh"  // packed float pairs, bf16 packing
#include "int4_rows.cuh"

namespace mla {

constexpr int kI4MaxRows = 64;           // rows of a CTA
constexpr int kI4Tile = 64;              // keys of a tile
constexpr int kI4Ahead = 4;              // tile records in shared memory
constexpr uint32_t kI4Page = 64 * kI4Row;
constexpr uint32_t kI4Blk = 8192;        // [64 keys][64 dims] bf16, 128-byte swizzle
constexpr uint32_t kI4Slot = 2 * kI4Blk;
static_assert(kI4Tile == kTile, "a tile of the plan is a page");

template <int N>
struct I4Smem {
  static constexpr int kWg = N == 64 ? 2 : N / 16;               // softmax warpgroups (64: four would be 34 warps)
  static constexpr int kNc = N / kWg;                            // columns of each
  static constexpr int kThreads = 128 * kWg + 576;
  static constexpr int kSlots = N == 64 ? 6 : N == 48 ? 7 : 8;  // a ring of quarter tiles
  static constexpr int kP = N > 32 ? 1 : 2;                      // tiles' weights
  static constexpr uint32_t V = 0;
  static constexpr uint32_t kPRow = N > 32 ? 128 : 2 * N;        // bytes of a key's weights
  static constexpr uint32_t R = V + kSlots * kI4Slot;            // RoPE keys: [tile parity] a block
  static constexpr uint32_t Q = R + 2 * kI4Blk;                  // 9 blocks [N rows][64 dims]
  static constexpr uint32_t P = Q + 9 * N * 128;                 // [kP][64 keys][kPRow]
  static constexpr uint32_t RAW = P + kP * 64 * kPRow;              // a page as it came
  static constexpr uint32_t FLAG = RAW + kI4Page;          // [tile parity][warp]: some score is far above the maximum
  static constexpr uint32_t MAX = FLAG + 32 * kWg;         // [warp][kNc]: the running maxima, log2 units
  static constexpr uint32_t FAC = MAX + 4 * kWg * kNc * 4;       // [warp][kNc]: factors of a rescale or of the output
  static constexpr uint32_t XCH = FAC + 4 * kWg * kNc * 4;       // [maxima, sums][warpgroup][warp][kNc]
  static constexpr uint32_t POISON = XCH + 8 * kWg * kNc * 4;    // [tile % 4][warpgroup][64 keys]
  static constexpr uint32_t RING = POISON + 256 * kWg;     // kI4Ahead tile records of 32 bytes
  static constexpr uint32_t BAR = RING + 32 * kI4Ahead;
  static constexpr uint32_t kBytes = BAR + 512 + 1024;           // + alignment slack
  static_assert(kBytes <= 232448, "shared memory");
};

enum : uint32_t {
  IB_FULL = 0,               // six or seven slots: + slot, else + tile parity: one arrival per expanding warp
  IB_EMPTY = IB_FULL + 7,    // + slot: the output product has read it
  IB_RAW = IB_EMPTY + 8,     // landed
  IB_RAW_EMPTY,              // one arrival per expanding warp
  IB_Q_FULL,
  IB_Q_EMPTY,
  IB_S_FULL,                 // + tile parity
  IB_P_FULL = IB_S_FULL + 2, // + tile parity: one arrival per softmax warp
  IB_FLAG = IB_P_FULL + 2,   // + 2 warpgroup + tile parity: one arrival per warp
  IB_XCH = IB_FLAG + 6,      // + warpgroup
  IB_TILE = IB_XCH + 3,      // + record: written
  IB_TILE_READ = IB_TILE + kI4Ahead,  // + record: one arrival per softmax warp, the last readers
  IB_DRAIN = IB_TILE_READ + kI4Ahead,
  kI4Bars = IB_DRAIN + 1
};
constexpr uint32_t kI4TmemSlot = 8 * kI4Bars, kI4Abort = kI4TmemSlot + 4;
static_assert(kI4Abort + 4 <= 512, "barrier area");

enum I4Site : int { kSiteI4Ring = 44, kSiteI4Q, kSiteI4Scores, kSiteI4Pv, kSiteI4Flag, kSiteI4Drain, kSiteI4Tile, kSiteI4Raw };

struct Int4Args {
  CUtensorMap map_q;     // q~ rows: bf16 {64, rows, 8 blocks 128 bytes apart}, box {64, N, 8}, 128-byte swizzle
  CUtensorMap map_qr;    // q^R rows: bf16 {64, rows}, box {64, N}
  const uint8_t* kv;
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* sched;
  void* out;
  float* lse;
  float* o_acc;          // split partials [slots][H][512], normalised
  float* lse_acc;        // [slots][H]
  float scale_log2;
  int32_t H, s_q, causal, max_pages, num_pages, out_f32, num_units, num_qb, group;
  int32_t parts, part_rows;  // CTAs of a unit, rows of each
  uint64_t timeout_ns;
};

// A tile's record, as it lies in shared memory.
struct I4Tile {
  int flags, nkeys;      // the tile has keys 0 .. nkeys - 1 of the page
  int some;              // keys of the tile that every token of the block sees (may lie outside 0 .. nkeys)
  int wb, split;
  enum { kValid = 1, kFirst = 2, kLast = 4 };  // first, last: of the unit's piece of the block
  __device__ bool valid() const { return flags & kValid; }
  __device__ bool first() const { return flags & kFirst; }
  __device__ bool last() const { return flags & kLast; }
};

// Walks the unit's tiles in order, across blocks.
struct I4Cursor {
  const int32_t* seqlens;
  int s_q, causal, G, wb0, tile0, wb1, tile1, split0, wb, t, end, vis, seq;
  __device__ void init(const Int4Args& a, const int32_t* rec) {
    seqlens = a.seqlens;
    s_q = a.s_q;
    causal = a.causal;
    G = a.group;
    wb0 = rec[0];
    tile0 = rec[1];
    wb1 = rec[2];
    tile1 = rec[3];
    split0 = rec[4];
    wb = wb0 - 1;
    t = end = 0;
  }
  __device__ bool next(I4Tile& r) {
    r.flags = 0;
    while (t >= end) {
      if (++wb > wb1) return false;
      const int qb = wb * G + G - 1;
      seq = qb / s_q;
      vis = visible_keys(seqlens[seq], s_q, qb % s_q, causal);
      t = wb == wb0 ? tile0 : 0;
      end = wb == wb1 ? tile1 : num_tiles(vis);
      r.flags = I4Tile::kFirst;
    }
    r.wb = wb;
    r.split = wb == wb0 ? split0 : 0;
    r.nkeys = min(vis - kTile * t, kI4Tile);
    r.some = vis - (causal ? G - 1 : 0) - kTile * t;
    ++t;
    r.flags |= I4Tile::kValid | (t >= end ? I4Tile::kLast : 0);
    return true;
  }
  __device__ int page() const { return t - 1; }  // of the tile that next() gave
};

// 16 lanes x 2 K columns of tensor memory and a warp, K = 8 or 16 values a lane: lane l gets, in r[2 b + h], column 4 b + l % 4 of
// lane l / 4 + 8 h.
template <int K>
__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t (&r)[K]) {
  if constexpr (K == 8) {
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    static_assert(K == 16, "values");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {  // multiples of 16
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void lds128f(uint32_t a, float& x, float& y, float& z, float& w) {
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x), "=f"(y), "=f"(z), "=f"(w) : "r"(a) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts32f(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

// The bounded waits of common.cuh in one piece; the timer is asked late, and rarely.
__device__ __forceinline__ bool i4_wait_warp(uint32_t bar, uint32_t parity, const WaitCtx& w, int site) {
  bool ok = true;
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 255) == 0) {
      if (*w.abort_local) {
        ok = false;
        break;
      }
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > w.timeout_ns) {
        raise_abort(w, site);
        ok = false;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// By one thread, which asks without being suspended and does other work meanwhile: busy() does a piece of it, or gives false.
template <class Busy>
__device__ __forceinline__ bool i4_wait_busy(uint32_t bar, uint32_t parity, const WaitCtx& w, int site, Busy busy) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (busy()) continue;
    if (mbar_test_wait(bar, parity)) return true;
    if ((i & 1023) == 0) {
      if (*w.abort_local) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > w.timeout_ns) {
        raise_abort(w, site);
        return false;
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void decode_int4_body(const Int4Args& args) {
  using S = I4Smem<N>;
  constexpr int NC = S::kNc, B = NC / 4, kSlots = S::kSlots;  // B: columns of a lane
  constexpr bool kWhole = kSlots >= 8;  // two tiles fit: their scores wait for whole ones
  constexpr uint32_t TO = 0, TS = 4 * N;  // tensor memory: O^T, two score buffers
  static_assert(TS + 2 * N <= 512, "tensor memory");
  constexpr int kExpand = 4 * S::kWg, kIssue = kExpand + 16;  // first warps of the roles
  extern __shared__ uint8_t i4_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(i4_smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / args.parts, part = blockIdx.x % args.parts;
  auto bar = [&](uint32_t i) { return base + S::BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::BAR + kI4Abort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::BAR + kI4TmemSlot);

  if (tid == 0) {
    for (uint32_t i = 0; i < kI4Bars; ++i) {
      uint32_t count = 1;
      if (i < IB_EMPTY) count = kWhole ? 16 : 4;
      if (i == IB_RAW_EMPTY) count = 16;
      if (i == IB_P_FULL || i == IB_P_FULL + 1 || (i >= IB_TILE_READ && i < IB_DRAIN)) count = 4 * S::kWg;
      if (i >= IB_FLAG && i < IB_TILE) count = 4;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (tid < 64 * S::kWg) asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + S::POISON + 4 * tid), "r"(0u) : "memory");
  if (warp == kIssue + 1) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (tid == 0) {
    prefetch_tensormap(&args.map_q);
    prefetch_tensormap(&args.map_qr);
  }
  pdl_wait_prerequisites();
  const int32_t* sched = args.sched;
  const bool bad_meta = sched[0] != kSchedMagic || sched[1] != args.num_units || sched[2] != args.num_qb || sched[5] != args.group;
  const int32_t* rec = sched + kSchedHeader + kUnitInts * unit;
  const bool idle = bad_meta || rec[0] < 0;
  if (bad_meta && tid == 0) atomicCAS(&g_mla_error, 0, 5);
  pdl_launch_dependents();
  WaitCtx wc;
  wc.abort_local = abort_flag;
  wc.abort_peer = 0;
  wc.timeout_ns = args.timeout_ns;
  // the t-th tile's record
  auto read_tile = [&](uint32_t t, I4Tile& r) -> bool {
    const uint32_t at = base + S::RING + 32 * (t % kI4Ahead);
    if (!i4_wait_warp(bar(IB_TILE + t % kI4Ahead), (t / kI4Ahead) & 1, wc, kSiteI4Tile)) return false;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.flags), "=r"(r.nkeys), "=r"(r.some), "=r"(r.wb) : "r"(at) : "memory");
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r.split) : "r"(at + 16) : "memory");
    return true;
  };
  // the output product of tile t is done
  auto wait_pv = [&](uint32_t t) -> bool {
    return i4_wait_warp(bar(IB_EMPTY + (4 * t + 3) % kSlots), (4 * t + 3) / kSlots & 1, wc, kSiteI4Pv);
  };
  const int block_rows = args.group * args.H, row0 = part * args.part_rows;

  if (idle) {
  } else if (warp >= kExpand && warp < kIssue) {
    // ================================================================ pages -> bf16
    // Four warps a quarter, 16 keys each: a quad has a key and, in the registers' other half, the key eight further; a lane 32 dims
    // (16 bytes of codes).  Neighbouring quads take keys two apart: 416 bytes are 26 chunks of 16, so that the quads of an
    // eight-lane phase read all eight bank groups.  (So row p of the slot is not key p.)
    const int w = warp & 3, m = (warp - kExpand) >> 2, j = lane & 3, u = lane >> 2;
    const int p0 = 16 * w + u, key0 = 16 * w + ((u & 4) | (u & 1) << 1 | (u & 2) >> 1);
    constexpr uint32_t kNext = 8 * kI4Row;  // the second key
    const uint32_t src_lane = base + S::RAW + key0 * kI4Row + 16 * j;
    // chunk q of a lane's 32 dims in its slot; lanes of the slot's second block take their words in another order, so that no two
    // of a quad meet in a bank
    const uint32_t turn = j & 2;
    uint32_t chunk[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      chunk[q] = base + S::V + (j >> 1) * kI4Blk + p0 * 128 + (((uint32_t)(4 * (j & 1)) ^ (uint32_t)(p0 & 7) ^ (uint32_t)q ^ turn) << 4);
    // RoPE keys: the first two quarters' warps take 32 values each, a lane a chunk of the row
    const uint32_t rope_dst = base + S::R + p0 * 128 + ((uint32_t)(4 * (m & 1) + j) ^ (uint32_t)(p0 & 7)) * 16;
    I4Tile a;
    for (uint32_t t = 0; read_tile(t, a); ++t) {
      const uint32_t slot = (4 * t + m) % kSlots, phase = (4 * t + m) / kSlots & 1, full = bar(IB_FULL + (kWhole ? t & 1 : slot));
      if (!a.valid()) {
        // (the issuing thread learns of the end as of a tile)
        if (i4_wait_warp(bar(IB_EMPTY + slot), phase ^ 1, wc, kSiteI4Ring) && lane == 0) mbar_arrive(full);
        break;
      }
      if (!i4_wait_warp(bar(IB_RAW), t & 1, wc, kSiteI4Raw)) break;
      uint32_t code[2][4], s2[2], a2[2], rope[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lds128(src_lane + i * kNext + 64 * m, code[i]);
        s2[i] = lds16(src_lane + i * kNext + kI4Codes + 8 * m - 14 * j);
        if (m < 2) lds128(src_lane + i * kNext + kI4Rope + 64 * (m & 1), rope[i]);
      }
      uint32_t poison = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = key0 + 8 * i;
        const bool over = int4_scale_overflows(s2[i]), late = key >= a.some;
        s2[i] |= s2[i] << 16;
        if (over) s2[i] = kI4Nan;
        // Zeros for what is no key, and for a key that only some of the tokens see and whose values must not reach the others (0 x NaN):
        // the softmax gives NaN to those that see it.
        if (over && late && key < a.nkeys) poison |= 1u << i;
        if (key >= a.nkeys || (over && late)) s2[i] = 0;
        a2[i] = int4_offset(s2[i]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(IB_RAW_EMPTY));
      uint32_t o[4][2][4];
      auto expand = [&]() {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i) expand_int4_word(turn ? code[i][q ^ 2] : code[i][q], s2[i], a2[i], o[q][i]);
      };
      // At 64 rows the next scores wait for the slots: the values are there before (ragged 128 heads 153 us instead of 155).  Below, the
      // expanding warps would only be in the others' way (64 streams x 16 heads 85 us instead of 83).
      if (!kWhole) expand();
      if (!i4_wait_warp(bar(IB_EMPTY + slot), phase ^ 1, wc, kSiteI4Ring)) break;
      // (only now: the softmax has read and reset the bytes of the tile four before)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (poison >> i & 1) for (int g = 0; g < S::kWg; ++g) smem[S::POISON + 64 * (S::kWg * (t & 3) + g) + p0 + 8 * i] = 1;
      if (kWhole) expand();
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) sts128(chunk[q] + slot * kI4Slot + i * 1024, o[q][i][0], o[q][i][1], o[q][i][2], o[q][i][3]);
      if (m < 2)
#pragma unroll
        for (int i = 0; i < 2; ++i) sts128(rope_dst + (t & 1) * kI4Blk + i * 1024, rope[i][0], rope[i][1], rope[i][2], rope[i][3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
  } else if (warp == kIssue) {
    // ================================================================ pages, queries and tile records
    I4Cursor cur;
    cur.init(args, rec);
    I4Tile r;
    bool more = true;
    uint32_t piece = 0;
    const uint64_t keep = l2_policy_evict_last();
    for (uint32_t t = 0; more; ++t) {
      more = cur.next(r);
      int page = 0;
      if (more) {
        const int lp = cur.page();
        page = lp < args.max_pages ? args.block_table[(int64_t)cur.seq * args.max_pages + lp] : -1;
      }
      if (t >= kI4Ahead && !i4_wait_warp(bar(IB_TILE_READ + t % kI4Ahead), (t / kI4Ahead - 1) & 1, wc, kSiteI4Tile)) break;
      if (lane == 0) {
        const uint32_t at = base + S::RING + 32 * (t % kI4Ahead);
        sts128(at, r.flags, r.nkeys, r.some, r.wb);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 16), "r"(r.split) : "memory");
        mbar_arrive(bar(IB_TILE + t % kI4Ahead));
      }
      __syncwarp();
      if (!more) break;
      if (page < 0 || page >= args.num_pages) {  // outside the contract: reported, another page read
        if (lane == 0) atomicCAS(&g_mla_error, 0, 1);
        page = 0;
      }
      if (!i4_wait_warp(bar(IB_RAW_EMPTY), t & 1 ^ 1, wc, kSiteI4Raw)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(IB_RAW), kI4Page);
        bulk_load(base + S::RAW, args.kv + (int64_t)page * kI4Page, kI4Page, bar(IB_RAW));
      }
      __syncwarp();
      if (r.first()) {  // blocks of 64 values [N rows][128 bytes], 128-byte swizzle
        if (piece > 0 && !i4_wait_warp(bar(IB_Q_EMPTY), (piece - 1) & 1, wc, kSiteI4Q)) break;
        if (lane == 0) {
          const int row = r.wb * block_rows + row0;
          mbar_arrive_expect_tx(bar(IB_Q_FULL), 9 * N * 128);
          tma_load_3d(base + S::Q, &args.map_q, bar(IB_Q_FULL), 0, row, 0, keep);
          tma_load_2d(base + S::Q + 8 * N * 128, &args.map_qr, bar(IB_Q_FULL), 0, row, keep);
        }
        __syncwarp();
        ++piece;
      }
    }
  } else if (warp > kIssue) {
    // ================================================================ MMAs
    constexpr uint32_t id_qk = idesc_bf16_f32(64, N, 0, 0), id_pv = idesc_bf16_f32(128, N, 1, 1);
    // descriptors: an address 16 n bytes further is n more in the low word
    const uint64_t desc_k = smem_desc(base + S::V, 16, 1024, kSwizzle128B), desc_r = smem_desc(base + S::R, 16, 1024, kSwizzle128B);
    const uint64_t desc_q = smem_desc(base + S::Q, 16, 1024, kSwizzle128B), desc_c = smem_desc(base + S::V, kI4Blk, 1024, kSwizzle128B);
    const uint64_t desc_p = smem_desc(base + S::P, 16, 8 * S::kPRow, N > 32 ? kSwizzle128B : N == 32 ? kSwizzle64B : kSwizzle32B);
    uint32_t el;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(el));
    if (el) {
      // One thread issues all of them, whatever is ready first: scores of the next tile, or the output of one before.  (MMAs of two
      // warps take turns one by one, and each turn costs: 59 cycles an MMA.  A warp that votes after every question is slower too,
      // one that asks with all its lanes at once is not faster.)
      bool ok = true;
      uint32_t piece = 0, t = 0, tp = 0, starts = 0;  // tile t's scores, tile tp's output; bit i: tile t - 1 - i starts a piece
      auto pv = [&]() {
        const uint32_t add = starts >> (t - 1 - tp) & 1 ? 0u : 1u;
        const uint64_t w = desc_p + (tp % S::kP) * (64 * S::kPRow >> 4);
        uint32_t slot = 4 * tp % kSlots;
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint64_t c = desc_c + slot * (kI4Slot >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_bf16_ss(tmem + TO + N * m, c + 128 * k, w + S::kPRow * k, id_pv, k ? 1u : add);
          mma_commit(bar(IB_EMPTY + slot));
          slot = slot + 1 == kSlots ? 0 : slot + 1;
        }
        ++tp;
      };
      // until the barrier's phase is over; the output meanwhile, when its weights are there
      auto wait = [&](uint32_t b, uint32_t phase, int site) -> bool {
        return i4_wait_busy(b, phase, wc, site, [&]() -> bool {
          if (!(tp < t && mbar_test_wait(bar(IB_P_FULL + (tp & 1)), tp >> 1 & 1))) return false;
          pv();
          return true;
        });
      };
      for (;;) {
        const uint32_t o = t & 1, d = tmem + TS + N * o;
        uint64_t bq = desc_q;
        uint32_t slot = 4 * t % kSlots, phase = 4 * t / kSlots & 1;
        // Where two tiles fit, a tile's quarters are mostly ready together, and one question (~120 cycles) is asked for all (one
        // for each: 64 streams x 16 heads 93 us instead of 86).  Where one and a half fit, they become ready one by one.
        if (!(ok = wait(bar(IB_FULL + (kWhole ? o : slot)), kWhole ? t >> 1 & 1 : phase, kSiteI4Ring))) break;
        uint32_t f;
        // (the expanding warps have seen the tile's record)
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(f) : "r"(base + S::RING + 32 * (t % kI4Ahead)) : "memory");
        if (!(f & I4Tile::kValid)) break;
        if ((f & I4Tile::kFirst) && !(ok = wait(bar(IB_Q_FULL), piece++ & 1, kSiteI4Q))) break;
        auto quarters = [&](int m, int end) {
#pragma unroll 1
          for (; m < end; ++m) {
            if (!kWhole && m > 0 && !(ok = wait(bar(IB_FULL + slot), phase, kSiteI4Ring))) break;
            tc_fence_after();
            const uint64_t ak = desc_k + slot * (kI4Slot >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_bf16_ss(d, ak + (k >> 2) * (kI4Blk >> 4) + 2 * (k & 3), bq + (k >> 2) * (N * 128 >> 4) + 2 * (k & 3), id_qk, m + k ? 1u : 0u);
            if (++slot == kSlots) {
              slot = 0;
              phase ^= 1;
            }
            bq += 2 * N * 128 >> 4;
          }
        };
        quarters(0, 2);
        if (!ok) break;
        // (the first two quarters' warps have brought the RoPE keys)
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16_ss(d, desc_r + o * (kI4Blk >> 4) + 2 * k, desc_q + (8 * N * 128 >> 4) + 2 * k, id_qk, 1u);
        quarters(2, 4);
        if (!ok) break;
        mma_commit(bar(IB_S_FULL + o));
        if (f & I4Tile::kLast) mma_commit(bar(IB_Q_EMPTY));
        starts = starts << 1 | (f & I4Tile::kFirst ? 1u : 0u);
        ++t;  // (the scores of tile t + 2 go over those of tile t, which have been read: its keys wait for tile t's output)
      }
      if (ok && t > 0) wait(bar(IB_EMPTY + (4 * t - 1) % kSlots), (4 * t - 1) / kSlots & 1, kSiteI4Pv);
      mma_commit(bar(IB_DRAIN));
    }
    __syncwarp();
    // no MMA may still run when the CTA leaves
    WaitCtx wd = wc;
    wd.timeout_ns = 100000000ull;
    volatile int no_abort = 0;
    wd.abort_local = &no_abort;
    i4_wait_warp(bar(IB_DRAIN), 0, wd, kSiteI4Drain);
  } else {
    // ================================================================ softmax
    // A lane: rows (of the warpgroup's NC) 4 b + j, b < B, for the keys in places p0 and p0 + 8.  Arrays over rows are kept in the
    // order of P's columns, j B + b.
    const int wg = warp >> 2, w = warp & 3, j = lane & 3, u = lane >> 2, col0 = NC * wg;
    const int p0 = 16 * w + u, key0 = 16 * w + ((u & 4) | (u & 1) << 1 | (u & 2) >> 1);
    const uint32_t lanes = (uint32_t)(32 * w) << 16;
    const uint32_t mx = base + S::MAX + warp * NC * 4, fac = base + S::FAC + warp * NC * 4, xch = base + S::XCH + wg * 4 * NC * 4;
    constexpr uint32_t kSums = 4 * S::kWg * NC * 4;  // from the place of the maxima to that of the sums
    const float sl2 = args.scale_log2;
    uint32_t exchanges = 0;
    float l[B];
    bool ok = true;
    I4Tile a;
    // reduces a lane's values over the quads, then over the warps: each lane has its columns' results.  (Maxima and sums each in a
    // place of their own: between two exchanges of a kind every warp has come past the flags, so that none still reads the one before.)
    auto exchange = [&](uint32_t at, float (&v)[B], bool sum) -> bool {
      auto op = [sum](float x, float y) { return sum ? x + y : fmaxf(x, y); };
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v[b] = op(v[b], __shfl_xor_sync(0xffffffffu, v[b], o));
      if (u == 0)
#pragma unroll
        for (int b = 0; b < B; ++b) sts32f(at + (w * NC + j * B + b) * 4, v[b]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(IB_XCH + wg));
      if (!i4_wait_warp(bar(IB_XCH + wg), exchanges++ & 1, wc, kSiteI4Flag)) return false;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const uint32_t c = at + (j * B + b) * 4;
        v[b] = op(op(lds32f(c), lds32f(c + NC * 4)), op(lds32f(c + 2 * NC * 4), lds32f(c + 3 * NC * 4)));
      }
      return true;
    };
    for (uint32_t t = 0; (ok = read_tile(t, a)) && a.valid(); ++t) {
      if (a.first()) {
#pragma unroll
        for (int b = 0; b < B; ++b) l[b] = 0.f;
        if (lane < NC) sts32f(mx + 4 * lane, -3.402823466e38f);  // (finite: a first score against it is no NaN)
        __syncwarp();
      }
      if (!(ok = i4_wait_warp(bar(IB_S_FULL + (t & 1)), (t >> 1) & 1, wc, kSiteI4Scores))) break;
      tc_fence_after();
      if (lane == 0) mbar_arrive(bar(IB_TILE_READ + t % kI4Ahead));
      float d[2][B];
      auto load_scores = [&]() {
        uint32_t v[2 * B];
        tmem_ld_16(tmem + lanes + TS + N * (t & 1) + col0, v);
        tmem_wait_ld();
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) d[i][b] = __uint_as_float(v[2 * b + i]);
      };
      int hidden[2] = {0, 0};  // rows [0, hidden) of the warpgroup's do not see the key
      bool bad[2] = {false, false};
      const bool masked = a.some < kI4Tile || a.nkeys < kI4Tile;
      if (masked)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = key0 + 8 * i;
          hidden[i] = (key >= a.nkeys ? 1 << 20 : args.causal ? max(key - a.some + 1, 0) * args.H : 0) - row0 - col0;
          uint8_t* poison = smem + S::POISON + 64 * (S::kWg * (t & 3) + wg) + p0 + 8 * i;
          bad[i] = *poison != 0;
          __syncwarp();
          if (bad[i] && j == 0) *poison = 0;
        }
      auto mask_scores = [&]() {
        if (masked)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < B; ++b)
              d[i][b] = 4 * b + j < hidden[i] ? -INFINITY : bad[i] ? __uint_as_float(0x7FC00000u) : d[i][b];
      };
      const uint64_t s2 = splat_f32x2(sl2);
      auto against_max = [&]() {  // in log2 units
#pragma unroll
        for (int q = 0; q < B / 4; ++q) {
          float m4[4];
          lds128f(mx + 4 * (j * B + 4 * q), m4[0], m4[1], m4[2], m4[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              unpack_f32x2(ffma_f32x2(pack_f32x2(d[i][4 * q + 2 * h], d[i][4 * q + 2 * h + 1]), s2, pack_f32x2(-m4[2 * h], -m4[2 * h + 1])),
                           d[i][4 * q + 2 * h], d[i][4 * q + 2 * h + 1]);
        }
      };
      load_scores();
      mask_scores();
      against_max();
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < B; ++b) top = fmax3(top, d[0][b], d[1][b]);
      const bool over = __any_sync(0xffffffffu, top > 8.f);
      if (lane == 0) {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + S::FLAG + 16 * S::kWg * (t & 1) + 4 * warp), "r"(over ? 1u : 0u) : "memory");
        mbar_arrive(bar(IB_FLAG + 2 * wg + (t & 1)));
      }
      __syncwarp();
      if (!(ok = i4_wait_warp(bar(IB_FLAG + 2 * wg + (t & 1)), (t >> 1) & 1, wc, kSiteI4Flag))) break;
      uint32_t f4[4];
      lds128(base + S::FLAG + 16 * S::kWg * (t & 1) + 16 * wg, f4);
      // (P is free: the scores' commit waited for all MMAs issued before them, the last output product that read it among them: for
      // two P that of tile t - 2, for one that of tile t - 1, which gave the place for this tile's last quarters)
      if ((f4[0] | f4[1] | f4[2] | f4[3]) != 0) {
        if (t > 0 && !(ok = wait_pv(t - 1))) break;  // the output so far is complete
        tc_fence_after();
        load_scores();
        mask_scores();
        float v[B];
#pragma unroll
        for (int b = 0; b < B; ++b) v[b] = fmaxf(d[0][b], d[1][b]) * sl2;
        if (!(ok = exchange(xch, v, false))) break;
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint32_t c = 4 * (j * B + b);
          const float old = lds32f(mx + c);
          const bool grow = v[b] > old + 8.f;
          __syncwarp();
          if (u == 0) {
            sts32f(mx + c, grow ? v[b] : old);
            sts32f(fac + c, grow ? ex2_approx(old - v[b]) : 1.f);
          }
        }
        __syncwarp();
        against_max();
        if (!a.first()) {
#pragma unroll
          for (int b = 0; b < B; ++b) l[b] *= lds32f(fac + 4 * (j * B + b));
#pragma unroll 1
          for (int c = 0; c < NC; c += 16) {
            float f[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) lds128f(fac + 4 * c + 16 * q, f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              uint32_t o[16];
              tmem_ld16(tmem + lanes + TO + N * m + col0 + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f[k]);
              tmem_st16(tmem + lanes + TO + N * m + col0 + c, o);
            }
          }
          tmem_wait_st();
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t pp[B / 2];
#pragma unroll
        for (int b = 0; b < B; b += 2) {
          const float x0 = ex2_approx(d[i][b]), x1 = ex2_approx(d[i][b + 1]);
          // P in bf16, the type of the values in the tensor cores (half a step is 2^-8 of a weight at most, of either sign); the
          // row's sum takes the float32 weights, so that lse is not rounded with them
          pp[b / 2] = pack_bf16(x0, x1);
          l[b] += x0;
          l[b + 1] += x1;
        }
        const int p = p0 + 8 * i;
        const uint32_t swz = N > 32 ? p & 7 : N == 32 ? (p >> 1) & 3 : (p >> 2) & 1, at = base + S::P + (t % S::kP) * (64 * S::kPRow) + p * S::kPRow;
        if constexpr (B == 8)
          sts128(at + (((uint32_t)(col0 / 8 + j) ^ swz) << 4), pp[0], pp[1], pp[2], pp[3]);
        else
          asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(at + (((uint32_t)(col0 / 8 + (j >> 1)) ^ swz) << 4) + 8 * (j & 1)), "r"(pp[0]), "r"(pp[1]) : "memory");
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(IB_P_FULL + (t & 1)));
      if (!a.last()) continue;

      // O / l of the finished piece -> its rows of out, or a split partial
      if (!(ok = exchange(xch + kSums, l, true))) break;
      const int32_t* num_splits = sched + kSchedHeader + kUnitInts * args.num_units;
      const int ns = num_splits[a.wb * args.group];
      const bool split = ns > 1;
      const int64_t off = split ? num_splits[args.num_qb + a.wb * args.group] : 0;
      auto row_of = [&](int r) -> int64_t {  // of the warpgroup's row r in out or in the partials, -1 for none
        const int rr = row0 + col0 + r;      // row of the block
        if (col0 + r >= args.part_rows || rr >= block_rows) return -1;
        if (!split) return (int64_t)a.wb * block_rows + rr;
        const int g = rr / args.H;
        return (off + g * ns + a.split) * args.H + (rr - g * args.H);
      };
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const uint32_t c = 4 * (j * B + b);
        const bool none = l[b] == 0.f;  // the row saw no key
        if (u == 0) sts32f(fac + c, none ? 0.f : 1.f / l[b]);
        if (u == 0 && w == 0) {
          const int64_t row = row_of(4 * b + j);
          const float lse = none ? -INFINITY : (lds32f(mx + c) + log2f(l[b])) * 0.69314718055994530942f;
          if (row >= 0) {
            if (split) args.lse_acc[row] = lse; else args.lse[row] = lse;
          }
        }
      }
      const int64_t row = row_of(4 * (lane % B) + (lane % NC) / B);  // of column lane % NC
      __syncwarp();
      if (!(ok = wait_pv(t))) break;
      tc_fence_after();
#pragma unroll 1
      for (int mc = 0; mc < 4 * (NC / 16); ++mc) {
        const int m = mc / (NC / 16), c = 16 * (mc % (NC / 16)), dim = 128 * m + 32 * w + lane;
        uint32_t o[16];
        tmem_ld16(tmem + lanes + TO + N * m + col0 + c, o);
        tmem_wait_ld();
        float f[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) lds128f(fac + 4 * c + 16 * q, f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float x0 = f[k] == 0.f ? 0.f : __uint_as_float(o[k]) * f[k], x1 = f[k + 1] == 0.f ? 0.f : __uint_as_float(o[k + 1]) * f[k + 1];
          const int64_t r0 = __shfl_sync(0xffffffffu, row, c + k), r1 = __shfl_sync(0xffffffffu, row, c + k + 1);
          if (split || args.out_f32) {
            float* dst = split ? args.o_acc : static_cast<float*>(args.out);
            if (r0 >= 0) dst[r0 * 512 + dim] = x0;
            if (r1 >= 0) dst[r1 * 512 + dim] = x1;
          } else {  // even lanes write two dims of the first row, odd lanes of the second
            const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x0 : x1, 1);
            const int64_t to = (lane & 1) ? r1 : r0;
            const uint32_t two = (lane & 1) ? pack_bf16(got, x1) : pack_bf16(x0, got);
            if (to >= 0) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(args.out) + to * 512 + (dim & ~1)) = two;
          }
        }
      }
    }
    tc_fence_before();
  }

  __syncwarp();
  __syncthreads();
  if (*abort_flag) drain_delay(200000);  // in-flight copies and MMAs land before release
  if (warp == kIssue + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

__global__ void __launch_bounds__(I4Smem<16>::kThreads, 1) mla_decode_int4_n16_kernel(const __grid_constant__ Int4Args args) {
  decode_int4_body<16>(args);
}
__global__ void __launch_bounds__(I4Smem<32>::kThreads, 1) mla_decode_int4_n32_kernel(const __grid_constant__ Int4Args args) {
  decode_int4_body<32>(args);
}
__global__ void __launch_bounds__(I4Smem<48>::kThreads, 1) mla_decode_int4_n48_kernel(const __grid_constant__ Int4Args args) {
  decode_int4_body<48>(args);
}
__global__ void __launch_bounds__(I4Smem<64>::kThreads, 1) mla_decode_int4_n64_kernel(const __grid_constant__ Int4Args args) {
  decode_int4_body<64>(args);
}

}  // namespace mla
