// Attention of ragged chunks of new tokens over the paged cache, in the absorbed form: for every
// new token and head, s_j = scale (q~ . c_j + q^R . k^R_j) over the keys the token may see,
// out = sum_j softmax(s)_j c_j (512 dims), lse = ln sum_j exp(s_j)  ("MLA inference: two
// computation paths and FlashMLA", section "Two equivalent paths", path two; the causal rule of
// "Which is faster: count new tokens and cached tokens": new tokens only see what precedes them).
//
// What bounds it: 2176 FLOP per (row, key) against 1152 bytes per key shared by all rows of a
// sequence's chunk -- from two tokens at 128 heads on it is the tensor cores, not HBM.
//
// Work split.  A block is 128 rows (128 / H tokens of one sequence).  Its fp32 output, 128 x 512,
// is one SM's whole tensor memory, so a CTA pair takes a block with tcgen05 cta_group::2, M = 128:
// each CTA holds 64 rows, as 128 lanes x half the columns (lanes 64..127 hold the upper half of an
// MMA's N columns for the same 64 rows): O takes 256 columns, two score buffers of a 256-key tile
// 128 each.  Measured issue rate of M = 128, N = 256: 64 cycles, the same FLOP/s as M = 256; with
// N = 128 it drops to 68%, which is why a tile is 256 keys.  Scores are complete in fp32 -- no
// exchange of partial scores between the CTAs, unlike the decode kernel's split by latent dims.
//
// The MMAs take half of each B operand from either CTA: QK wants 128 keys x 576 dims per CTA (two
// of the tile's four pages), PV all 256 keys x 128 dims of every 256.  Both stream through one
// ring of seven 16 KB slots (K: 128 keys x 64 dims; V: 64 keys x 128 dims), 17 slots a tile.  Six
// warps share the copies: a warp issues a TMA copy every ~0.18 us whatever its size.
//
// Roles (512 threads a CTA): warps 0..5 copy pages, warp 6 issues the MMAs of the pair (first CTA
// only), warp 7 copies queries, warps 8..15 (two warpgroups, half of a tile's score columns each)
// run the softmax.  A row's 256 scores lie in four threads, which agree on its maximum through
// shared memory; O is rescaled only when the maximum grows by more than 2^8.
//
// Measured, from a graph / through the Python entry on changing inputs: 512 tokens x 128 heads after 32,768 rows in
// 2.50-2.56 / 2.60 ms, 1810-1880 TFLOP/s (the power cap; cuBLAS held for seconds would take 2.76); 4 x ~430 tokens x
// 16 heads after ~3000 rows in 122-125 / 133 us, 1500-1630 TFLOP/s; 32 streams of 1..24 tokens x 128 heads in
// 167-172 / 187 us, 1460-1640 TFLOP/s; the plan of the step, 10 to 24 us once for all layers, not counted.  A long
// append's tile takes 4840 cycles, of which the tensor cores' own are 4352; the prompts' 5110 and the
// streams' 5670, where slots wait for pages from L2 and HBM.  With many short blocks add the change of block
// (~3/4 of a tile: the last softmax and the first have no MMAs beside them), what the units' shares
// differ by, and the launches.
//
// Rows of a block see different numbers of keys where it holds several tokens.  P is zero past a
// row's limit, but 0 x NaN is NaN, so in the pages that some row does not see in full the copying
// warp zeroes what no row sees and whatever is not finite.  A row that sees a key whose score is not
// finite gets NaN, in out and lse alike and whichever tile the key lies in.
#pragma once
#include <type_traits>

#include "chunk_plan.h"
#include "common.cuh"
#include "decode_kernel.cuh"  // packed float pairs, bf16 packing
#include "int4_rows.cuh"

namespace mla {

constexpr int kCkThreads = 512;
constexpr int kCkCopyWarps = 6;
constexpr int kCkSlots = 7;
constexpr int kCkPageBytes = 64 * 1152;
constexpr uint32_t kCkBlk = 8192;                            // [64 rows][64 bf16], 128-byte swizzle
constexpr uint32_t kCkSlot = 2 * kCkBlk;
constexpr uint32_t CK_Q = 0;                                 // 9 blocks: 64 rows x 576 dims
constexpr uint32_t CK_P = 9 * kCkBlk;                        // 4 blocks: 64 rows x 256 keys
constexpr uint32_t CK_RING = CK_P + 4 * kCkBlk;
constexpr uint32_t CK_RED = CK_RING + kCkSlots * kCkSlot;    // row maxima [tile parity][4][64]
constexpr uint32_t CK_SUM = CK_RED + 2 * 4 * 64 * 4;         // row sums [4][64]
constexpr uint32_t CK_BAR = CK_SUM + 4 * 64 * 4;
constexpr uint32_t kCkSmem = CK_BAR + 512 + 1024;            // + alignment slack
static_assert(kCkSmem <= 232448, "shared memory");

// Barriers.  "leader": used in the first CTA only, arrived on by both.
enum : uint32_t {
  CB_FULL = 0,                        // + slot, leader: one arrival and the bytes of each CTA
  CB_EMPTY = CB_FULL + kCkSlots,      // + slot: the MMAs that read it are done
  CB_RAW = CB_EMPTY + kCkSlots,       // + copying warp: a page it looks through has landed
  CB_Q_FULL = CB_RAW + kCkCopyWarps,  // leader
  CB_Q_EMPTY,
  CB_S_FULL,                          // + tile parity
  CB_P_FULL = CB_S_FULL + 2,          // leader: one arrival per softmax warp; its scores are read, too
  CB_P_FREE,                          // PV done
  CB_RED,                             // + tile parity: row maxima in shared memory, one arrival per softmax warp
  CB_SUM = CB_RED + 2,                // row sums in shared memory
  CB_DRAIN,
  kCkBars
};
constexpr uint32_t kCkTmemSlot = 8 * kCkBars, kCkAbort = kCkTmemSlot + 4;
static_assert(kCkAbort + 4 <= 512, "barrier area");

// tensor memory columns
constexpr uint32_t CT_S = 0, CT_O = 256;  // S buffers at 0 and 128

enum ChunkSite : int { kSiteCkRing = 32, kSiteCkRaw, kSiteCkQ, kSiteCkScores, kSiteCkP, kSiteCkPv, kSiteCkRed, kSiteCkDrain };

struct ChunkArgs {
  CUtensorMap map_q;    // q~ rows: bf16 {64, T * H, 8 blocks 128 bytes apart}, box {64, 64, 8}, 128-byte swizzle
  CUtensorMap map_qr;   // q^R rows: bf16 {64, T * H}, box {64, 64}
  CUtensorMap map_k;    // cache rows: bf16 {576, pages * 64}, box {64, 64}
  CUtensorMap map_v;    // the same rows as {64, pages * 64, 9 blocks 128 bytes apart}, box {64, 64, 2}
  const uint8_t* kv;    // the cache rows themselves (bf16)
  const int32_t* block_table;
  const int32_t* sched;
  __nv_bfloat16* out;   // [T][H][512]
  float* lse;           // [T][H]
  float* o_acc;         // split partials, normalised, 128 x 512 each in the accumulators' order
  float* lse_acc;       // [slots][128]
  float scale_log2;
  ChunkKey key;
  int32_t num_pages;
  int32_t expanded;     // the cache rows are the expanded ones: page = page_off[seq] + logical page
  uint64_t timeout_ns;
};

// ----------------------------------------------------------------- CTA-pair instructions
// (mbar: a barrier of either CTA of the pair, shared::cluster address)
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t mbar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(mbar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma2_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t mbar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(mbar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {  // multiples of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
               : "memory");
}
// (relaxed: the copies themselves order their bytes; a release arrive on the other CTA's barrier waits
// for this thread's earlier writes, ~1400 cycles measured)
__device__ __forceinline__ void mbar_arrive_expect_tx_remote(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mma2_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Two MMAs with the same A one after the other: it is read from shared memory once.
__device__ __forceinline__ void mma2_bf16_ss_twice(uint32_t d0, uint32_t d1, uint64_t a_desc, uint64_t b0, uint64_t b1, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16.collector::a::fill [%0], %2, %3, %5, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16.collector::a::lastuse [%1], %2, %4, %5, p;\n\t}" ::"r"(d0),
      "r"(d1), "l"(a_desc), "l"(b0), "l"(b1), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive (once) on the barrier at this offset in both CTAs when this thread's MMAs so far are done.
__device__ __forceinline__ void mma2_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ uint64_t fmul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Arrive on a barrier of either CTA after writes to this CTA's own shared memory that the pair's MMA
// (here: this CTA's tensor cores) will read.  The proxy fence before it has put them into shared memory,
// so the arrive need not wait for anything else of this thread's; a release at cluster scope did, for
// ~1000 cycles (5% of the kernel).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// One lane of a converged warp.  The issuing roles below run converged, with one lane's predicate on
// the instruction alone: descriptors and addresses then stay in uniform registers.  (One lane in a
// branch of its own instead: 12,100 cycles a tile for the MMAs' issue alone, against 4352 of MMA time.)
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// One tile of a unit's work.
struct ChunkTileRef {
  ChunkBlock b;
  int blk, tile, vis;  // vis: keys the block's last token sees
  int split;           // this unit's share of the block
  bool first, last;
  __device__ int pages() const { return min(max((vis - kChunkTile * tile + 63) >> 6, 0), 4); }
};

// The header's words 0..3, 8..11 and 12..15 against the call's.
__device__ __forceinline__ bool chunk_plan_is(int4 h0, int4 h2, int4 h3, const ChunkKey& k) {
  static_assert(kChMagic == 0 && kChUnits == 1 && kChCapacity == 2 && kChBatch == 10 && kChCausal == 11 && kChMaxTokens == 12 &&
                kChHeads == 13 && kChMaxPages == 14 && kChKvPages == 15, "header");
  return h0.x == kChunkMagic && h0.y == k.units && h0.z == k.capacity && h2.z == k.batch && h2.w == k.causal &&
         h3.x == k.max_tokens && h3.y == k.heads && h3.z == k.max_pages && h3.w == k.kv_pages;
}

// Walks the unit's tiles in order, across blocks.
struct ChunkCursor {
  const ChunkBlock* blocks;
  int causal, blk, blk0, blk1, tile0, tile1, split0, t, end;
  bool open;
  ChunkBlock b;
  int vis;
  __device__ void set_block(int4 lo, int4 hi) {
    b.tok0 = lo.x; b.ntok = lo.y; b.seq = lo.z; b.base = lo.w;
    b.len = hi.x; b.nt = hi.y; b.splits = hi.z; b.offset = hi.w;
  }
  // r: the unit's record {first block, first tile, last block, end tile | split, ... | the first block}
  __device__ void init(const ChunkBlock* blk_records, int4 r0, int split, int4 lo, int4 hi, int causal_) {
    blocks = blk_records;
    causal = causal_;
    blk = blk0 = r0.x;
    tile0 = r0.y;
    blk1 = r0.z;
    tile1 = r0.w;
    split0 = split;
    open = false;
    set_block(lo, hi);
  }
  __device__ bool next(ChunkTileRef& r) {
    if (!open || t >= end) {
      if (open) {
        if (++blk > blk1) return false;
        const int4* src = reinterpret_cast<const int4*>(blocks + blk);
        set_block(src[0], src[1]);
      }
      vis = chunk_visible(b, b.ntok - 1, causal);
      t = blk == blk0 ? tile0 : 0;
      end = blk == blk1 ? tile1 : b.nt;
      open = true;
      r.first = true;
    } else {
      r.first = false;
    }
    r.b = b;
    r.blk = blk;
    r.vis = vis;
    r.split = blk == blk0 ? split0 : 0;
    r.tile = t++;
    r.last = t >= end;
    return true;
  }
  __device__ void skip_block() { t = end; }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kCkThreads, 1)
    mla_chunk_kernel(const __grid_constant__ ChunkArgs args) {
  extern __shared__ uint8_t ck_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ck_smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  auto bar = [&](uint32_t i) { return base + CK_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + CK_BAR + kCkAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + CK_BAR + kCkTmemSlot);

  if (tid == 0) {
    for (uint32_t i = 0; i < kCkBars; ++i) {
      uint32_t count = 1;
      if (i < CB_EMPTY || i == CB_Q_FULL) count = 2;                                    // one per CTA
      if (i == CB_P_FULL) count = 16;                                                   // 8 softmax warps per CTA
      if (i >= CB_RED && i <= CB_SUM) count = 8;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 6) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (tid == 0) {
    prefetch_tensormap(&args.map_q);
    prefetch_tensormap(&args.map_qr);
    prefetch_tensormap(&args.map_k);
    prefetch_tensormap(&args.map_v);
  }
  pdl_wait_prerequisites();
  const int32_t* sched = args.sched;
  const ChunkLayout lay = chunk_layout(args.key.units, args.key.capacity, args.key.batch);
  const int4* rec = reinterpret_cast<const int4*>(sched + lay.units + kChunkUnitInts * (blockIdx.x >> 1));
  // (header and record in whole vectors: one memory latency for all of it)
  const int4 h0 = reinterpret_cast<const int4*>(sched)[0], h2 = reinterpret_cast<const int4*>(sched)[2],
             h3 = reinterpret_cast<const int4*>(sched)[3], r0 = rec[0], r1 = rec[1], r2 = rec[2], r3 = rec[3];
  const bool bad_meta = !chunk_plan_is(h0, h2, h3, args.key);
  const bool idle = bad_meta || r0.x < 0;  // the same in both CTAs
  if (bad_meta && tid == 0) atomicCAS(&g_mla_error, 0, 5);
  pdl_launch_dependents();

  WaitCtx wc;
  wc.abort_local = abort_flag;
  wc.abort_peer = map_to_rank(smem_addr((const void*)abort_flag), rank ^ 1);
  wc.timeout_ns = args.timeout_ns;
  const uint32_t lead0 = map_to_rank(bar(0), 0);  // the leader's barrier i is at lead0 + 8 i
  ChunkCursor cur;
  if (!idle) cur.init(reinterpret_cast<const ChunkBlock*>(sched + lay.blocks), r0, r1.x, r2, r3, args.key.causal);

  if (idle) {
  } else if (warp < kCkCopyWarps) {
    // ================================================================ page copies
    const int32_t* page_off = sched + lay.page_off;
    const bool el = elect_one();
    // Slots are taken in turn: warp i the slots i, i + 6, ... of the whole stream.  The ring position
    // of the section at hand (a tile's K or V slots): its first slot, that slot's phase (the waits of the
    // first round pass: "the phase before" of a fresh barrier) and its number modulo the warps.
    int first_slot = 0, first_turn = 0;
    uint32_t first_phase = 1, n_raw = 0;
    bool ok = true;
    uint32_t slot = 0, phase = 0;
    auto locate = [&](int k) {  // slot k < 14 - kCkSlots + 1 of the section
      const int q = first_slot + k, wraps = (q >= kCkSlots) + (q >= 2 * kCkSlots);
      slot = q - kCkSlots * wraps;
      phase = first_phase ^ (wraps & 1);
    };
    auto mine = [&]() -> int {  // this warp's first slot of the section
      const int k = warp - first_turn;
      return k < 0 ? k + kCkCopyWarps : k;
    };
    auto leave = [&](int n) {  // the section had n <= 9 slots
      locate(n);
      first_slot = slot;
      first_phase = phase;
      first_turn = (first_turn + n) % kCkCopyWarps;
    };
    // lane j < 4: physical page of the tile's page j, as the table has it (looked at when it is used, so
    // that the load's latency is not waited for)
    auto page_of = [&](const ChunkTileRef& r) -> int {
      const int lp = 4 * r.tile + lane;
      if (lane >= 4 || lane >= r.pages()) return 0;
      if (args.expanded) return page_off[r.b.seq] + lp;
      return args.block_table[(int64_t)r.b.seq * args.key.max_pages + lp];
    };
    auto checked = [&](int page) -> int {
      if (!args.expanded && (page < 0 || page >= args.num_pages)) {  // outside the contract: reported, another page read
        atomicCAS(&g_mla_error, 0, 1);
        page = 0;
      }
      return page;
    };
    // The copies take 128 or 256 bytes of a row at a time, and where nothing else has brought the rows they wait
    // on HBM: the last block of a sequence brings them into L2 in order.
    //   The sequence's only block: a tile's rows in one sweep, right before their copies (64 sequences of one
    //   token over 8192 keys, 16 heads 122 against 134 us; a tile earlier it is 147).
    //   With other blocks beside it: a tile ahead, in pieces of 8 KB spread over the slots of the tile before (20
    //   sequences of 16 tokens x 128 heads over 8192 keys 418 against 454 us, 64 of 2 over 4096 97 against 107; in
    //   one sweep it costs, prompt pieces 134 against 131 us).
    enum { kNoPrefetch, kSweep, kAhead };
    auto bring = [&](const ChunkTileRef& r) -> int {
      if (r.b.base + r.b.ntok - 1 != r.b.len) return kNoPrefetch;  // not the sequence's last
      const int32_t* off = sched + lay.blk_off + r.b.seq;
      return off[1] - off[0] == 1 ? kSweep : kAhead;
    };
    auto sweep = [&](const ChunkTileRef& r, int page) {
      const bool here = (uint32_t)(lane - 2 * (int)rank) < 2u && lane < r.pages();
      if (here && r.tile % kCkCopyWarps == warp)
        prefetch_l2(args.kv + (int64_t)page * kCkPageBytes, min(r.vis - kChunkTile * r.tile - 64 * lane, 64) * 1152);
      __syncwarp();
    };
    // (ahead: tile n's rows are prefetched meanwhile)
    auto copy_k = [&](const ChunkTileRef& r, int page, const ChunkTileRef& n, int n_page, bool ahead) -> bool {
      const int np = min(max(r.pages() - 2 * (int)rank, 0), 2);
      const int y0 = 64 * __shfl_sync(0xffffffffu, page, 2 * rank), y1 = 64 * __shfl_sync(0xffffffffu, page, 2 * rank + 1);
      const int n0 = __shfl_sync(0xffffffffu, n_page, 2 * rank), n1 = __shfl_sync(0xffffffffu, n_page, 2 * rank + 1);
      const int n_np = ahead ? min(max(n.pages() - 2 * (int)rank, 0), 2) : 0;
#pragma unroll 1
      for (int d = mine(); d < 9; d += kCkCopyWarps) {
        locate(d);
        if (el && n_np > 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // two of the 18 pieces of 8 KB of the CTA's two pages
            const int piece = 2 * d + h, second = piece >= 9;
            if (second < n_np)
              prefetch_l2(args.kv + (int64_t)(second ? n1 : n0) * kCkPageBytes + (piece - 9 * second) * 8192, 8192);
          }
        }
        __syncwarp();
        if (!wait_warp<true>(bar(CB_EMPTY + slot), phase, wc, kSiteCkRing)) return false;
        const uint32_t full = lead0 + 8 * (CB_FULL + slot), dst = base + CK_RING + slot * kCkSlot;
        if (el) {
          if (np == 0) {
            mbar_arrive_remote_relaxed(full, 0);
          } else {
            mbar_arrive_expect_tx_remote(full, np * kCkBlk);
            tma2_load_2d(dst, &args.map_k, full, 64 * d, y0);
            if (np == 2) tma2_load_2d(dst + kCkBlk, &args.map_k, full, 64 * d, y1);
          }
        }
        __syncwarp();
      }
      leave(9);
      return true;
    };
    auto copy_v = [&](const ChunkTileRef& r, int page) -> bool {
      const int np = r.pages(), some = chunk_visible(r.b, 0, args.key.causal);  // keys every row of the block sees
#pragma unroll 1
      for (int k = mine(); k < 2 * np; k += kCkCopyWarps) {
        const int kb = k >> 1, n = k & 1;
        const int y = 64 * __shfl_sync(0xffffffffu, page, kb), key0 = kChunkTile * r.tile + 64 * kb;
        locate(k);
        if (!wait_warp<true>(bar(CB_EMPTY + slot), phase, wc, kSiteCkRing)) return false;
        const uint32_t full = lead0 + 8 * (CB_FULL + slot), dst = base + CK_RING + slot * kCkSlot;
        const int z = 4 * n + 2 * (int)rank;  // dims 256 n + 128 rank, in blocks of 64
        if (key0 + 64 <= some) {
          if (el) {
            mbar_arrive_expect_tx_remote(full, kCkSlot);
            tma2_load_3d(dst, &args.map_v, full, 0, y, z);
          }
          __syncwarp();
          continue;
        }
        // some row does not see all of this page: rows [from, to) of it are looked through
        const uint32_t raw = bar(CB_RAW + warp);
        if (el) {
          mbar_arrive_expect_tx(raw, kCkSlot);
          tma2_load_3d(dst, &args.map_v, map_to_rank(raw, rank), 0, y, z);
        }
        __syncwarp();
        if (!wait_warp(raw, n_raw & 1, wc, kSiteCkRaw)) return false;
        ++n_raw;
        const int from = max(some - key0, 0), seen = min(r.vis - key0, 64), to = (seen + 15) & ~15;
        for (int i = from * 16 + lane; i < to * 16; i += 32) {  // 16-byte chunks: two blocks of 8 a row
          const int row = i >> 4;
          const uint32_t a = dst + ((i >> 3) & 1) * kCkBlk + row * 128 + (i & 7) * 16;
          uint32_t v[4];
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
          bool bad = row >= seen;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            bad |= (v[q] & 0x7F80u) == 0x7F80u || (v[q] & 0x7F800000u) == 0x7F800000u;
          if (bad) asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(0u) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(full);
        __syncwarp();
      }
      leave(2 * np);
      return true;
    };
    // the order of the MMA warp: K of the next tile, then V of the current one (the other way at a block's
    // end); a tile's page numbers are read two tiles ahead of their use
    ChunkTileRef a, b, c, d;
    bool has_b, has_c, has_d;
    cur.next(a);
    int pa = page_of(a), pb = 0, pc = 0, pd = 0;
    has_b = cur.next(b);
    if (has_b) pb = page_of(b);
    has_c = has_b && cur.next(c);
    if (has_c) pc = page_of(c);
    pa = checked(pa);
    ok = copy_k(a, pa, a, 0, false);
    int bring_b = bring(has_b ? b : a), bring_c = has_c && c.first ? bring(c) : bring_b;
    if (has_b) pb = checked(pb);
    while (ok) {
      has_d = has_c && cur.next(d);
      if (has_d) pd = page_of(d);
      if (has_c) pc = checked(pc);
      if (has_b && bring_b == kSweep) sweep(b, pb);
      const bool ahead = has_c && bring_c == kAhead;
      if (has_b && !b.first && !(ok = copy_k(b, pb, c, pc, ahead))) break;
      if (!(ok = copy_v(a, pa)) || !has_b) break;
      if (b.first && !(ok = copy_k(b, pb, c, pc, ahead))) break;
      a = b;
      pa = pb;
      b = c;
      pb = pc;
      bring_b = bring_c;
      c = d;
      pc = pd;
      if (has_d && d.first) bring_c = bring(d);
      has_b = has_c;
      has_c = has_d;
    }
  } else if (warp == 6) {
    // ================================================================ MMAs
    if (rank == 0) {
      constexpr uint32_t id_qk = idesc_bf16_f32(128, 256, 0, 0), id_pv = idesc_bf16_f32(128, 256, 0, 1);
      // descriptors: an address 16 n bytes further is n more in the low word
      const uint64_t desc_q = smem_desc(base + CK_Q, 16, 1024, kSwizzle128B), desc_p = smem_desc(base + CK_P, 16, 1024, kSwizzle128B);
      const uint64_t desc_k = smem_desc(base + CK_RING, 16, 1024, kSwizzle128B);
      const uint64_t desc_v = smem_desc(base + CK_RING, kCkBlk, 1024, kSwizzle128B);
      const bool el = elect_one();
      uint32_t slot = 0, phase = 0, g = 0, piece = 0;
      uint32_t at = 0;  // the slot at hand
      // Each lane waits for itself: a vote on every slot costs 3% of the kernel.  Lanes can part only
      // where a wait runs out; no lane waits for another before all have left these loops.
      auto wait = [&](uint32_t b, uint32_t parity, int site) -> bool { return wait_one<true>(b, parity, wc, site); };
      // (bytes that a copy brought are the barrier's to order; rows that a warp of the other CTA wrote --
      // `written` -- need an acquire of the pair's scope)
      auto take = [&](bool written) -> bool {
        const uint32_t full = bar(CB_FULL + slot);
        if (!((!written && mbar_try_wait(full, phase)) || wait(full, phase, kSiteCkRing))) return false;
        at = slot;
        if (++slot == kCkSlots) {
          slot = 0;
          phase ^= 1;
        }
        return true;
      };
      auto qk = [&](const ChunkTileRef& r, uint32_t t) -> bool {
        if (r.first) {
          if (!wait(bar(CB_Q_FULL), piece & 1, kSiteCkQ)) return false;
          ++piece;
        }
        // (tile t - 2's scores are read: its P has been waited for)
        tc_fence_after();
        const uint32_t d_tmem = tmem + CT_S + 128 * (t & 1);
#pragma unroll
        for (int d = 0; d < 9; ++d) {
          if (!take(false)) return false;
          const uint64_t da = desc_q + d * (kCkBlk >> 4), db = desc_k + at * (kCkSlot >> 4);
          if (el) {
            mma2_bf16_ss(d_tmem, da, db, id_qk, d ? 1u : 0u);
            mma2_bf16_ss(d_tmem, da + 2, db + 2, id_qk, 1u);
            mma2_bf16_ss(d_tmem, da + 4, db + 4, id_qk, 1u);
            mma2_bf16_ss(d_tmem, da + 6, db + 6, id_qk, 1u);
            mma2_commit_both(bar(CB_EMPTY + at));
          }
        }
        if (el) {
          mma2_commit_both(bar(CB_S_FULL + (t & 1)));
          if (r.last) mma2_commit_both(bar(CB_Q_EMPTY));
        }
        return true;
      };
      auto pv = [&](const ChunkTileRef& r, uint32_t t) -> bool {
        if (!wait(bar(CB_P_FULL), t & 1, kSiteCkP)) return false;
        tc_fence_after();
        const int np = r.pages(), some = chunk_visible(r.b, 0, args.key.causal);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          if (kb >= np) break;
          const bool written = kChunkTile * r.tile + 64 * kb + 64 > some;  // the copying warp looked through it
          const int steps = (min(r.vis - kChunkTile * r.tile - 64 * kb, 64) + 15) >> 4;
          const uint32_t acc = !r.first || kb > 0 ? 1u : 0u;
          const uint64_t da = desc_p + kb * (kCkBlk >> 4);
          // Both halves of the dims together: one pause for two slots (133.1 against 139.9 us for prompt pieces,
          // 2.68 against 2.82 ms for a long append), and P read once for two MMAs (132.7 us, 2.65 ms).
          if (!take(written)) return false;
          const uint32_t first = at;
          if (!take(written)) return false;
          const uint64_t b0 = desc_v + first * (kCkSlot >> 4), b1 = desc_v + at * (kCkSlot >> 4);
          if (el) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k == 0 || k < steps)
                mma2_bf16_ss_twice(tmem + CT_O, tmem + CT_O + 128, da + 2 * k, b0 + 128 * k, b1 + 128 * k, id_pv, k ? 1u : acc);
            mma2_commit_both(bar(CB_EMPTY + first));
            mma2_commit_both(bar(CB_EMPTY + at));
          }
        }
        if (el) mma2_commit_both(bar(CB_P_FREE));
        return true;
      };
      ChunkTileRef a, b;
      cur.next(a);
      bool ok = qk(a, 0);
      while (ok) {
        // scores of the next tile first, so that the softmax always has one; but a block's last PV before
        // the next block's first QK, whose query is loaded meanwhile
        const bool more = cur.next(b);
        if (more && !b.first && !(ok = qk(b, g + 1))) break;
        if (!(ok = pv(a, g)) || !more) break;
        if (b.first && !(ok = qk(b, g + 1))) break;
        a = b;
        ++g;
      }
      // no MMA may still run, and no copy may still land, when the pair leaves
      if (el) mma2_commit_both(bar(CB_DRAIN));
      __syncwarp();
      WaitCtx wd = wc;
      wd.timeout_ns = 100000000ull;
      volatile int no_abort = 0;
      wd.abort_local = &no_abort;
      wd.abort_peer = 0;
      wait_warp<true>(bar(CB_DRAIN), 0, wd, kSiteCkDrain);
    }
  } else if (warp == 7) {
    // ================================================================ query copies
    // (the next block's rows are brought into L2 while this block runs)
    ChunkTileRef r;
    uint32_t piece = 0;
    const uint32_t full = lead0 + 8 * CB_Q_FULL;
    const bool el = elect_one();
    while (cur.next(r)) {
      const int row = r.b.tok0 * args.key.heads + 64 * (int)rank;
      if (piece > 0) {
        if (el) {
          tma_prefetch_3d(&args.map_q, 0, row, 0);
          tma_prefetch_2d(&args.map_qr, 0, row);
        }
        __syncwarp();
        if (!wait_warp<true>(bar(CB_Q_EMPTY), (piece - 1) & 1, wc, kSiteCkQ)) break;
      }
      if (el) {
        mbar_arrive_expect_tx_remote(full, 9 * kCkBlk);
        tma2_load_3d(base + CK_Q, &args.map_q, full, 0, row, 0);
        tma2_load_2d(base + CK_Q + 8 * kCkBlk, &args.map_qr, full, 0, row);
      }
      __syncwarp();
      ++piece;
      cur.skip_block();
    }
  } else {
    // ================================================================ softmax
    const int w = (warp - 8) >> 2, quarter = warp & 3;
    const int L = 32 * quarter + lane, row = L & 63, hi = L >> 6;
    const int part = 2 * hi + w;                     // this thread's keys of a tile: [64 part, 64 part + 64)
    const int r = 64 * (int)rank + row;              // row of the block
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const uint32_t prow = base + CK_P + part * kCkBlk + row * 128;
    float* red = reinterpret_cast<float*>(smem + CK_RED);
    float* sums = reinterpret_cast<float*>(smem + CK_SUM);
    const float sl2 = args.scale_log2;
    const int col0 = 256 * w + 128 * hi;             // output dims [col0, col0 + 128)
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;

    // O / l of a finished piece -> its rows of out, or a split partial
    uint32_t pieces = 0;
    auto epilogue = [&](const ChunkTileRef& e) -> bool {
      sums[part * 64 + row] = l_run;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(CB_SUM));
      if (!wait_warp(bar(CB_SUM), pieces & 1, wc, kSiteCkRed)) return false;
      ++pieces;
      const float l = sums[row] + sums[64 + row] + sums[128 + row] + sums[192 + row];
      const int rows = e.b.ntok * args.key.heads - (r - lane);  // rows of this warp's 32 that the block has
      const bool split = e.b.splits > 1;
      const bool none = e.vis == 0;  // no tile had keys: the accumulator was never written
      const uint64_t inv = splat_f32x2(l == 0.f ? 0.f : 1.f / l);
      const int64_t q_row = (int64_t)e.b.tok0 * args.key.heads + r, slot = e.b.offset + e.split;
      const uint32_t acc = tmem + lane_off + CT_O + 128 * w;
      if (split) {
        // partials stay in the accumulator's order, [slot][CTA][warp][4 columns][lane]: whole 512-byte
        // stores straight from the registers
        float4* dst = reinterpret_cast<float4*>(args.o_acc) + (((slot * 2 + rank) * 8 + (warp - 8)) * 32) * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(acc + 32 * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float x[4];
            unpack_f32x2(fmul_f32x2(pack_b32x2(v[4 * q], v[4 * q + 1]), inv), x[0], x[1]);
            unpack_f32x2(fmul_f32x2(pack_b32x2(v[4 * q + 2], v[4 * q + 3]), inv), x[2], x[3]);
            if (lane < rows) dst[(8 * c + q) * 32] = make_float4(x[0], x[1], x[2], x[3]);
          }
        }
      } else {
        // rows through the warp's own 4 KB of the P buffer (its rows' chunks, free once PV is done), so
        // that eight lanes write 128 bytes of a row: 16-byte chunks, XOR-swizzled by row both ways
        const int sub = lane >> 3, chk = lane & 7;
        const uint32_t mine = prow + ((uint32_t)(row & 7) << 4), region = prow - lane * 128;
        uint8_t* dst = reinterpret_cast<uint8_t*>(args.out + (q_row - lane + sub) * 512 + col0) + 16 * chk;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {  // 64 columns a round: 128 bytes of a row
          uint32_t v[64];
          tmem_ld32(acc + 64 * c, *reinterpret_cast<uint32_t(*)[32]>(v));
          tmem_ld32(acc + 64 * c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x0, x1;
              unpack_f32x2(fmul_f32x2(pack_b32x2(v[8 * q + 2 * k], v[8 * q + 2 * k + 1]), inv), x0, x1);
              o[k] = none ? 0u : pack_bf16(x0, x1);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(mine ^ (uint32_t)(q << 4)), "r"(o[0]), "r"(o[1]),
                         "r"(o[2]), "r"(o[3])
                         : "memory");
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rw = 4 * i + sub;
            uint4 o;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                         : "r"(region + rw * 128 + ((uint32_t)(chk ^ (rw & 7)) << 4))
                         : "memory");
            if (rw < rows) *reinterpret_cast<uint4*>(dst + 4096 * i + 128 * c) = o;
          }
          __syncwarp();
        }
      }
      if (lane < rows && part == 0) {
        const float lse = l == 0.f ? -INFINITY : (m_run + log2f(l)) * 0.69314718055994530942f;
        if (split) args.lse_acc[slot * kChunkRows + r] = lse; else args.lse[q_row] = lse;
      }
      return true;
    };

    ChunkTileRef a;
    int lim = 0, some = 0;
    uint32_t g = 0;
    for (; ok && cur.next(a); ++g) {
      if (a.first) {
        const int j = r / args.key.heads;  // this row's token of the block
        lim = j < a.b.ntok ? chunk_visible(a.b, j, args.key.causal) : 0;
        some = chunk_visible(a.b, 0, args.key.causal);
      }
      const uint32_t sb = g & 1;
      if (!(ok = wait_warp<true>(bar(CB_S_FULL + sb), (g >> 1) & 1, wc, kSiteCkScores))) break;
      tc_fence_after();
      uint32_t sv[64];
      float least[2];
      tmem_ld32_min(tmem + lane_off + CT_S + 128 * sb + 64 * w, *reinterpret_cast<uint32_t(*)[32]>(sv), least[0]);
      tmem_ld32_min(tmem + lane_off + CT_S + 128 * sb + 64 * w + 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32), least[1]);
      tmem_wait_ld();
      // A seen score of -inf makes the row NaN.  (The maximum and exp(-inf) = 0 would lose it, and whether a token feels
      // such a key would depend on the tile it lies in; +inf and NaN show by themselves.)  The least score comes with
      // the load: found by instructions of its own it cost 1% of prompt pieces and 2-3% of a long append.
      if (kChunkTile * (a.tile + 1) > some || r >= a.b.ntok * args.key.heads) {
        // keys this row sees of the thread's 64 (what is not finite in their value rows was zeroed)
        const int nv = lim - (kChunkTile * a.tile + 64 * part);
#pragma unroll
        for (int j = 0; j < 64; ++j)
          sv[j] = j < nv ? (sv[j] == 0xFF800000u ? 0x7FC00000u : sv[j]) : 0xFF800000u;
      } else if (fminf(least[0], least[1]) == -INFINITY) {
        sv[0] = 0x7FC00000u;
      }
      float mt;
      {
        float c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) c[q] = fmaxf(__uint_as_float(sv[2 * q]), __uint_as_float(sv[2 * q + 1]));
#pragma unroll
        for (int j = 8; j < 64; j += 2)
          c[(j >> 1) & 3] = fmax3(c[(j >> 1) & 3], __uint_as_float(sv[j]), __uint_as_float(sv[j + 1]));
        mt = fmax3(c[0], c[1], fmaxf(c[2], c[3]));
      }
      red[(sb * 4 + part) * 64 + row] = mt;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(CB_RED + sb));
      if (!(ok = wait_warp(bar(CB_RED + sb), (g >> 1) & 1, wc, kSiteCkRed))) break;
      const float* rr = red + sb * 256 + row;
      const float cm = fmax3(rr[0], rr[64], fmaxf(rr[128], rr[192])) * sl2;  // log2 units (sl2 > 0)
      const float m_old = a.first ? -INFINITY : m_run;
      const bool grow = cm > m_old + 8.f;  // also the first keys that the row sees
      const float m_new = grow ? cm : m_old;
      const float alpha = grow ? exp2f(m_old - cm) : 1.f;
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      uint32_t pp[32];
      float ls;
      {
        const uint64_t s2 = splat_f32x2(sl2), nm = splat_f32x2(-m_use);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float x0, x1;
          unpack_f32x2(ffma_f32x2(pack_b32x2(sv[2 * j], sv[2 * j + 1]), s2, nm), x0, x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          // P in bf16, the type of V in the tensor cores (half a step is 2^-8 of a weight at most, of either sign); the row's sum
          // takes the float32 weights, so that lse is not rounded with them
          pp[j] = pack_bf16(p0, p1);
          acc[j & 3] = fadd_f32x2(acc[j & 3], pack_f32x2(p0, p1));
        }
        float z0, z1;
        unpack_f32x2(fadd_f32x2(fadd_f32x2(acc[0], acc[1]), fadd_f32x2(acc[2], acc[3])), z0, z1);
        ls = z0 + z1;
      }
      // PV of the tile before is done: P may be overwritten, O read and rescaled
      if (g > 0 && !(ok = wait_warp<true>(bar(CB_P_FREE), (g - 1) & 1, wc, kSiteCkPv))) break;
      tc_fence_after();
      if (!a.first && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_off + CT_O + 128 * w + 32 * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
          tmem_st32(tmem + lane_off + CT_O + 128 * w + 32 * c, v);
        }
        tmem_wait_st();
      }
      l_run = (a.first ? 0.f : l_run * alpha) + ls;
      m_run = m_new;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(prow + ((uint32_t)(c ^ (row & 7)) << 4)), "r"(pp[4 * c]),
                     "r"(pp[4 * c + 1]), "r"(pp[4 * c + 2]), "r"(pp[4 * c + 3])
                     : "memory");
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(lead0 + 8 * CB_P_FULL);
      if (a.last) {  // (the next block's scores are computed meanwhile)
        if (!(ok = wait_warp<true>(bar(CB_P_FREE), g & 1, wc, kSiteCkPv))) break;
        tc_fence_after();
        if (!(ok = epilogue(a))) break;
      }
    }
    tc_fence_before();
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  __syncthreads();
  if (*abort_flag) drain_delay(200000);  // in-flight copies and MMAs land before release
  cluster_sync();
  if (warp == 6) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ----------------------------------------------------------------- merge of split blocks
// out = sum_i exp(lse_i - lse) out_i over the units that shared a block.  Three blocks of eight warps per SM
// stride over the items.  An item is the 32 rows x 128 dims that one of the 2 x 8 warps of the attention wrote,
// or a quarter of them by pieces:
//   Fewer than eight pieces a block on average: a warp takes 16 of the dims (32 bytes of a bf16 row) over all
//   pieces, two in flight; nothing is exchanged.  24 blocks of three pieces 66 us with the attention, 75 the
//   other way; 75 blocks of two 202 against 225 (dealt out whole since then, they need none).
//   Eight or more (then there are few blocks, and a warp of a row's own would run alone through them): an item
//   is 16 of the dims, each warp takes every eighth piece, and they meet in shared memory.  One block of 74
//   pieces 52 us with the attention, 84 the other way; 2 of 32 16 against 29; 8 of 8 28.6 against 29.0.
// Merging inside the attention kernel instead, by whichever unit comes last (a counter per warp), took as
// long: 7 us more there against 9 us here.
template <int kCols>
struct ChunkMerge {  // running log-sum-exp merge of one row's float4 columns
  float M = -INFINITY, S = 0.f;
  bool nan = false;  // a partial of NaN keys: the maximum would not show it
  float4 acc[kCols];
  __device__ ChunkMerge() {
#pragma unroll
    for (int f = 0; f < kCols; ++f) acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // partials k: sums of weights s_k and of weighted rows v_k, both relative to exp(x_k)
  template <int kN>
  __device__ void add(const float (&x)[kN], const float (&s)[kN], const float4 (&v)[kN][kCols]) {
    float top = M;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      nan |= isnan(x[k]);
      top = fmaxf(top, x[k]);
    }
    const float scale = top == M ? 1.f : expf(M - top);  // (0 before the first keys)
    M = top;
    S *= scale;
#pragma unroll
    for (int f = 0; f < kCols; ++f) acc[f] = make_float4(acc[f].x * scale, acc[f].y * scale, acc[f].z * scale, acc[f].w * scale);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const float wk = M == -INFINITY ? 0.f : expf(x[k] - M);
      S += wk * s[k];
#pragma unroll
      for (int f = 0; f < kCols; ++f) {
        acc[f].x += wk * v[k][f].x;
        acc[f].y += wk * v[k][f].y;
        acc[f].z += wk * v[k][f].z;
        acc[f].w += wk * v[k][f].w;
      }
    }
  }
  __device__ void store(__nv_bfloat16* dst, float* lse_row) const {
    const float inv = nan ? NAN : M == -INFINITY ? 0.f : 1.f / S;
    uint32_t o[2 * kCols];
#pragma unroll
    for (int f = 0; f < kCols; ++f) {
      o[2 * f] = pack_bf16(acc[f].x * inv, acc[f].y * inv);
      o[2 * f + 1] = pack_bf16(acc[f].z * inv, acc[f].w * inv);
    }
    if constexpr (kCols == 1) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
    } else {
#pragma unroll
      for (int f = 0; f < kCols / 2; ++f)
        *reinterpret_cast<uint4*>(dst + 8 * f) = make_uint4(o[4 * f], o[4 * f + 1], o[4 * f + 2], o[4 * f + 3]);
    }
    if (lse_row) *lse_row = nan ? NAN : M == -INFINITY ? -INFINITY : M + logf(S);
  }
};

__global__ void __launch_bounds__(256) mla_chunk_combine_kernel(const int32_t* sched, ChunkKey key, const float* o_acc,
                                                                const float* lse_acc, __nv_bfloat16* out, float* lse) {
  __shared__ float4 sh_acc[8][4][32];
  __shared__ float sh_m[8][32], sh_s[8][32];
  pdl_wait_prerequisites();
  const ChunkLayout lay = chunk_layout(key.units, key.capacity, key.batch);
  const int H = key.heads;
  const int4 *h = reinterpret_cast<const int4*>(sched), h0 = h[0], h1 = h[1], h2 = h[2], h3 = h[3];
  static_assert(kChSlots == 4 && kChNumSplit == 7, "header");
  if (!chunk_plan_is(h0, h2, h3, key)) return;
  const bool fine = h1.x >= 8 * h1.w;  // slots against split blocks
  const int per = fine ? 128 : 16, step = fine ? 8 : 1, items = per * h1.w, lane = threadIdx.x & 31, j = threadIdx.x >> 5;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int4* rec = reinterpret_cast<const int4*>(sched + lay.split_list) + 2 * (it / per);
    const int4 lo = rec[0], hi = rec[1];
    ChunkBlock b;
    b.tok0 = lo.x; b.ntok = lo.y; b.splits = hi.z; b.offset = hi.w;
    const int writer = it & 15, wi = writer & 7, L = 32 * (wi & 3) + lane, row = 64 * (writer >> 3) + (L & 63);
    const bool on = row < b.ntok * H;
    const int col = fine ? 4 * ((it >> 4) & 7) : 4 * j;  // float4 columns [col, col + 4) of the 32
    const int64_t q_row = (int64_t)b.tok0 * H + row;
    __nv_bfloat16* dst = out + q_row * 512 + 256 * (wi >> 2) + 128 * (L >> 6) + 4 * col;
    float* lse_row = wi < 2 && col == 0 ? lse + q_row : nullptr;  // (one of the four lanes that hold the row)
    const float* lsrc = lse_acc + (int64_t)b.offset * kChunkRows + row;
    const float4* src = reinterpret_cast<const float4*>(o_acc) + (((int64_t)b.offset * 16 + writer) * 32 + col) * 32 + lane;
    constexpr int64_t kStep = 16 * 32 * 32;  // float4 per piece
    ChunkMerge<4> m;
    for (int i0 = fine ? j : 0; on && i0 < b.splits; i0 += 2 * step) {
      float4 v[2][4];
      float x[2], s[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = i0 + k * step;
        const bool in = i < b.splits;
        x[k] = in ? lsrc[(int64_t)i * kChunkRows] : -INFINITY;
        s[k] = 1.f;
#pragma unroll
        for (int f = 0; f < 4; ++f) v[k][f] = in ? __ldcs(src + i * kStep + 32 * f) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      m.add(x, s, v);
    }
    if (!fine) {
      if (on) m.store(dst, lse_row);
      continue;
    }
    __syncthreads();  // (the item before has been read)
    sh_m[j][lane] = m.nan ? NAN : m.M;
    sh_s[j][lane] = m.S;
#pragma unroll
    for (int f = 0; f < 4; ++f) sh_acc[j][f][lane] = m.acc[f];
    __syncthreads();
    if (j < 4 && on) {
      ChunkMerge<1> t;
      float4 v[8][1];
      float x[8], s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = sh_m[i][lane];
        s[i] = sh_s[i][lane];
        v[i][0] = sh_acc[i][j][lane];
      }
      t.add(x, s, v);
      t.store(dst + 4 * j, j == 0 ? lse_row : nullptr);
    }
  }
}

// ----------------------------------------------------------------- FP8 and INT4 rows -> bf16 rows
// Formats of a cached token, as in mla_kv_dtype.
enum : int { kKvBf16 = 0, kKvFp8 = 1, kKvInt4 = 2 };

// A quantised row by a warp, 16 latent values a lane: bf16(code x scale), RoPE copied.
template <int kFmt>
__device__ __forceinline__ void expand_row(const uint8_t* src, __nv_bfloat16* dst, int lane) {
  uint32_t o[8];
  if constexpr (kFmt == kKvFp8) {
    const uint4 c = *reinterpret_cast<const uint4*>(src + 16 * lane);
    const float s = *reinterpret_cast<const float*>(src + 512 + 4 * (lane >> 3));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[q >> 1] >> (16 * (q & 1)));
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3));  // exact
      const float2 f = __half22float2(h);
      o[q] = pack_bf16(f.x * s, f.y * s);
    }
  } else {
    static_assert(kFmt == kKvInt4, "format");
    const uint2 c = *reinterpret_cast<const uint2*>(src + 8 * lane);
    const uint32_t s = *reinterpret_cast<const uint16_t*>(src + kI4Codes + (lane & ~1));
    const uint32_t s2 = int4_scale_overflows(s) ? kI4Nan : s | s << 16, a2 = int4_offset(s2);
    expand_int4_word(c.x, s2, a2, reinterpret_cast<uint32_t(&)[4]>(o[0]));
    expand_int4_word(c.y, s2, a2, reinterpret_cast<uint32_t(&)[4]>(o[4]));
  }
  uint4* d = reinterpret_cast<uint4*>(dst + 16 * lane);
  d[0] = make_uint4(o[0], o[1], o[2], o[3]);
  d[1] = make_uint4(o[4], o[5], o[6], o[7]);
  if (lane < 8) *reinterpret_cast<uint4*>(dst + 512 + 8 * lane) = *reinterpret_cast<const uint4*>(src + (kFmt == kKvFp8 ? 528 : kI4Rope) + 16 * lane);
}

// The pages of the sequences that have new tokens, expanded once per call into consecutive bf16
// pages (sequence b's from page_off[b]): value = bf16(code x scale), RoPE copied.  A chunk's rows
// read every cached row many times over, so 1808 bytes of traffic a cached token stand against
// 278,528 FLOP per new token at 128 heads.  A warp takes a row: lane l the codes [16 l, 16 l + 16).
// 63,900 rows in 26 us, 4.5 TB/s, 3% of the attention over them; two or eight rows of a warp in flight
// instead of four, or half a page a block, changed nothing.  Where a row has one reader nothing pays for
// it: 64 x 1 token x 16 heads over 8192 FP8 rows take 307 us, over bf16 rows 122.
template <int kFmt>
__global__ void __launch_bounds__(256) mla_chunk_expand_kernel(const int32_t* sched, ChunkKey key, const uint8_t* pages,
                                                               const int32_t* block_table, int num_pages, const int32_t* lens,
                                                               __nv_bfloat16* rows) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int4* h = reinterpret_cast<const int4*>(sched);
  if (!chunk_plan_is(h[0], h[2], h[3], key)) return;
  const ChunkLayout lay = chunk_layout(key.units, key.capacity, key.batch);
  const int32_t* page_off = sched + lay.page_off;
  const int total = sched[kChPages], warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int pg = blockIdx.x; pg < total; pg += gridDim.x) {
    const int b = chunk_find(page_off, key.batch, pg), lp = pg - page_off[b];
    int page = block_table[(int64_t)b * key.max_pages + lp];
    if (page < 0 || page >= num_pages) {
      if (threadIdx.x == 0) atomicCAS(&g_mla_error, 0, 1);
      page = 0;
    }
    const int n = min(lens[b] - 64 * lp, 64);  // rows past the sequence's end are not expanded
#pragma unroll 4
    for (int r = warp; r < n; r += 8) {
      constexpr int kRow = kFmt == kKvFp8 ? 656 : kI4Row;
      expand_row<kFmt>(pages + ((int64_t)page * 64 + r) * kRow, rows + ((int64_t)pg * 64 + r) * 576, lane);
    }
  }
}

// ----------------------------------------------------------------- scheduler
// Exclusive prefix sum over the 1024 threads of a CTA; total of all threads in *sum.
__device__ __forceinline__ int64_t block_scan_1024(int64_t v, int64_t* sh, int64_t* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // (sh may still be read from the scan before)
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t s = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sh[lane] = s;
  }
  __syncthreads();
  *sum = sh[31];
  return x - v + (warp > 0 ? sh[warp - 1] : 0);
}

// One CTA of 1024 threads; the phases of chunk_plan_host with the sums in parallel.
// 10 us with 8 blocks, 14-24 with 225 to 580 to deal (cold): dependent trips to L2 and barriers, once a step
// for all layers.
__global__ void __launch_bounds__(1024) mla_chunk_sched_kernel(const int32_t* cu, const int32_t* lens, int B,
                                                               int64_t max_tokens, int H, int causal, int max_pages,
                                                               int64_t max_kv_pages, int U, int64_t cap, int32_t* sched) {
  __shared__ int64_t sh[32];
  __shared__ int bad, sh_share;
  __shared__ int sort_key[kChunkSortSeqs], sort_blocks[kChunkSortSeqs], sort_at[kChunkSortSeqs];
  __shared__ int load[kChunkDealUnits], unit_at[kChunkDealUnits], sh_most;
  const int tid = threadIdx.x, tb = chunk_tokens_per_block(H);
  const ChunkLayout l = chunk_layout(U, cap, B);
  ChunkBlock* blocks = reinterpret_cast<ChunkBlock*>(sched + l.blocks);
  int32_t *page_off = sched + l.page_off, *blk_off = sched + l.blk_off, *pos = sched + l.pos;
  if (tid == 0) bad = cu[0] != 0;
  if (tid < kChunkHeader) sched[tid] = 0;
  __syncthreads();
  for (int b = tid; b < B; b += 1024)
    if (!chunk_sequence_ok(cu[b], cu[b + 1], lens[b], max_tokens, max_pages)) bad = 1;
  __syncthreads();
  auto refuse = [&]() {  // (the header without the magic word stands)
    if (tid == 0) atomicCAS(&g_mla_error, 0, 1);
  };
  if (bad) return refuse();
  int64_t pages = 0, nb = 0, sum;
  for (int b0 = 0; b0 < B; b0 += 1024) {
    const int b = b0 + tid;
    const int32_t n = b < B ? cu[b + 1] - cu[b] : 0;
    const int64_t pe = block_scan_1024(n > 0 ? num_tiles(lens[b]) : 0, sh, &sum);
    if (b < B) page_off[b] = (int32_t)(pages + pe);
    pages += sum;
    const int64_t be = block_scan_1024(chunk_seq_blocks(n, tb), sh, &sum);
    if (b < B) blk_off[b] = (int32_t)(nb + be);
    nb += sum;
  }
  if (pages > max_kv_pages) return refuse();
  if (tid == 0) {
    page_off[B] = (int32_t)pages;
    blk_off[B] = (int32_t)nb;
  }
  const bool sorted = nb > U && B <= kChunkSortSeqs;
  if (sorted && tid < B) {
    const int32_t n = cu[tid + 1] - cu[tid];
    sort_key[tid] = chunk_sort_key(n, lens[tid]);
    sort_blocks[tid] = chunk_seq_blocks(n, tb);
  }
  if (tid == 0) sh_most = 0;
  __syncthreads();
  if (sorted && tid < B) {
    int at = 0;
    for (int o = 0; o < B; ++o)
      if (chunk_sorts_before(sort_key[o], o, sort_key[tid], tid)) at += sort_blocks[o];
    sort_at[tid] = at;
  }
  __syncthreads();
  for (int64_t k = tid; k < nb; k += 1024) {
    const int b = chunk_find(blk_off, B, (int32_t)k), first = blk_off[b];
    blocks[sorted ? sort_at[b] + (k - first) : k] = chunk_make_block(cu, lens, b, (int)k, first, tb, causal);
  }
  __syncthreads();
  auto positions = [&]() -> int64_t {  // the blocks' places on the line, and its length
    int64_t all = 0;
    for (int64_t k0 = 0; k0 < nb; k0 += 1024) {
      const int64_t k = k0 + tid;
      const int32_t cost = k < nb ? chunk_cost(blocks[k].nt) : 0;
      const int64_t e = block_scan_1024(cost, sh, &sum);
      if (k < nb) pos[k] = (int32_t)(all + e);
      all += sum;
    }
    return all;
  };
  const int64_t total = positions();
  if (total > kMaxPlanPositions) return refuse();
  __syncthreads();
  bool shares = nb <= U;
  int64_t budget = plan_budget(total, U);
  if (shares) {
    if (tid < 32) {  // the least share that U units suffice for
      int32_t longest = 1;
      for (int k = tid; k < nb; k += 32) longest = max(longest, blocks[k].nt);
      longest = __reduce_max_sync(0xffffffffu, longest);
      int32_t lo = 1, hi = longest;
      while (lo < hi) {
        const int32_t m = (lo + hi) / 2;
        int32_t need = 0;  // (at most U + NB < 2^18 until it no longer matters)
        for (int k = tid; k < nb; k += 32) need = min(need + chunk_shares(blocks[k].nt, m), 1 << 24);
        if (__reduce_add_sync(0xffffffffu, need) <= U) hi = m; else lo = m + 1;
      }
      if (tid == 0) sh_share = chunk_share_tiles(longest, lo, budget);
    }
    __syncthreads();
    shares = sh_share > 0;
    if (shares) budget = sh_share;
  }
  bool dealt = false;
  if (sorted && U <= kChunkDealUnits) {
    int32_t* owner = pos;  // (for a while)
    int mine = 0, count = 0;
    for (int64_t k0 = 0; k0 < nb; k0 += U) {
      if (tid < U) load[tid] = mine;
      __syncthreads();
      if (tid < U) {
        int64_t k = k0;
        for (int v = 0; v < U; ++v) k += load[v] < mine || (load[v] == mine && v < tid);
        if (k < nb) {
          mine += chunk_cost(blocks[k].nt);
          ++count;
          owner[k] = tid;
        }
      }
      __syncthreads();
    }
    if (tid < U) atomicMax(&sh_most, mine);
    const int64_t first = block_scan_1024(count, sh, &sum);
    if (tid < U) unit_at[tid] = (int)first;
    __syncthreads();
    dealt = chunk_is_dealt(sh_most, budget, pages);
    if (dealt) {  // the blocks of a unit one after another
      budget = sh_most;
      for (int64_t k = tid; k < nb; k += 1024) {
        const int b = chunk_find(blk_off, B, (int32_t)k), lead = blk_off[b];
        const int64_t s = sort_at[b] + (k - lead);
        blocks[unit_at[owner[s]] + s / U] = chunk_make_block(cu, lens, b, (int)k, lead, tb, causal);
      }
      __syncthreads();
      for (int u = tid; u < U; u += 1024) load[u] = u + 1 < U ? unit_at[u + 1] : (int)nb;
    }
    __syncthreads();
    positions();
    __syncthreads();
  }
  int64_t slots = 0, ns = 0, at = 0;
  for (int64_t k0 = 0; k0 < nb; k0 += 1024) {
    const int64_t k = k0 + tid;
    const int32_t s = k >= nb ? 0
                      : dealt ? 1
                      : shares ? chunk_shares(blocks[k].nt, (int32_t)budget)
                               : chunk_splits(pos[k], blocks[k].nt, budget);
    const int64_t oe = block_scan_1024(s > 1 ? s : 0, sh, &sum);
    const int64_t o = slots + oe;
    slots += sum;
    const int64_t le = block_scan_1024(s > 1 ? 1 : 0, sh, &sum);
    if (k < nb) {
      blocks[k].splits = s;
      blocks[k].offset = (int32_t)o;
      if (s > 1) reinterpret_cast<ChunkBlock*>(sched + l.split_list)[ns + le] = blocks[k];
    }
    ns += sum;
    if (shares) {
      const int64_t ae = block_scan_1024(s, sh, &sum);
      if (k < nb) pos[k] = (int32_t)(at + ae);
      at += sum;
    }
  }
  __syncthreads();
  for (int u = tid; u < U; u += 1024) {
    int32_t* rec = sched + l.units + kChunkUnitInts * u;
    if (dealt)
      chunk_deal_unit(blocks, unit_at[u], load[u], rec);
    else if (shares)
      chunk_share_unit(blocks, pos, (int)nb, at, u, rec);
    else
      chunk_unit(blocks, pos, (int)nb, total, budget, u, rec);
  }
  if (tid == 0) {
    chunk_write_key(sched, {U, (int32_t)cap, B, causal, (int32_t)max_tokens, H, max_pages, (int32_t)max_kv_pages});
    sched[kChBlocks] = (int32_t)nb;
    sched[kChSlots] = (int32_t)slots;
    sched[kChBudget] = (int32_t)budget;
    sched[kChTokens] = tb;
    sched[kChNumSplit] = (int32_t)ns;
    sched[kChPages] = (int32_t)pages;
    sched[kChShares] = dealt ? 2 : shares;
    sched[kChMagic] = kChunkMagic;
  }
}

}  // namespace mla
