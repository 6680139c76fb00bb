// Absorbed-MLA decode over INT4 pages: for every new token and head s_j = scale (q~ . c_j + q^R . k^R_j) over
// the keys it may see, out = sum_j softmax(s)_j c_j, lse = ln sum_j exp(s_j), where the latent c_j is
// held as 512 four-bit codes n and 16 scales, c = (n - 8) scale  ("MLA inference: two computation paths and
// FlashMLA", section "Decode attention becomes a compute problem").
//
// What bounds it: a key is 416 bytes and 2176 FLOP for each row (token and head) that reads it, so up to ~50 rows a key
// HBM, beyond that the tensor cores; and a key's 512 values have to become bf16 in every SM that reads it.
//
// Work split.  The keys are the M dimension: S^T = K Q^T and O^T = C^T P^T.  A tile is 128 keys (two pages),
// expanded once into shared memory as bf16, and that one copy is both products' A operand (K-major for the scores, MN-major for
// the output), so a CTA needs no other's help: up to 64 rows are its N = 16, 32 or 64 columns, O^T is 4 x [128 dims x N]
// in tensor memory.  A unit of the plan is one CTA, or two for 65 to 128 heads, which read the same pages at the
// same time (the second from L2).  With several new tokens a sequence, as many as fit into 64 rows share every key.
//
// MMA rates, M = 128, K = 16, cta_group::1: A from shared memory 39 / 40 / 48 cycles for N = 16 / 32 / 64 (4 KB of A and
// 32 N bytes of B at 128 bytes a cycle, K- or MN-major alike, stores beside it cost nothing); A from tensor memory 12 / 17 / 32.
//
// The quarters of a tile (128 dims, 32 KB) go through a ring of four slots (five up to 32 rows): a quarter is
// expanded into its slot as soon as the output product of the tile before has left it.
//
// Roles (five warpgroups): warps 0..7 softmax (two warpgroups, half of the columns each; a thread holds one key, so a
// row's maximum lies across lanes: scores are taken against the maximum so far, and only where one exceeds it by 2^8 are the
// new maxima found and O rescaled); warps 8..15 read the pages into registers, a tile ahead, and expand them; warp 16
// loads the queries; warp 17 issues the MMAs; two are idle and give their registers to the others.
#pragma once
#include "common.cuh"
#include "decode_kernel.cuh"  // packed float pairs, bf16 packing, mma_bf16_ts
#include "int4_rows.cuh"

namespace mla {

constexpr int kI4Threads = 640;
constexpr int kI4MaxRows = 64;         // rows of a CTA
constexpr int kI4Tile = 128;           // keys of a tile
constexpr uint32_t kI4Blk = 16384;     // [128 keys][64 dims] bf16, 128-byte swizzle
constexpr uint32_t kI4Slot = 2 * kI4Blk;

template <int N>
struct I4Smem {
  static constexpr int kSlots = N == 64 ? 4 : 5;
  static constexpr int kNc = N / 2;    // columns of a softmax warpgroup
  // registers of a thread by warpgroup: 96 each at launch (65,536 over 640 threads), dealt out anew
  static constexpr int kRegsSoftmax = N == 64 ? 112 : N == 32 ? 96 : 80, kRegsExpand = N == 64 ? 96 : N == 32 ? 104 : 112;
  static constexpr int kRegsIssue = 480 - 2 * kRegsSoftmax - 2 * kRegsExpand;
  static_assert(kRegsIssue >= 48 && kRegsIssue % 8 == 0, "registers");
  static constexpr uint32_t V = 0;
  static constexpr uint32_t Q = V + kSlots * kI4Slot;           // 9 blocks [N rows][64 dims]
  static constexpr uint32_t P = Q + 9 * N * 128;                // [128 keys][N]
  static constexpr uint32_t FLAG = P + N * 256;                 // [tile parity][warp]: some score is far above the maximum
  static constexpr uint32_t MAX = FLAG + 64;                    // [warp][kNc]: the running maxima, log2 units
  static constexpr uint32_t FAC = MAX + 8 * kNc * 4;            // [warp][kNc]: factors of a rescale or of the output
  static constexpr uint32_t XCH = FAC + 8 * kNc * 4;            // [maxima, sums][warpgroup][warp][kNc]
  static constexpr uint32_t POISON = XCH + 16 * kNc * 4;        // [tile parity][warpgroup][128 keys]
  static constexpr uint32_t BAR = POISON + 512;
  static constexpr uint32_t kBytes = BAR + 256 + 1024;          // + alignment slack
  static_assert(kBytes <= 232448, "shared memory");
};

enum : uint32_t {
  IB_FULL = 0,               // + slot: one arrival per expanding warp
  IB_EMPTY = IB_FULL + 5,    // + slot: the output product has read it
  IB_Q_FULL = IB_EMPTY + 5,
  IB_Q_EMPTY,
  IB_S_FULL,                 // + tile parity
  IB_P_FULL = IB_S_FULL + 2, // one arrival per softmax warp
  IB_PV,                     // a piece's last output product is done
  IB_FLAG,                   // + 2 warpgroup + tile parity: one arrival per warp
  IB_XCH = IB_FLAG + 4,      // + warpgroup
  IB_DRAIN = IB_XCH + 2,
  kI4Bars
};
constexpr uint32_t kI4TmemSlot = 8 * kI4Bars, kI4Abort = kI4TmemSlot + 4;
static_assert(kI4Abort + 4 <= 256, "barrier area");

enum I4Site : int { kSiteI4Ring = 44, kSiteI4Q, kSiteI4Scores, kSiteI4P, kSiteI4Pv, kSiteI4Flag, kSiteI4Drain };

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

struct I4Tile {
  int wb, key0, nkeys;   // keys [key0, key0 + nkeys) are this tile's, nkeys <= 128
  int seq, vis, split;   // vis: keys the block's last token sees
  bool first, last;      // of the unit's piece of the block
  __device__ int pages() const { return (nkeys + 63) >> 6; }
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
    r.first = false;
    while (t >= end) {
      if (++wb > wb1) return false;
      const int qb = wb * G + G - 1;
      seq = qb / s_q;
      vis = visible_keys(seqlens[seq], s_q, qb % s_q, causal);
      t = wb == wb0 ? tile0 : 0;
      end = wb == wb1 ? tile1 : num_tiles(vis);
      r.first = true;
    }
    r.wb = wb;
    r.seq = seq;
    r.vis = vis;
    r.split = wb == wb0 ? split0 : 0;
    r.key0 = kTile * t;
    r.nkeys = min(min(vis, kTile * end) - kTile * t, kI4Tile);
    t += 2;
    r.last = t >= end;
    return true;
  }
  __device__ void skip_block() { t = end; }
};

template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[NC]) {
  if constexpr (NC == 32) {
    tmem_ld32(taddr, r);
  } else if constexpr (NC == 16) {
    tmem_ld16(taddr, r);
  } else {
    static_assert(NC == 8, "columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  }
}
template <int NC>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[NC]) {
  if constexpr (NC == 32) {
    tmem_st32(taddr, r);
  } else if constexpr (NC == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  } else {
    static_assert(NC == 8, "columns");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  }
}

// Reduces NC columns held by every lane over the 32 lanes; afterwards lane l has column l / (32 / NC).
template <int NC, class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[NC], int lane, Op op) {
  int n = NC;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int k = 0; k < NC / 2; ++k)
        if (k < n) {
          const float send = (lane & o) ? v[k] : v[k + n], keep = (lane & o) ? v[k + n] : v[k];
          v[k] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return v[0];
}

__device__ __forceinline__ void ldg128(const uint8_t* p, uint32_t& x, uint32_t& y, uint32_t& z, uint32_t& w) {
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w) : "l"(p) : "memory");
}
template <int kRegs>
__device__ __forceinline__ void set_registers() {  // of a warpgroup; more than at launch once others have given theirs
  if constexpr (kRegs > 96)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else if constexpr (kRegs < 96)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
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

// The bounded waits of common.cuh in one piece: a warpgroup whose registers are dealt out anew makes no calls.
__device__ __forceinline__ bool i4_wait(uint32_t bar, uint32_t parity, const WaitCtx& w, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31) == 0) {
      if (*w.abort_local) return false;
      if (globaltimer_ns() - t0 > w.timeout_ns) {
        raise_abort(w, site);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool i4_wait_warp(uint32_t bar, uint32_t parity, const WaitCtx& w, int site) {
  return __all_sync(0xffffffffu, i4_wait(bar, parity, w, site));
}

template <int N>
__device__ __forceinline__ void decode_int4_body(const Int4Args& args) {
  using S = I4Smem<N>;
  constexpr int NC = S::kNc, kSlots = S::kSlots;
  constexpr uint32_t TO = 0, TS = 4 * N, TR = 6 * N;  // tensor memory: O^T, two score buffers, two RoPE key buffers
  static_assert(TR + 64 <= 512, "tensor memory");
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
      if (i < IB_EMPTY || i == IB_P_FULL) count = 8;
      if (i >= IB_FLAG && i < IB_DRAIN) count = 4;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (tid < 128) asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + S::POISON + 4 * tid), "r"(0u) : "memory");
  if (warp == 17) {
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
  I4Cursor cur;
  if (!idle) cur.init(args, rec);
  const int block_rows = args.group * args.H, row0 = part * args.part_rows;

  if (idle) {
  } else if (warp >= 8 && warp < 16) {
    set_registers<S::kRegsExpand>();
    // ================================================================ pages -> bf16
    // Codes: four lanes a key, 32 dims of a quarter each (16 bytes), the warp's keys 16 dw + lane / 4 (+ 8).  RoPE: a lane
    // a key, half of its 64 values; they go to tensor memory as they are.  A tile's bytes are asked for as the tile before
    // is expanded, each into the registers that its bytes have left, and its pages a tile before that.
    const int dw = warp - 8, j = lane & 3, ckey = 16 * dw + (lane >> 2), cpage = dw >> 2;
    const int rkey = 32 * (warp & 3) + lane, rpage = (warp & 3) >> 1, rhalf = dw >> 2;
    const uint32_t rope_dst = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + TR + 16 * rhalf;
    uint32_t code[8][4], scale[4], rope[16];
    // the table's entry for page `which` of a tile; a page that the tile does not have reads as the first
    auto entry_of = [&](const I4Tile& r, int which) -> int {
      const int lp = (r.key0 >> 6) + (which < r.pages() ? which : 0);
      return lp < args.max_pages ? args.block_table[(int64_t)r.seq * args.max_pages + lp] : -1;
    };
    auto row_of = [&](int page, int key) {
      if (page < 0 || page >= args.num_pages) {  // outside the contract: reported, another page read
        if (lane == 0) atomicCAS(&g_mla_error, 0, 1);
        page = 0;
      }
      return args.kv + ((int64_t)page * 64 + (key & 63)) * kI4Row;
    };
    auto load_scales = [&](const uint8_t* src) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + i * 8 * kI4Row + kI4Codes + 8 * j);
        scale[2 * i] = v.x;
        scale[2 * i + 1] = v.y;
      }
    };
    auto load_rope = [&](const uint8_t* src) {
#pragma unroll
      for (int q = 0; q < 4; ++q) ldg128(src + 16 * q, rope[4 * q], rope[4 * q + 1], rope[4 * q + 2], rope[4 * q + 3]);
    };
    I4Tile a, n, nn;
    cur.next(a);
    bool has_n = cur.next(n), ok = true;
    int table_c = 0, table_r = 0;
    {
      const uint8_t* src = row_of(entry_of(a, cpage), ckey);
      const uint8_t* src_r = row_of(entry_of(a, rpage), rkey) + kI4Rope + 64 * rhalf;
      if (has_n) {
        table_c = entry_of(n, cpage);
        table_r = entry_of(n, rpage);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t (&w)[4] = code[2 * m + i];
          ldg128(src + i * 8 * kI4Row + 64 * m + 16 * j, w[0], w[1], w[2], w[3]);
        }
      load_scales(src);
      load_rope(src_r);
    }
    uint32_t slot = 0, phase = 1;
    for (uint32_t t = 0;; ++t) {
      const uint8_t *next_c = nullptr, *next_r = nullptr;
      const bool has_nn = has_n && cur.next(nn);
      if (has_n) {
        next_c = row_of(table_c, ckey);
        next_r = row_of(table_r, rkey) + kI4Rope + 64 * rhalf;
        if (has_nn) {
          table_c = entry_of(nn, cpage);
          table_r = entry_of(nn, rpage);
        }
      }
      const int some = a.vis - (args.causal ? args.group - 1 : 0) - a.key0;  // keys from here on are not seen by every token
      const uint32_t sc[4] = {scale[0], scale[1], scale[2], scale[3]};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        ok = ok && i4_wait_warp(bar(IB_EMPTY + slot), phase, wc, kSiteI4Ring);  // (the same in all lanes)
        if (ok) {
          const uint32_t dst0 = base + S::V + slot * kI4Slot + (j >> 1) * kI4Blk;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = ckey + 8 * i;
            // the quad's lane m has the quarter's four scales
            const uint32_t lo = __shfl_sync(0xffffffffu, sc[2 * i], (lane & ~3) + m), hi = __shfl_sync(0xffffffffu, sc[2 * i + 1], (lane & ~3) + m);
            uint32_t s2 = __byte_perm((j & 2) ? hi : lo, 0, (j & 1) ? 0x3232 : 0x1010);
            if (key >= a.nkeys) {
              s2 = 0;  // no key: the products must see zeros
            } else if (key >= some && (s2 & 0x7F80u) == 0x7F80u) {
              // a key that only some of the tokens see: its values must not reach the others (0 x NaN); the softmax
              // gives NaN to those that see it
              s2 = 0;
              smem[S::POISON + 256 * (t & 1) + key] = smem[S::POISON + 256 * (t & 1) + 128 + key] = 1;
            }
            const uint32_t a2 = int4_offset(s2);
            const uint32_t dst = dst0 + key * 128, x = (uint32_t)(4 * (j & 1)) ^ (uint32_t)(key & 7);
            // lanes of the slot's second block write their chunks in another order, so that no two of a quad meet in a bank
            uint32_t (&w)[4] = code[2 * m + i];
            const uint32_t turn = j & 2;
            const uint32_t v[4] = {turn ? w[2] : w[0], turn ? w[3] : w[1], turn ? w[0] : w[2], turn ? w[1] : w[3]};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t o[4];
              expand_int4_word(v[q], s2, a2, o);
              sts128(dst + ((x ^ (uint32_t)q ^ turn) << 4), o[0], o[1], o[2], o[3]);
            }
            if (has_n) ldg128(next_c + i * 8 * kI4Row + 64 * m + 16 * j, w[0], w[1], w[2], w[3]);
          }
          if (m == 0 && has_n) load_scales(next_c);
          if (m == 2) {  // (the scores of two tiles ago are done: this tile's first slot was waited for)
            tmem_st_cols(rope_dst + 32 * (t & 1), rope);
            tmem_wait_st();
            if (has_n) load_rope(next_r);
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(IB_FULL + slot));
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok || !has_n) break;
      a = n;
      n = nn;
      has_n = has_nn;
    }
  } else if (warp >= 16) {
    set_registers<S::kRegsIssue>();
    if (warp == 16) {
    // ================================================================ queries
    I4Tile r;
    uint32_t piece = 0;
    const uint64_t keep = l2_policy_evict_last();
    while (cur.next(r)) {
      if (piece > 0 && !i4_wait_warp(bar(IB_Q_EMPTY), (piece - 1) & 1, wc, kSiteI4Q)) break;
      if (lane == 0) {
        const int row = r.wb * block_rows + row0;
        mbar_arrive_expect_tx(bar(IB_Q_FULL), 9 * N * 128);
        tma_load_3d(base + S::Q, &args.map_q, bar(IB_Q_FULL), 0, row, 0, keep);
        tma_load_2d(base + S::Q + 8 * N * 128, &args.map_qr, bar(IB_Q_FULL), 0, row, keep);
      }
      __syncwarp();
      ++piece;
      cur.skip_block();
    }
    } else if (warp == 17) {
    // ================================================================ MMAs
    constexpr uint32_t id_qk = idesc_bf16_f32(128, N, 0, 0), id_pv = idesc_bf16_f32(128, N, 1, 1);
    const uint64_t desc_k = smem_desc(base + S::V, 16, 1024, kSwizzle128B), desc_q = smem_desc(base + S::Q, 16, 1024, kSwizzle128B);
    const uint64_t desc_c = smem_desc(base + S::V, kI4Blk, 1024, kSwizzle128B);
    const uint64_t desc_p = smem_desc(base + S::P, 16, N * 16, N == 64 ? kSwizzle128B : N == 32 ? kSwizzle64B : kSwizzle32B);
    uint32_t el_;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(el_));
    const bool el = el_ != 0;
    uint32_t slot = 0, phase = 0, pv_slot = 0, piece = 0;
    // Each lane waits for itself; lanes can part only where a wait runs out, and none waits for another before all have
    // left these loops.
    auto wait = [&](uint32_t b, uint32_t parity, int site) -> bool { return i4_wait(b, parity, wc, site); };
    auto qk_quarter = [&](const I4Tile& r, uint32_t t, int m) -> bool {
      if (m == 0 && r.first) {
        if (!wait(bar(IB_Q_FULL), piece & 1, kSiteI4Q)) return false;
        ++piece;
      }
      if (!wait(bar(IB_FULL + slot), phase, kSiteI4Ring)) return false;
      tc_fence_after();
      const uint32_t d = tmem + TS + N * (t & 1);
      const uint64_t da = desc_k + slot * (kI4Slot >> 4), db = desc_q + m * (2 * N * 128 >> 4);
      if (el) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ss(d, da + (k >> 2) * (kI4Blk >> 4) + 2 * (k & 3), db + (k >> 2) * (N * 128 >> 4) + 2 * (k & 3), id_qk, m + k ? 1u : 0u);
      }
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
      return true;
    };
    auto qk_rope = [&](const I4Tile& r, uint32_t t) {  // (the RoPE keys came with the last quarter)
      if (el) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_ts(tmem + TS + N * (t & 1), tmem + TR + 32 * (t & 1) + 8 * k, desc_q + (8 * N * 128 >> 4) + 2 * k, id_qk, 1u);
        mma_commit(bar(IB_S_FULL + (t & 1)));
        if (r.last) mma_commit(bar(IB_Q_EMPTY));
      }
    };
    auto pv = [&](const I4Tile& r, uint32_t t) -> bool {
      if (!wait(bar(IB_P_FULL), t & 1, kSiteI4P)) return false;
      tc_fence_after();
      const int steps = (r.nkeys + 15) >> 4;
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        const uint64_t da = desc_c + pv_slot * (kI4Slot >> 4);
        if (el) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < steps) mma_bf16_ss(tmem + TO + N * m, da + 128 * k, desc_p + (N * 32 >> 4) * k, id_pv, r.first && k == 0 ? 0u : 1u);
          mma_commit(bar(IB_EMPTY + pv_slot));
        }
        if (++pv_slot == kSlots) pv_slot = 0;
      }
      if (el && r.last) mma_commit(bar(IB_PV));
      return true;
    };
    I4Tile a, b;
    cur.next(a);
    bool ok = true;
    for (int m = 0; ok && m < 4; ++m) ok = qk_quarter(a, 0, m);
    if (ok) qk_rope(a, 0);
    for (uint32_t t = 0; ok; ++t) {
      const bool more = cur.next(b);
      // the spare slot's quarter before the output product: it runs beside the softmax (but not before a new query is there)
      int m = 0;
      if (kSlots > 4 && more && !b.first) {
        if (!(ok = qk_quarter(b, t + 1, 0))) break;
        m = 1;
      }
      if (!(ok = pv(a, t)) || !more) break;
      for (; ok && m < 4; ++m) ok = qk_quarter(b, t + 1, m);
      if (!ok) break;
      qk_rope(b, t + 1);
      a = b;
    }
    __syncwarp();
    // no MMA may still run when the CTA leaves
    if (el) mma_commit(bar(IB_DRAIN));
    __syncwarp();
    WaitCtx wd = wc;
    wd.timeout_ns = 100000000ull;
    volatile int no_abort = 0;
    wd.abort_local = &no_abort;
    i4_wait_warp(bar(IB_DRAIN), 0, wd, kSiteI4Drain);
    }
  } else {
    set_registers<S::kRegsSoftmax>();
    // ================================================================ softmax
    const int wg = warp >> 2, w = warp & 3, key = 32 * w + lane;
    const uint32_t lanes = (uint32_t)(32 * w) << 16;
    constexpr int kC = NC < 16 ? NC : 16;               // columns at a time
    constexpr int kSpread = 32 / NC;                    // lanes that hold a column after reduce_columns
    const int mine = lane / kSpread, col0 = NC * wg;    // this lane's column of the warpgroup's
    const uint32_t mx = base + S::MAX + warp * NC * 4, fac = base + S::FAC + warp * NC * 4, xch = base + S::XCH + wg * 4 * NC * 4;
    const uint32_t prow = base + S::P + key * (2 * N);
    const uint32_t swz = N == 64 ? key & 7 : N == 32 ? (key >> 1) & 3 : (key >> 2) & 1;
    const float sl2 = args.scale_log2;
    uint32_t exchanges = 0, piece = 0;
    float l[NC];
    bool ok = true;
    I4Tile a;
    // the four warps' values of this lane's column, once all have written theirs (maxima and sums each in a place of their own:
    // between two exchanges of a kind every warp has come past the flags, so that none still reads the one before)
    auto exchange = [&](uint32_t at, float v) -> bool {
      if (lane % kSpread == 0) sts32f(at + (w * NC + mine) * 4, v);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(IB_XCH + wg));
      return i4_wait_warp(bar(IB_XCH + wg), exchanges++ & 1, wc, kSiteI4Flag);
    };
    for (uint32_t t = 0; ok && cur.next(a); ++t) {
      if (a.first) {
#pragma unroll
        for (int c = 0; c < NC; ++c) l[c] = 0.f;
        if (lane < NC) sts32f(mx + 4 * lane, -3.402823466e38f);  // (finite: a first score against it is no NaN)
        __syncwarp();
      }
      if (!(ok = i4_wait_warp(bar(IB_S_FULL + (t & 1)), (t >> 1) & 1, wc, kSiteI4Scores))) break;
      tc_fence_after();
      const int some = a.vis - (args.causal ? args.group - 1 : 0) - a.key0;
      const bool masked = some < kI4Tile || a.nkeys < kI4Tile;
      int hidden = 0;  // rows [0, hidden) of the warpgroup's columns do not see this key
      bool bad = false;
      if (masked) {
        hidden = (key >= a.nkeys ? 1 << 20 : args.causal ? max(key - some + 1, 0) * args.H : 0) - row0 - col0;
        uint8_t* poison = smem + S::POISON + 256 * (t & 1) + 128 * wg + key;
        bad = *poison != 0;
        if (bad) *poison = 0;
      }
      // kC columns of scores from column c on
      auto load_scores = [&](int c, float (&v)[kC]) {
        uint32_t u[kC];
        tmem_ld_cols(tmem + lanes + TS + N * (t & 1) + col0 + c, u);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kC; ++k) v[k] = __uint_as_float(u[k]);
        if (masked)
#pragma unroll
          for (int k = 0; k < kC; ++k) v[k] = c + k < hidden ? -INFINITY : bad ? __uint_as_float(0x7FC00000u) : v[k];
      };
      const uint64_t s2 = splat_f32x2(sl2);
      auto scores = [&](int c, float (&v)[kC]) {  // against the maxima, in log2 units
        load_scores(c, v);
#pragma unroll
        for (int q = 0; q < kC / 4; ++q) {
          float m4[4];
          lds128f(mx + 4 * c + 16 * q, m4[0], m4[1], m4[2], m4[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            unpack_f32x2(ffma_f32x2(pack_f32x2(v[4 * q + 2 * h], v[4 * q + 2 * h + 1]), s2, pack_f32x2(-m4[2 * h], -m4[2 * h + 1])),
                         v[4 * q + 2 * h], v[4 * q + 2 * h + 1]);
        }
      };
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < NC; c += kC) {
        float d[kC];
        scores(c, d);
#pragma unroll
        for (int k = 0; k < kC; k += 2) top = fmax3(top, d[k], d[k + 1]);
      }
      const bool over = __any_sync(0xffffffffu, top > 8.f);
      if (lane == 0) {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + S::FLAG + 32 * (t & 1) + 4 * warp), "r"(over ? 1u : 0u) : "memory");
        mbar_arrive(bar(IB_FLAG + 2 * wg + (t & 1)));
      }
      __syncwarp();
      if (!(ok = i4_wait_warp(bar(IB_FLAG + 2 * wg + (t & 1)), (t >> 1) & 1, wc, kSiteI4Flag))) break;
      float f4[4];
      lds128f(base + S::FLAG + 32 * (t & 1) + 16 * wg, f4[0], f4[1], f4[2], f4[3]);
      const bool raise = (__float_as_uint(f4[0]) | __float_as_uint(f4[1]) | __float_as_uint(f4[2]) | __float_as_uint(f4[3])) != 0;
      if (raise) {
        float wm;
        {
          float v[NC];
#pragma unroll
          for (int c = 0; c < NC; c += kC) {
            float u[kC];
            load_scores(c, u);
#pragma unroll
            for (int k = 0; k < kC; ++k) v[c + k] = u[k] * sl2;
          }
          wm = reduce_columns<NC>(v, lane, [](float x, float y) { return fmaxf(x, y); });
        }
        if (!(ok = exchange(xch, wm))) break;
        float cm = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) cm = fmaxf(cm, lds32f(xch + (k * NC + mine) * 4));
        const float old = lds32f(mx + 4 * mine);
        const bool grow = cm > old + 8.f;
        __syncwarp();
        if (lane % kSpread == 0) {
          sts32f(mx + 4 * mine, grow ? cm : old);
          sts32f(fac + 4 * mine, grow ? ex2_approx(old - cm) : 1.f);
        }
        __syncwarp();
        if (!a.first) {  // the output so far (the tile before has been added to it before this one's scores were done)
#pragma unroll
          for (int c = 0; c < NC; c += kC) {
            float f[kC];
#pragma unroll
            for (int q = 0; q < kC / 4; ++q) lds128f(fac + 4 * c + 16 * q, f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
#pragma unroll
            for (int k = 0; k < kC; ++k) l[c + k] *= f[k];
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              uint32_t o[kC];
              tmem_ld_cols(tmem + lanes + TO + N * m + col0 + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < kC; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f[k]);
              tmem_st_cols(tmem + lanes + TO + N * m + col0 + c, o);
            }
          }
          tmem_wait_st();
        }
      }
      // (P is free: the output product of the tile before came before this tile's scores)
#pragma unroll
      for (int c = 0; c < NC; c += kC) {
        float d[kC];
        scores(c, d);
        uint32_t pp[kC / 2];
#pragma unroll
        for (int k = 0; k < kC; k += 2) {
          const float p0 = ex2_approx(d[k]), p1 = ex2_approx(d[k + 1]);
          // P in bf16, the type of the values in the tensor cores (half a step is 2^-8 of a weight at most, of either sign); the
          // row's sum takes the float32 weights, so that lse is not rounded with them
          pp[k / 2] = pack_bf16(p0, p1);
          l[c + k] += p0;
          l[c + k + 1] += p1;
        }
#pragma unroll
        for (int q = 0; q < kC / 8; ++q)
          sts128(prow + (((uint32_t)((col0 + c) / 8 + q) ^ swz) << 4), pp[4 * q], pp[4 * q + 1], pp[4 * q + 2], pp[4 * q + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(IB_P_FULL));
      if (!a.last) continue;

      // O / l of the finished piece -> its rows of out, or a split partial
      const float wl = reduce_columns<NC>(l, lane, [](float x, float y) { return x + y; });
      if (!(ok = exchange(xch + 8 * NC * 4, wl))) break;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum += lds32f(xch + 8 * NC * 4 + (k * NC + mine) * 4);
      const float m_run = lds32f(mx + 4 * mine);
      const bool none = sum == 0.f;  // the row saw no key
      const int r = col0 + mine, rr = row0 + r;  // row of the part, of the block
      const bool on = r < args.part_rows && rr < block_rows;
      const int32_t* num_splits = sched + kSchedHeader + kUnitInts * args.num_units;
      const int ns = num_splits[a.wb * args.group];
      const bool split = ns > 1;
      int64_t row = (int64_t)a.wb * block_rows + rr;
      if (split) {
        const int g = rr / args.H;
        row = ((int64_t)num_splits[args.num_qb + a.wb * args.group] + g * ns + a.split) * args.H + (rr - g * args.H);
      }
      if (lane % kSpread == 0) {
        sts32f(fac + 4 * mine, none ? 0.f : 1.f / sum);
        if (on && w == 0) {
          const float lse = none ? -INFINITY : (m_run + log2f(sum)) * 0.69314718055994530942f;
          if (split) args.lse_acc[row] = lse; else args.lse[row] = lse;
        }
      }
      if (!on) row = -1;
      __syncwarp();
      if (!(ok = i4_wait_warp(bar(IB_PV), piece++ & 1, wc, kSiteI4Pv))) break;
      tc_fence_after();
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        const int dim = 128 * m + 32 * w + lane;
#pragma unroll
        for (int c = 0; c < NC; c += kC) {
          uint32_t o[kC];
          tmem_ld_cols(tmem + lanes + TO + N * m + col0 + c, o);
          tmem_wait_ld();
          float f[kC];
#pragma unroll
          for (int q = 0; q < kC / 4; ++q) lds128f(fac + 4 * c + 16 * q, f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
#pragma unroll
          for (int k = 0; k < kC; k += 2) {
            const float x0 = f[k] == 0.f ? 0.f : __uint_as_float(o[k]) * f[k], x1 = f[k + 1] == 0.f ? 0.f : __uint_as_float(o[k + 1]) * f[k + 1];
            const int64_t r0 = __shfl_sync(0xffffffffu, row, (c + k) * kSpread), r1 = __shfl_sync(0xffffffffu, row, (c + k + 1) * kSpread);
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
    }
    tc_fence_before();
  }

  __syncwarp();
  __syncthreads();
  if (*abort_flag) drain_delay(200000);  // in-flight copies and MMAs land before release
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

__global__ void __launch_bounds__(kI4Threads, 1) mla_decode_int4_n16_kernel(const __grid_constant__ Int4Args args) {
  decode_int4_body<16>(args);
}
__global__ void __launch_bounds__(kI4Threads, 1) mla_decode_int4_n32_kernel(const __grid_constant__ Int4Args args) {
  decode_int4_body<32>(args);
}
__global__ void __launch_bounds__(kI4Threads, 1) mla_decode_int4_n64_kernel(const __grid_constant__ Int4Args args) {
  decode_int4_body<64>(args);
}

}  // namespace mla
