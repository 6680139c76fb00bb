// The paged cache's own upkeep: new tokens' rows written through the block table, and pages
// copied, shared, taken, given back and drawn together.  All of it is memory-bound: rows and pages
// are moved once, in 16-byte accesses, and the bookkeeping -- reference counts, block table,
// lengths -- is kept on the device, so that a serving step needs no host synchronisation.
//
// ref_counts[page] is the number of block-table entries that hold the page; 0 = free.  Pages are
// always taken lowest first and in the order of the caller's list, so every result is determined
// by the inputs (the atomics are integer additions).
//
// Measured: compaction of 226 pages x 16 layers, 533 MB read and written, in 78 us (6.8 TB/s, 102% of
// the measured copy rate); 300 pages x 8 layers, 202 MB, copied in 27-32 us; the kernels
// that only keep books take 4-8 us cold, 2-5 in a run of calls.
#pragma once
#include "chunk_kernel.cuh"  // block_scan_1024
#include "common.cuh"

namespace mla {

constexpr int kPageRows = 64;
// What reserve writes for a sequence.
constexpr int kReserveDone = 1, kReserveNoPages = 0, kReserveRefused = -2;

struct PoolArgs {
  int32_t batch, num_pages, max_pages, num_layers, row_bytes;
  int64_t layer_stride;  // bytes
};

__device__ __forceinline__ void pool_error(int code) { atomicCAS(&g_mla_error, 0, code); }
__device__ __forceinline__ int pages_held(int L) { return (L + kPageRows - 1) / kPageRows; }

// ----------------------------------------------------------------- row quantiser
// 16 latent values of a lane (8 lanes a 128-value tile) -> the tile's scale and 16 E4M3 codes by
// the cache rule: scale = amax / 448 (1 for an all-zero tile), code = E4M3(x / scale), RNE.
// kKeepNan: a quotient that is NaN gives a NaN code (else it is clamped like any other).
// The quotient is q = x r, r = 1 / scale, corrected once by its remainder: q + (x - q scale) r (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).  x and amax
// have 8 significant bits, so all 128 x 128 pairs of significands can be gone through: every corrected quotient
// is the correctly rounded one (tests/test_quotients.py).  The exponents play no part while
// nothing under- or overflows; a scale outside (2^-60, 2^100) is divided by.  Inside, what underflows
// belongs to quotients far below the least code.  (-0 would come out as +0: the sign is put back.)
template <bool kKeepNan>
__device__ __forceinline__ void quantize_tile16(const float (&x)[16], uint32_t (&codes)[4], float& scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  scale = amax > 0.f ? amax / 448.f : 1.f;
  float z[16];
  if (__all_sync(0xffffffffu, scale > 0x1p-60f && scale < 0x1p100f)) {
    const float r = 1.f / scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q = x[i] * r;
      z[i] = copysignf(fmaf(fmaf(-q, scale, x[i]), r, q), x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = x[i] / scale;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!kKeepNan)
#pragma unroll
      for (int k = 4 * i; k < 4 * i + 4; ++k) z[k] = fminf(fmaxf(z[k], -448.f), 448.f);
    // (the conversion saturates by itself, and keeps NaN)
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(z[4 * i], z[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z[4 * i + 2], z[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    codes[i] = lo | (hi << 16);
  }
}
__device__ __forceinline__ void widen16(const uint4& a, const uint4& b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// ----------------------------------------------------------------- append
// Token t of the ragged buffer belongs to the sequence b with cu[b] <= t < cu[b + 1] and goes to
// row L_b - n_b + (t - cu[b]) of that sequence.  A warp takes a token: its row is loaded first,
// then the sequence is found by a 32-way search (one round for up to 31 sequences, two for up to
// ~1000).  kServed: the tokens of a sequence that did not get its pages go nowhere -- its length is
// still the old one, and row L_b - n_b one that it (or, in a shared page, another) holds; a kernel of
// its own, since as a question at run time it cost the other 7%.  From a graph 64 rows in 1.9-2.2 us;
// 22,500 rows quantised in 10.2-10.6 us, 3.9 TB/s (11.4 us with the divisions; 11.0-11.3 cold), as bf16 in 9.5 us,
// 5.5 TB/s: the search and the launch are the rest.
template <bool kFp8, bool kServed>
__global__ void __launch_bounds__(256) mla_append_kernel(PoolArgs p, int64_t max_tokens, const __nv_bfloat16* latent,
                                                         int64_t latent_stride, const __nv_bfloat16* rope,
                                                         int64_t rope_stride, const int32_t* cu, const int32_t* lens,
                                                         const int32_t* block_table, const int32_t* served, uint8_t* pages) {
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (t >= max_tokens) return;
  const uint4* src = reinterpret_cast<const uint4*>(latent + t * latent_stride);
  const uint4 a = src[kFp8 ? 2 * lane : lane], b = src[kFp8 ? 2 * lane + 1 : lane + 32];
  uint4 kr = make_uint4(0, 0, 0, 0);
  if (lane < 8) kr = *reinterpret_cast<const uint4*>(rope + t * rope_stride + 8 * lane);
  const int32_t end = cu[p.batch];
  int lo = 0, hi = p.batch;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 31) {
    const int step = (hi - lo + 31) >> 5, at = lo + step * lane;
    const uint32_t le = __ballot_sync(0xffffffffu, at < hi && cu[at] <= t);
    const int k = le ? 31 - __clz(le) : 0;
    hi = min(hi, lo + step * (k + 1));
    lo = lo + step * k;
  }
  // the last round: lane j holds cu[lo + j], the length of sequence lo + j and whether it takes its tokens
  const int32_t start = lo + lane <= p.batch ? cu[lo + lane] : INT32_MAX;
  const int32_t len = lo + lane < p.batch ? lens[lo + lane] : 0;
  const bool takes = kServed && lo + lane < p.batch && served[lo + lane] == kReserveDone;
  if (t >= end) return;  // rows behind the last sequence
  const uint32_t le = __ballot_sync(0xffffffffu, lo + lane < hi && start <= t);
  const int k = le ? 31 - __clz(le) : 0;  // (at most 30: the next sequence's start is a lane's too)
  if (kServed && !((__ballot_sync(0xffffffffu, takes) >> k) & 1)) return;
  lo += k;
  const int first = __shfl_sync(0xffffffffu, start, k), n = __shfl_sync(0xffffffffu, start, k + 1) - first;
  const int64_t pos = (int64_t)__shfl_sync(0xffffffffu, len, k) - n + (t - first);
  if (n < 0 || t < first || pos < 0 || pos >= (int64_t)p.max_pages * kPageRows) {
    if (lane == 0) pool_error(1);
    return;
  }
  const int page = block_table[(int64_t)lo * p.max_pages + pos / kPageRows];
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) pool_error(1);
    return;
  }
  uint8_t* dst = pages + ((int64_t)page * kPageRows + pos % kPageRows) * p.row_bytes;
  if (kFp8) {
    float x[16], scale;
    uint32_t c[4];
    widen16(a, b, x);
    quantize_tile16<true>(x, c, scale);
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(c[0], c[1], c[2], c[3]);
    if ((lane & 7) == 0) *reinterpret_cast<float*>(dst + 512 + 4 * (lane >> 3)) = scale;
    if (lane < 8) *reinterpret_cast<uint4*>(dst + 528 + 16 * lane) = kr;
  } else {
    uint4* d = reinterpret_cast<uint4*>(dst);
    d[lane] = a;
    d[lane + 32] = b;
    if (lane < 8) d[64 + lane] = kr;
  }
}

// ----------------------------------------------------------------- moving bytes
// n 16-byte words by the block's threads, up to kDeep loads in flight each.
template <int kDeep>
__device__ __forceinline__ void copy_words(uint4* dst, const uint4* src, int n) {
  for (int i = threadIdx.x; i < n; i += kDeep * blockDim.x) {
    uint4 v[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if (i + k * (int)blockDim.x < n) v[k] = __ldcs(src + i + k * blockDim.x);
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if (i + k * (int)blockDim.x < n) __stcs(dst + i + k * blockDim.x, v[k]);
  }
}

constexpr int kCopyParts = 4;  // a page is copied by this many blocks, a quarter of its rows each

// grid (pairs, layers * kCopyParts)
__global__ void __launch_bounds__(256) mla_copy_pages_kernel(PoolArgs p, uint8_t* pages, const int32_t* src,
                                                             const int32_t* dst) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int from = src[blockIdx.x], to = dst[blockIdx.x];
  if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
    if (threadIdx.x == 0) pool_error(1);
    return;
  }
  if (from == to) return;
  const int layer = blockIdx.y / kCopyParts, part = blockIdx.y % kCopyParts, words = (kPageRows / kCopyParts) * p.row_bytes / 16;
  uint8_t* pool = pages + (int64_t)layer * p.layer_stride;
  const int64_t page_bytes = (int64_t)kPageRows * p.row_bytes;
  copy_words<5>(reinterpret_cast<uint4*>(pool + to * page_bytes) + part * words,
                reinterpret_cast<const uint4*>(pool + from * page_bytes) + part * words, words);
}

// ----------------------------------------------------------------- free pages, lowest first
// Calls take(rank, page) for the free pages of rank < want, in order of their number; returns how
// many there were (at most want).  All 1024 threads of the one CTA.  4096 pages a round.
template <class F>
__device__ __forceinline__ int64_t scan_free_pages(const int32_t* ref, int num_pages, int64_t want, int64_t* sh, F take) {
  int64_t found = 0;
  for (int64_t p0 = 0; p0 < num_pages && found < want; p0 += 4096) {
    const int64_t q = p0 + 4 * threadIdx.x;
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = 1;
    if (q + 3 < num_pages) {
      const int4 x = *reinterpret_cast<const int4*>(ref + q);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (q + k < num_pages) v[k] = ref[q + k];
    }
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) n += v[k] == 0;
    int64_t sum, rank = found + block_scan_1024(n, sh, &sum);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v[k] == 0) {
        if (rank < want) take(rank, (int)(q + k));
        ++rank;
      }
    found += sum;
  }
  return found < want ? found : want;
}

// ----------------------------------------------------------------- fork
// Outcomes in new_pages: a page, or one of these.
constexpr int kForkShared = -1;   // done; no page was needed (the parent ends on a page boundary)
constexpr int kForkRefused = -2;  // a row out of range, a child that is not empty or is named twice
constexpr int kForkNoPage = -3;   // no free page left; the child stays empty

// One CTA: checks the forks, gives each its page, sets the children's lengths.  ws: per fork the
// parent's length, then per table row the first fork that names it as child.
__global__ void __launch_bounds__(1024) mla_fork_plan_kernel(PoolArgs p, const int32_t* parents, const int32_t* children, int n,
                                                             int32_t* seqlens, int32_t* ref, int32_t* new_pages, int32_t* ws) {
  __shared__ int64_t sh[32];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  int32_t *len = ws, *claim = ws + n;
  for (int i = tid; i < p.batch; i += 1024) claim[i] = INT32_MAX;
  __syncthreads();
  for (int i = tid; i < n; i += 1024) {
    const int a = parents[i], c = children[i];
    int L = -1;
    if (a >= 0 && a < p.batch && c >= 0 && c < p.batch && seqlens[c] == 0) {
      L = seqlens[a];
      if (L < 0 || (int64_t)L > (int64_t)p.max_pages * kPageRows) L = -1;
    }
    len[i] = L;
    if (L >= 0) atomicMin(&claim[c], i);
  }
  __syncthreads();
  int64_t need = 0;
  for (int i0 = 0; i0 < n; i0 += 1024) {  // rank of each fork that needs a page, kept in new_pages for now
    const int i = i0 + tid;
    bool ok = false, part = false;
    if (i < n) {
      ok = len[i] >= 0 && claim[children[i]] == i;
      part = ok && len[i] % kPageRows != 0;
    }
    int64_t sum;
    const int64_t e = block_scan_1024(part, sh, &sum);
    if (i < n) {
      if (!ok) {
        pool_error(1);
        len[i] = -1;
      }
      new_pages[i] = part ? (int32_t)(need + e) : ok ? kForkShared : kForkRefused;
    }
    need += sum;
  }
  __syncthreads();
  int32_t* page_of_rank = claim + p.batch;
  const int64_t found = scan_free_pages(ref, p.num_pages, need, sh, [&](int64_t rank, int page) {
    page_of_rank[rank] = page;
  });
  __syncthreads();
  for (int i = tid; i < n; i += 1024) {
    const int rank = new_pages[i];
    if (rank >= 0) {
      if (rank < found) {
        const int page = page_of_rank[rank];
        new_pages[i] = page;
        ref[page] = 1;
      } else {
        new_pages[i] = kForkNoPage;
        len[i] = -1;
      }
    }
    if (len[i] >= 0) seqlens[children[i]] = len[i];
  }
}

// grid (forks, 1 + layers): y = 0 writes the child's table row and counts the shared pages, y > 0
// copies the rows of the parent's last, partly filled page in layer y - 1.
__global__ void __launch_bounds__(256) mla_fork_kernel(PoolArgs p, uint8_t* pages, const int32_t* parents,
                                                       const int32_t* children, int32_t* block_table, int32_t* ref,
                                                       const int32_t* new_pages, const int32_t* ws) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int i = blockIdx.x, L = ws[i];
  if (L < 0) return;
  const int full = L / kPageRows, rows = L % kPageRows, fresh = new_pages[i];
  const int32_t* from = block_table + (int64_t)parents[i] * p.max_pages;
  if (blockIdx.y == 0) {
    int32_t* to = block_table + (int64_t)children[i] * p.max_pages;
    for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x) {
      int page = -1;
      if (j < full) {
        page = from[j];
        if (page >= 0 && page < p.num_pages)
          atomicAdd(&ref[page], 1);
        else
          pool_error(1);
      } else if (j == full && rows > 0) {
        page = fresh;
      }
      to[j] = page;
    }
    return;
  }
  if (rows == 0) return;
  const int src = from[full];
  if (src < 0 || src >= p.num_pages) {
    if (threadIdx.x == 0) pool_error(1);
    return;
  }
  uint8_t* pool = pages + (int64_t)(blockIdx.y - 1) * p.layer_stride;
  const int64_t page_bytes = (int64_t)kPageRows * p.row_bytes;
  copy_words<4>(reinterpret_cast<uint4*>(pool + fresh * page_bytes), reinterpret_cast<const uint4*>(pool + src * page_bytes),
                rows * p.row_bytes / 16);
}

// ----------------------------------------------------------------- reserve
// One CTA.  Sequence b needs pages for num_new[b] more rows.  Those served are the sequences up to
// the first whose pages are no longer there, and all that need none.  ws: pages needed by the
// sequences before b [batch + 1].
__global__ void __launch_bounds__(1024) mla_reserve_kernel(PoolArgs p, const int32_t* num_new, int32_t* block_table,
                                                           int32_t* seqlens, int32_t* ref, int32_t* served, int32_t* ws) {
  __shared__ int64_t sh[32];
  __shared__ int limit_sh;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  int64_t need = 0;
  if (tid == 0) limit_sh = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 1024) {
    const int b = b0 + tid;
    int k = 0;
    if (b < p.batch) {
      const int64_t L = seqlens[b], n = num_new[b];
      const bool ok = L >= 0 && n >= 0 && L + n <= (int64_t)p.max_pages * kPageRows;
      if (ok)
        k = pages_held((int)(L + n)) - pages_held((int)L);
      else
        pool_error(1);
      served[b] = ok ? kReserveDone : kReserveRefused;
    }
    int64_t sum;
    const int64_t e = block_scan_1024(k, sh, &sum);
    if (b < p.batch) ws[b] = (int32_t)min(need + e, (int64_t)INT32_MAX);
    need += sum;
  }
  if (tid == 0) ws[p.batch] = (int32_t)min(need, (int64_t)INT32_MAX);
  __syncthreads();
  const int64_t free_pages = scan_free_pages(ref, p.num_pages, need, sh, [](int64_t, int) {});
  for (int b = tid; b < p.batch; b += 1024)  // the pages of the last sequence that is served in full end at the limit
    if (ws[b + 1] <= free_pages) atomicMax(&limit_sh, ws[b + 1]);
  __syncthreads();
  const int limit = limit_sh;
  scan_free_pages(ref, p.num_pages, limit, sh, [&](int64_t rank, int page) {
    const int b = chunk_find(ws, p.batch, (int32_t)rank);  // the last sequence that starts at or before this rank
    block_table[(int64_t)b * p.max_pages + pages_held(seqlens[b]) + (int)(rank - ws[b])] = page;
    ref[page] = 1;
  });
  __syncthreads();  // (the lengths are read above)
  for (int b = tid; b < p.batch; b += 1024) {
    if (served[b] == kReserveRefused) continue;
    if (ws[b + 1] > limit && ws[b + 1] > ws[b])
      served[b] = kReserveNoPages;
    else
      seqlens[b] += num_new[b];
  }
}

// ----------------------------------------------------------------- free
// grid: one block per listed sequence; the block that swaps the length for 0 owns the row, so a
// sequence listed twice is freed once.
__global__ void __launch_bounds__(128) mla_free_kernel(PoolArgs p, const int32_t* ids, int32_t* block_table, int32_t* seqlens,
                                                       int32_t* ref) {
  __shared__ int len_sh;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int b = ids[blockIdx.x];
  if (b < 0 || b >= p.batch) {
    if (threadIdx.x == 0) pool_error(1);
    return;
  }
  if (threadIdx.x == 0) {
    const int L = seqlens[b];
    const bool ok = L >= 0 && (int64_t)L <= (int64_t)p.max_pages * kPageRows;
    if (!ok) pool_error(1);
    len_sh = ok ? atomicExch(&seqlens[b], 0) : 0;
  }
  __syncthreads();
  const int L = len_sh;
  int32_t* row = block_table + (int64_t)b * p.max_pages;
  for (int j = threadIdx.x; j < pages_held(L); j += blockDim.x) {
    const int page = row[j];
    row[j] = -1;
    if (page < 0 || page >= p.num_pages)
      pool_error(1);
    else if (atomicSub(&ref[page], 1) <= 0) {  // nobody held it: the counts do not belong to the table
      atomicAdd(&ref[page], 1);
      pool_error(1);
    }
  }
}

// ----------------------------------------------------------------- compact
// One CTA: the used pages at or above their count, in order, are paired with the free pages below
// it, in order.  ws: [0] moves, then map [num_pages], from and to [num_pages / 2 + 1] each.
__global__ void __launch_bounds__(1024) mla_compact_plan_kernel(PoolArgs p, int32_t* ref, int32_t* num_used, int32_t* ws) {
  __shared__ int64_t sh[32];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int tid = threadIdx.x, P = p.num_pages;
  int32_t *map = ws + 4, *from = map + P, *to = from + P / 2 + 1;
  int mine = 0;
  for (int q = tid; q < P; q += 1024) mine += ref[q] != 0;
  int64_t used, moves = 0, holes = 0;
  block_scan_1024(mine, sh, &used);
  for (int q0 = 0; q0 < P; q0 += 1024) {
    const int q = q0 + tid;
    const bool held = q < P && ref[q] != 0, src = held && q >= used, dst = q < P && !held && q < used;
    int64_t sum;
    const int64_t a = block_scan_1024((int64_t)src | ((int64_t)dst << 32), sh, &sum);
    if (src) from[moves + (a & 0xffffffff)] = q;
    if (dst) to[holes + (a >> 32)] = q;
    if (q < P) map[q] = q;
    moves += sum & 0xffffffff;
    holes += sum >> 32;
  }
  __syncthreads();
  for (int k = tid; k < moves; k += 1024) {
    map[from[k]] = to[k];
    ref[to[k]] = ref[from[k]];
    ref[from[k]] = 0;
  }
  if (tid == 0) {
    ws[0] = (int32_t)moves;
    *num_used = (int32_t)used;
  }
}

// Blocks stride over (move, layer, quarter page), then over the table's rows.
__global__ void __launch_bounds__(256) mla_compact_kernel(PoolArgs p, uint8_t* pages, int32_t* block_table,
                                                          const int32_t* seqlens, const int32_t* ws) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int P = p.num_pages, moves = ws[0];
  const int32_t *map = ws + 4, *from = map + P, *to = from + P / 2 + 1;
  const int words = (kPageRows / kCopyParts) * p.row_bytes / 16;
  const int64_t page_bytes = (int64_t)kPageRows * p.row_bytes, items = (int64_t)moves * p.num_layers * kCopyParts;
  for (int64_t it = blockIdx.x; it < items + p.batch; it += gridDim.x) {
    if (it >= items) {
      const int b = (int)(it - items), L = seqlens[b];
      if (L < 0 || (int64_t)L > (int64_t)p.max_pages * kPageRows) {
        if (threadIdx.x == 0) pool_error(1);
        continue;
      }
      int32_t* row = block_table + (int64_t)b * p.max_pages;
      for (int j = threadIdx.x; j < pages_held(L); j += blockDim.x) {
        const int page = row[j];
        if (page < 0 || page >= P)
          pool_error(1);
        else
          row[j] = map[page];
      }
      continue;
    }
    const int part = (int)(it % kCopyParts), layer = (int)(it / kCopyParts % p.num_layers), k = (int)(it / kCopyParts / p.num_layers);
    uint8_t* pool = pages + (int64_t)layer * p.layer_stride;
    copy_words<5>(reinterpret_cast<uint4*>(pool + to[k] * page_bytes) + part * words,
                  reinterpret_cast<const uint4*>(pool + from[k] * page_bytes) + part * words, words);
  }
}

}  // namespace mla
