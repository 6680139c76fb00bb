// Host side of the chunk attention and of the paged cache's upkeep (argument checks, tensor maps,
// launches).  Part of mla_decode.cu: it uses that file's device table and map encoder.
#pragma once
#include <initializer_list>
#include <new>

namespace {

// Launch on `stream` as a programmatic dependent of the kernel before it (every kernel here waits
// for that one before it touches global memory).
template <class... P, class... A>
int32_t launch_after(void* stream, dim3 grid, int threads, size_t smem, void (*kernel)(P...), A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  pdl_config(&cfg, attr, stream);
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

// Bytes of a cached token, 0 for what is no mla_kv_dtype.
int kv_row_bytes(int32_t kv_dtype) {
  return kv_dtype == MLA_KV_BF16 ? 1152 : kv_dtype == MLA_KV_FP8_E4M3 ? 656 : kv_dtype == MLA_KV_INT4 ? kI4Row : 0;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ------------------------------------------------------------------ chunk attention
int32_t check_chunk(const mla_chunk_params* p) {
  if (!p) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->max_tokens < 1 || p->num_heads < 1 || p->num_pages < 1 || p->page_size < 1 ||
      p->max_pages_per_seq < 1 || p->num_units < 0 || p->timeout_us < 0 || p->max_kv_tokens < 0)
    return MLA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (p->reserved[i] != 0) return MLA_ERR_INVALID_ARG;
  if (kv_row_bytes(p->kv_dtype) == 0) return MLA_ERR_INVALID_ARG;
  if (p->kv_dtype != MLA_KV_BF16 && p->max_kv_tokens < 64) return MLA_ERR_INVALID_ARG;
  if (p->page_size != 64 || p->num_heads > 128) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->max_tokens * p->num_heads > INT32_MAX - 256 || (int64_t)p->num_pages * 64 > INT32_MAX ||
      p->max_kv_tokens > INT32_MAX - 64 || (int64_t)p->max_pages_per_seq * 64 > INT32_MAX - kChunkTile ||
      p->batch > (1 << 24) || p->num_units > 65535)
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

int32_t chunk_units(const mla_chunk_params* p, int32_t* U) {
  if (p->num_units > 0) {
    *U = p->num_units;
    return MLA_OK;
  }
  DeviceInfo* d = nullptr;
  const int32_t st = device_info(&d);
  if (st != MLA_OK) return st;
  *U = d->max_clusters[1];
  return MLA_OK;
}

struct ChunkBuffers {
  int64_t cap;
  size_t sched, o_acc, lse_acc, rows, workspace;  // bytes
};

// Partial slots: a unit boundary lies in at most one block, and a block split over k units (k - 1
// boundaries) takes k slots, so U units make at most 2 (U - 1).
ChunkBuffers chunk_buffers(const mla_chunk_params* p, int32_t U) {
  ChunkBuffers b;
  b.cap = chunk_block_capacity(p->max_tokens, p->batch, p->num_heads);
  b.sched = sizeof(int32_t) * (size_t)chunk_layout(U, b.cap, p->batch).total;
  b.o_acc = (size_t)2 * U * kChunkRows * 512 * sizeof(float);
  b.lse_acc = (size_t)2 * U * kChunkRows * sizeof(float);
  b.rows = p->kv_dtype != MLA_KV_BF16 ? (size_t)(p->max_kv_tokens / 64) * 64 * 1152 : 0;
  b.workspace = b.o_acc + align256(b.lse_acc) + b.rows;
  return b;
}

int64_t chunk_kv_pages(const mla_chunk_params* p) {  // pages a plan may name in all
  return p->kv_dtype != MLA_KV_BF16 ? p->max_kv_tokens / 64 : INT32_MAX;
}

// ------------------------------------------------------------------ page pool
int32_t check_pool(const mla_pool_params* p) {
  if (!p) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->num_pages < 1 || p->page_size < 1 || p->max_pages_per_seq < 1 || p->num_layers < 1 ||
      p->layer_stride < 0)
    return MLA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (p->reserved[i] != 0) return MLA_ERR_INVALID_ARG;
  if (kv_row_bytes(p->kv_dtype) == 0) return MLA_ERR_INVALID_ARG;
  const int64_t packed = (int64_t)p->num_pages * 64 * kv_row_bytes(p->kv_dtype);
  if (p->layer_stride != 0 && (p->layer_stride < packed || p->layer_stride % 16 != 0)) return MLA_ERR_INVALID_ARG;
  if (p->page_size != 64) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->num_pages * 64 > INT32_MAX || (int64_t)p->max_pages_per_seq * 64 > INT32_MAX || p->batch > (1 << 24) ||
      p->num_layers > 16383)
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

PoolArgs pool_args(const mla_pool_params* p) {
  PoolArgs a;
  a.batch = p->batch;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages_per_seq;
  a.num_layers = p->num_layers;
  a.row_bytes = kv_row_bytes(p->kv_dtype);
  a.layer_stride = p->layer_stride ? p->layer_stride : (int64_t)p->num_pages * 64 * a.row_bytes;
  return a;
}

bool all_int_arrays(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return false;
  return true;
}

int32_t append_kv(const mla_pool_params* p, int64_t max_tokens, const void* latent, int64_t latent_stride,
                  const void* k_rope, int64_t rope_stride, const int32_t* cu_seqlens, const int32_t* cache_seqlens,
                  const int32_t* block_table, const int32_t* served, void* kv_pages, void* stream) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (max_tokens < 0 || !latent || !k_rope || !cu_seqlens || !cache_seqlens || !block_table || !kv_pages)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(latent) || !aligned16(k_rope) || !aligned16(kv_pages) || !aligned(cu_seqlens, 4) ||
      !aligned(cache_seqlens, 4) || !aligned(block_table, 4))
    return MLA_ERR_INVALID_ARG;
  if (latent_stride < 512 || latent_stride % 8 != 0 || rope_stride < 64 || rope_stride % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (max_tokens > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  if (max_tokens == 0) return MLA_OK;
  const dim3 grid((unsigned)((max_tokens + 7) / 8));
  const __nv_bfloat16 *c = static_cast<const __nv_bfloat16*>(latent), *r = static_cast<const __nv_bfloat16*>(k_rope);
  auto* kernel = p->kv_dtype == MLA_KV_INT4       ? (served ? mla_append_kernel<kKvInt4, true> : mla_append_kernel<kKvInt4, false>)
                 : p->kv_dtype == MLA_KV_FP8_E4M3 ? (served ? mla_append_kernel<kKvFp8, true> : mla_append_kernel<kKvFp8, false>)
                                                  : (served ? mla_append_kernel<kKvBf16, true> : mla_append_kernel<kKvBf16, false>);
  return launch_after(stream, grid, 256, 0, kernel, pool_args(p), max_tokens, c, latent_stride, r, rope_stride, cu_seqlens,
                      cache_seqlens, block_table, served, static_cast<uint8_t*>(kv_pages));
}

}  // namespace

extern "C" {

int32_t mla_chunk_workspace_size(const mla_chunk_params* p, size_t* sched_bytes, size_t* workspace_bytes) {
  int32_t st = check_chunk(p);
  if (st != MLA_OK) return st;
  if (!sched_bytes || !workspace_bytes) return MLA_ERR_INVALID_ARG;
  int32_t U = 0;
  if ((st = chunk_units(p, &U)) != MLA_OK) return st;
  const ChunkBuffers b = chunk_buffers(p, U);
  *sched_bytes = b.sched;
  *workspace_bytes = b.workspace;
  return MLA_OK;
}

int32_t mla_chunk_plan_host(const mla_chunk_params* p, int32_t num_units, const int32_t* cu_seqlens,
                            const int32_t* cache_seqlens, void* sched) {
  int32_t st = check_chunk(p);
  if (st != MLA_OK) return st;
  if (num_units < 1 || num_units > 65535 || !cu_seqlens || !cache_seqlens || !sched) return MLA_ERR_INVALID_ARG;
  try {
    return chunk_plan_host(cu_seqlens, cache_seqlens, p->batch, p->max_tokens, p->num_heads, p->causal != 0,
                           p->max_pages_per_seq, chunk_kv_pages(p), num_units, static_cast<int32_t*>(sched))
               ? MLA_OK
               : MLA_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {  // no room to deal the blocks in
    return MLA_ERR_WORKSPACE;
  }
}

int32_t mla_chunk_schedule(const mla_chunk_params* p, const int32_t* cu_seqlens, const int32_t* cache_seqlens, void* sched,
                           void* stream) {
  int32_t st = check_chunk(p);
  if (st != MLA_OK) return st;
  if (!cu_seqlens || !cache_seqlens || !sched || !aligned(cu_seqlens, 4) || !aligned(cache_seqlens, 4) || !aligned16(sched))
    return MLA_ERR_INVALID_ARG;
  int32_t U = 0;
  if ((st = chunk_units(p, &U)) != MLA_OK) return st;
  mla_chunk_sched_kernel<<<1, 1024, 0, static_cast<cudaStream_t>(stream)>>>(
      cu_seqlens, cache_seqlens, p->batch, p->max_tokens, p->num_heads, p->causal != 0, p->max_pages_per_seq,
      chunk_kv_pages(p), U, chunk_block_capacity(p->max_tokens, p->batch, p->num_heads), static_cast<int32_t*>(sched));
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int32_t mla_chunk_attend(const mla_chunk_params* p, const void* q_nope_absorbed, const void* q_rope, const void* kv_pages,
                         const int32_t* block_table, const int32_t* cache_seqlens, float scale, void* out, float* lse,
                         const void* sched, void* workspace, void* stream) {
  int32_t st = check_chunk(p);
  if (st != MLA_OK) return st;
  for (const void* q : {q_nope_absorbed, q_rope, kv_pages, (const void*)out, (const void*)lse, sched})
    if (!q || !aligned16(q)) return MLA_ERR_INVALID_ARG;
  if (!block_table || !aligned(block_table, 4) || !cache_seqlens || !aligned(cache_seqlens, 4) || !workspace ||
      !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return MLA_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  if ((st = device_info(&d)) != MLA_OK) return st;
  {
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MLA_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(mla_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCkSmem) != cudaSuccess)
        return MLA_ERR_CUDA;
      attr_set[dev] = true;
    }
  }
  int32_t U = 0;
  if ((st = chunk_units(p, &U)) != MLA_OK) return st;
  const ChunkBuffers bufs = chunk_buffers(p, U);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int32_t* sc = static_cast<const int32_t*>(sched);
  const bool expanded = p->kv_dtype != MLA_KV_BF16;

  ChunkArgs a;
  std::memset(&a, 0, sizeof a);
  a.o_acc = reinterpret_cast<float*>(ws);
  a.lse_acc = reinterpret_cast<float*>(ws + bufs.o_acc);
  void* rows = ws + bufs.o_acc + align256(bufs.lse_acc);
  const uint64_t q_rows = (uint64_t)p->max_tokens * p->num_heads;
  const uint64_t kv_rows = expanded ? (uint64_t)(p->max_kv_tokens / 64) * 64 : (uint64_t)p->num_pages * 64;
  const void* kv = expanded ? rows : kv_pages;
  const uint32_t box2[2] = {64, 64}, box3[3] = {64, 64, 2}, boxq[3] = {64, 64, 8};
  {
    const uint64_t dq[3] = {64, q_rows, 8}, sq[2] = {1024, 128}, dr[2] = {64, q_rows}, sr[1] = {128};
    const uint64_t dk[2] = {576, kv_rows}, sk[1] = {1152}, dv[3] = {64, kv_rows, 9}, sv[2] = {1152, 128};
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if ((st = encode_map(&a.map_q, bf, 3, q_nope_absorbed, dq, sq, boxq, CU_TENSOR_MAP_SWIZZLE_128B)) ||
        (st = encode_map(&a.map_qr, bf, 2, q_rope, dr, sr, box2, CU_TENSOR_MAP_SWIZZLE_128B)) ||
        (st = encode_map(&a.map_k, bf, 2, kv, dk, sk, box2, CU_TENSOR_MAP_SWIZZLE_128B)) ||
        (st = encode_map(&a.map_v, bf, 3, kv, dv, sv, box3, CU_TENSOR_MAP_SWIZZLE_128B)))
      return st;
  }
  a.kv = static_cast<const uint8_t*>(kv);
  a.block_table = block_table;
  a.sched = sc;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.key = {U, (int32_t)bufs.cap, p->batch, p->causal != 0, p->max_tokens, p->num_heads, p->max_pages_per_seq, (int32_t)chunk_kv_pages(p)};
  a.num_pages = p->num_pages;
  a.expanded = expanded;
  a.timeout_ns = (uint64_t)(p->timeout_us > 0 ? p->timeout_us : 2000000) * 1000ull;
  if (expanded) {
    const int64_t pages = p->max_kv_tokens / 64, most = (int64_t)d->sm_count * 8;
    if ((st = launch_after(stream, dim3((unsigned)(pages < most ? pages : most)), 256, 0,
                           p->kv_dtype == MLA_KV_INT4 ? mla_chunk_expand_kernel<kKvInt4> : mla_chunk_expand_kernel<kKvFp8>, sc, a.key,
                           static_cast<const uint8_t*>(kv_pages), block_table, p->num_pages, cache_seqlens, static_cast<__nv_bfloat16*>(rows))))
      return st;
  }
  if ((st = launch_after(stream, dim3(2 * U), kCkThreads, kCkSmem, mla_chunk_kernel, a))) return st;
  const int64_t items = (int64_t)U * 128, most = (int64_t)d->sm_count * 3;  // at most U blocks are split
  return launch_after(stream, dim3((unsigned)(items < most ? items : most)), 256, 0, mla_chunk_combine_kernel, sc,
                      a.key, (const float*)a.o_acc, (const float*)a.lse_acc, a.out, lse);
}

int32_t mla_append_kv(const mla_pool_params* p, int64_t max_tokens, const void* latent, int64_t latent_stride,
                      const void* k_rope, int64_t rope_stride, const int32_t* cu_seqlens, const int32_t* cache_seqlens,
                      const int32_t* block_table, void* kv_pages, void* stream) {
  return append_kv(p, max_tokens, latent, latent_stride, k_rope, rope_stride, cu_seqlens, cache_seqlens, block_table, nullptr,
                   kv_pages, stream);
}

int32_t mla_append_served_kv(const mla_pool_params* p, int64_t max_tokens, const void* latent, int64_t latent_stride,
                             const void* k_rope, int64_t rope_stride, const int32_t* cu_seqlens,
                             const int32_t* cache_seqlens, const int32_t* block_table, const int32_t* served,
                             void* kv_pages, void* stream) {
  if (!served || !aligned(served, 4)) return MLA_ERR_INVALID_ARG;
  return append_kv(p, max_tokens, latent, latent_stride, k_rope, rope_stride, cu_seqlens, cache_seqlens, block_table, served,
                   kv_pages, stream);
}

int32_t mla_append_rotated_kv(const mla_pool_params* p, const mla_rotate_params* r, const void* latent, const void* k_rope,
                              const void* norm_weight, const float* cos_sin, const int32_t* positions, const void* q_rope,
                              void* q_out, const int32_t* cu_seqlens, const int32_t* cache_seqlens, const int32_t* block_table,
                              const int32_t* served, void* kv_pages, void* stream) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (!r || r->max_tokens < 0 || r->num_heads < 0 || r->max_positions < 1 || (r->interleaved != 0 && r->interleaved != 1))
    return MLA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (r->reserved[i] != 0) return MLA_ERR_INVALID_ARG;
  if (!all_int_arrays({latent, k_rope, cos_sin, kv_pages}) || (norm_weight && !aligned16(norm_weight)) || !cu_seqlens ||
      !cache_seqlens || !block_table || !aligned(cu_seqlens, 4) || !aligned(cache_seqlens, 4) || !aligned(block_table, 4) ||
      !aligned(positions, 4) || !aligned(served, 4))
    return MLA_ERR_INVALID_ARG;
  if (norm_weight && !(r->norm_eps >= 0.f && r->norm_eps < INFINITY)) return MLA_ERR_INVALID_ARG;
  if (r->latent_stride < 512 || r->latent_stride % 8 != 0 || r->rope_stride < 64 || r->rope_stride % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (r->num_heads > 0 && (!all_int_arrays({q_rope, q_out}) || r->q_token_stride % 8 != 0 || r->q_head_stride % 8 != 0 ||
                           r->q_token_stride < 0 || r->q_head_stride < 0))
    return MLA_ERR_INVALID_ARG;
  if (r->max_tokens > INT32_MAX || r->num_heads > 65535) return MLA_ERR_UNSUPPORTED;
  if (r->max_tokens == 0) return MLA_OK;
  RotateArgs a;
  std::memset(&a, 0, sizeof a);
  a.p = pool_args(p);
  a.max_tokens = r->max_tokens;
  a.latent_stride = r->latent_stride;
  a.rope_stride = r->rope_stride;
  a.q_token_stride = r->q_token_stride;
  a.q_head_stride = r->q_head_stride;
  a.latent = static_cast<const __nv_bfloat16*>(latent);
  a.rope = static_cast<const __nv_bfloat16*>(k_rope);
  a.weight = static_cast<const __nv_bfloat16*>(norm_weight);
  a.q = static_cast<const __nv_bfloat16*>(q_rope);
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.cu = cu_seqlens;
  a.lens = cache_seqlens;
  a.block_table = block_table;
  a.served = served;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.pages = static_cast<uint8_t*>(kv_pages);
  a.eps = r->norm_eps;
  a.heads = r->num_heads;
  a.max_positions = r->max_positions;
  a.warps = r->num_heads > 64 ? 4 : r->num_heads > 32 ? 2 : 1;
  const dim3 grid((unsigned)((r->max_tokens * a.warps + 7) / 8));
  const int pick = (served ? 1 : 0) + (r->interleaved ? 2 : 0);
  using Kernel = void (*)(RotateArgs);
#define MLA_ROTATE(F) {mla_append_rotated_kernel<F, false, false>, mla_append_rotated_kernel<F, true, false>, \
                       mla_append_rotated_kernel<F, false, true>, mla_append_rotated_kernel<F, true, true>}
  static const Kernel kernels[3][4] = {MLA_ROTATE(kKvBf16), MLA_ROTATE(kKvFp8), MLA_ROTATE(kKvInt4)};
#undef MLA_ROTATE
  return launch_after(stream, grid, 256, 0, kernels[p->kv_dtype][pick], a);
}

int32_t mla_quantize_kv_int4(const void* kv_bf16, void* kv_int4, int64_t num_tokens, void* stream) {
  if (!kv_bf16 || !kv_int4 || num_tokens < 0 || !aligned16(kv_bf16) || !aligned16(kv_int4)) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  const int64_t blocks = (num_tokens + 7) / 8;
  if (blocks > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  mla_quantize_int4_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(kv_bf16), static_cast<uint8_t*>(kv_int4), num_tokens);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int32_t mla_dequantize_kv(int32_t kv_dtype, const void* kv_rows, void* kv_bf16, int64_t num_tokens, void* stream) {
  const int row = kv_row_bytes(kv_dtype);
  if (row == 0 || !kv_rows || !kv_bf16 || num_tokens < 0 || !aligned16(kv_rows) || !aligned16(kv_bf16)) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  const int64_t blocks = (num_tokens + 7) / 8;
  if (blocks > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (kv_dtype == MLA_KV_BF16)
    return cudaMemcpyAsync(kv_bf16, kv_rows, (size_t)num_tokens * row, cudaMemcpyDeviceToDevice, s) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
  const uint8_t* rows = static_cast<const uint8_t*>(kv_rows);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(kv_bf16);
  if (kv_dtype == MLA_KV_FP8_E4M3)
    mla_dequantize_kernel<kKvFp8><<<(unsigned)blocks, 256, 0, s>>>(rows, out, num_tokens);
  else
    mla_dequantize_kernel<kKvInt4><<<(unsigned)blocks, 256, 0, s>>>(rows, out, num_tokens);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int32_t mla_pool_workspace_size(const mla_pool_params* p, int32_t max_forks, size_t* workspace_bytes) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (max_forks < 0 || !workspace_bytes) return MLA_ERR_INVALID_ARG;
  const size_t fork = (size_t)2 * max_forks + p->batch, reserve = (size_t)p->batch + 1;
  const size_t compact = 4 + (size_t)p->num_pages + 2 * ((size_t)p->num_pages / 2 + 1);
  size_t n = fork > reserve ? fork : reserve;
  n = n > compact ? n : compact;
  *workspace_bytes = align256(n * sizeof(int32_t));
  return MLA_OK;
}

int32_t mla_copy_pages(const mla_pool_params* p, void* kv_pages, const int32_t* src_pages, const int32_t* dst_pages,
                       int32_t num_copies, void* stream) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (num_copies < 0 || !kv_pages || !aligned16(kv_pages) || !src_pages || !dst_pages || !aligned(src_pages, 4) ||
      !aligned(dst_pages, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_copies == 0) return MLA_OK;
  return launch_after(stream, dim3(num_copies, p->num_layers * kCopyParts), 256, 0, mla_copy_pages_kernel, pool_args(p),
                      static_cast<uint8_t*>(kv_pages), src_pages, dst_pages);
}

int32_t mla_fork_sequences(const mla_pool_params* p, void* kv_pages, const int32_t* parents, const int32_t* children,
                           int32_t num_forks, int32_t* block_table, int32_t* cache_seqlens, int32_t* ref_counts,
                           int32_t* new_pages, void* workspace, void* stream) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (num_forks < 0 || !kv_pages || !aligned16(kv_pages) || !all_int_arrays({block_table, cache_seqlens, ref_counts, workspace}) ||
      !parents || !children || !new_pages || !aligned(parents, 4) || !aligned(children, 4) || !aligned(new_pages, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_forks == 0) return MLA_OK;
  int32_t* ws = static_cast<int32_t*>(workspace);
  const PoolArgs a = pool_args(p);
  if ((st = launch_after(stream, dim3(1), 1024, 0, mla_fork_plan_kernel, a, parents, children, num_forks, cache_seqlens,
                         ref_counts, new_pages, ws)))
    return st;
  return launch_after(stream, dim3(num_forks, 1 + p->num_layers), 256, 0, mla_fork_kernel, a,
                      static_cast<uint8_t*>(kv_pages), parents, children, block_table, ref_counts,
                      (const int32_t*)new_pages, (const int32_t*)ws);
}

int32_t mla_reserve_pages(const mla_pool_params* p, const int32_t* num_new, int32_t* block_table, int32_t* cache_seqlens,
                          int32_t* ref_counts, int32_t* served, void* workspace, void* stream) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (!all_int_arrays({block_table, cache_seqlens, ref_counts, workspace}) || !num_new || !served || !aligned(num_new, 4) ||
      !aligned(served, 4))
    return MLA_ERR_INVALID_ARG;
  return launch_after(stream, dim3(1), 1024, 0, mla_reserve_kernel, pool_args(p), num_new, block_table, cache_seqlens,
                      ref_counts, served, static_cast<int32_t*>(workspace));
}

int32_t mla_free_sequences(const mla_pool_params* p, const int32_t* sequences, int32_t num_sequences, int32_t* block_table,
                           int32_t* cache_seqlens, int32_t* ref_counts, void* stream) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (num_sequences < 0 || !all_int_arrays({block_table, cache_seqlens, ref_counts}) || !sequences || !aligned(sequences, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_sequences == 0) return MLA_OK;
  return launch_after(stream, dim3(num_sequences), 128, 0, mla_free_kernel, pool_args(p), sequences, block_table,
                      cache_seqlens, ref_counts);
}

int32_t mla_compact_pages(const mla_pool_params* p, void* kv_pages, int32_t* block_table, const int32_t* cache_seqlens,
                          int32_t* ref_counts, int32_t* num_used, void* workspace, void* stream) {
  int32_t st = check_pool(p);
  if (st != MLA_OK) return st;
  if (!kv_pages || !aligned16(kv_pages) || !all_int_arrays({block_table, cache_seqlens, ref_counts, workspace}) || !num_used ||
      !aligned(num_used, 4))
    return MLA_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  if ((st = device_info(&d)) != MLA_OK) return st;
  int32_t* ws = static_cast<int32_t*>(workspace);
  const PoolArgs a = pool_args(p);
  if ((st = launch_after(stream, dim3(1), 1024, 0, mla_compact_plan_kernel, a, ref_counts, num_used, ws))) return st;
  // at most num_pages / 2 pages move: no more blocks than there could be work for
  const int64_t items = (int64_t)(p->num_pages / 2) * p->num_layers * kCopyParts + p->batch, most = (int64_t)d->sm_count * 8;
  return launch_after(stream, dim3((unsigned)(items < most ? items : most)), 256, 0, mla_compact_kernel, a,
                      static_cast<uint8_t*>(kv_pages), block_table, cache_seqlens, (const int32_t*)ws);
}

}  // extern "C"
