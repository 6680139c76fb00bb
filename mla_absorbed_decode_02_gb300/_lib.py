"""ctypes binding of libmla_decode.so (names mirror include/mla_decode.h).

Argument marshalling only: tensors go in as raw device pointers, the stream as
the CUDA stream handle.  Every step of the decode runs in the library's
kernels; there is no fallback path -- if the library is missing, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

(MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA, MLA_ERR_TIMEOUT, MLA_ERR_WORKSPACE,
 MLA_ERR_SCRATCH_LIMIT) = range(7)
MLA_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_INT4 = 0, 1, 2
_ROW_BYTES = (1152, 656, 416)  # of a cached token, by format
MLA_OUT_BF16, MLA_OUT_F32 = 0, 1
SCHED_MAGIC = 0x4D4C4131

_PKG = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return os.path.join(_PKG, "libmla_decode.so")


class MlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_name(status)} ({status})")


class MlaDecodeParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("s_q", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("causal", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("num_units", ctypes.c_int32), ("timeout_us", ctypes.c_int32),
                ("token_group", ctypes.c_int32), ("qk_fp8", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]

    @classmethod
    def make(cls, batch, s_q, num_heads, num_pages, max_pages_per_seq, causal=True, kv_dtype=MLA_KV_BF16,
             out_dtype=MLA_OUT_BF16, num_units=0, timeout_us=0, page_size=64, token_group=0, qk_fp8=0):
        return cls(batch, s_q, num_heads, num_pages, page_size, max_pages_per_seq, int(bool(causal)), kv_dtype,
                   out_dtype, num_units, timeout_us, token_group, int(qk_fp8))


class MlaExtendParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("s_q", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("d_nope", ctypes.c_int32), ("d_v", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32), ("max_seqlen", ctypes.c_int32),
                ("chunk_tokens", ctypes.c_int32), ("timeout_us", ctypes.c_int32), ("reserved", ctypes.c_int32 * 5)]

    @classmethod
    def make(cls, batch, s_q, num_heads, num_pages, max_pages_per_seq, max_seqlen, chunk_tokens=4096, d_nope=128,
             d_v=128, timeout_us=0, page_size=64):
        return cls(batch, s_q, num_heads, d_nope, d_v, num_pages, page_size, max_pages_per_seq, max_seqlen,
                   chunk_tokens, timeout_us)


class MlaChunkParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("kv_dtype", ctypes.c_int32), ("num_units", ctypes.c_int32),
                ("timeout_us", ctypes.c_int32), ("max_kv_tokens", ctypes.c_int64), ("reserved", ctypes.c_int32 * 4)]

    @classmethod
    def make(cls, batch, max_tokens, num_heads, num_pages, max_pages_per_seq, causal=True, kv_dtype=MLA_KV_BF16,
             max_kv_tokens=0, num_units=0, timeout_us=0, page_size=64):
        return cls(batch, max_tokens, num_heads, num_pages, page_size, max_pages_per_seq, int(bool(causal)), kv_dtype,
                   num_units, timeout_us, max_kv_tokens)


class MlaPoolParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("kv_dtype", ctypes.c_int32), ("num_layers", ctypes.c_int32),
                ("layer_stride", ctypes.c_int64), ("reserved", ctypes.c_int32 * 4)]

    @classmethod
    def make(cls, batch, num_pages, max_pages_per_seq, kv_dtype=MLA_KV_BF16, num_layers=1, layer_stride=0, page_size=64):
        return cls(batch, num_pages, page_size, max_pages_per_seq, kv_dtype, num_layers, layer_stride)


class MlaRotateParams(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int64), ("latent_stride", ctypes.c_int64), ("rope_stride", ctypes.c_int64),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("max_positions", ctypes.c_int32), ("norm_eps", ctypes.c_float),
                ("reserved", ctypes.c_int32 * 4)]


def load_library():
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with mla_absorbed_decode_02_gb300.build.build()")
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER(MlaDecodeParams)
        X = ctypes.POINTER(MlaExtendParams)
        C = ctypes.POINTER(MlaChunkParams)
        K = ctypes.POINTER(MlaPoolParams)
        R = ctypes.POINTER(MlaRotateParams)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "mla_get_workspace_size": ([P, ctypes.POINTER(sz), ctypes.POINTER(sz)], i32),
            "mla_get_scheduler_metadata": ([P, vp, vp, vp], i32),
            "mla_decode": ([P, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp], i32),
            "mla_decode_splitkv": ([P, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp], i32),
            "mla_combine": ([P, vp, vp, vp, vp, vp], i32),
            "mla_plan_host": ([P, i32, vp, vp], i32),
            "mla_resolve_num_units": ([P, ctypes.POINTER(i32)], i32),
            "mla_device_error": ([ctypes.POINTER(i32), i32], i32),
            "mla_wait_selftest": ([i32, vp], i32),
            "mla_decode_noalloc": ([P, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp], i32),
            "mla_quantize_kv_fp8": ([vp, vp, ctypes.c_int64, vp], i32),
            "mla_quantize_kv_int4": ([vp, vp, ctypes.c_int64, vp], i32),
            "mla_dequantize_kv": ([i32, vp, vp, ctypes.c_int64, vp], i32),
            "mla_append_rotated_kv": ([K, R] + [vp] * 13, i32),
            "mla_quantize_q_fp8": ([vp, vp, vp, ctypes.c_int64, vp], i32),
            "mla_absorb_query": ([i32, i32, i32, vp, vp, vp, vp], i32),
            "mla_project_output": ([i32, i32, i32, vp, vp, vp, vp], i32),
            "mla_extend_workspace_size": ([X, ctypes.POINTER(sz)], i32),
            "mla_expand_kv": ([X, vp, vp, vp, vp, vp, i32, vp, vp, vp], i32),
            "mla_extend": ([X, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp], i32),
            "mla_chunk_workspace_size": ([C, ctypes.POINTER(sz), ctypes.POINTER(sz)], i32),
            "mla_chunk_plan_host": ([C, i32, vp, vp, vp], i32),
            "mla_chunk_schedule": ([C, vp, vp, vp, vp], i32),
            "mla_chunk_attend": ([C, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp], i32),
            "mla_append_kv": ([K, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp], i32),
            "mla_append_served_kv": ([K, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp], i32),
            "mla_pool_workspace_size": ([K, i32, ctypes.POINTER(sz)], i32),
            "mla_copy_pages": ([K, vp, vp, vp, i32, vp], i32),
            "mla_fork_sequences": ([K, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp], i32),
            "mla_reserve_pages": ([K, vp, vp, vp, vp, vp, vp, vp], i32),
            "mla_free_sequences": ([K, vp, i32, vp, vp, vp, vp], i32),
            "mla_compact_pages": ([K, vp, vp, vp, vp, vp, vp, vp], i32),
            "mla_status_string": ([i32], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def _status_name(status: int) -> str:
    names = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_CUDA",
             4: "MLA_ERR_TIMEOUT", 5: "MLA_ERR_WORKSPACE", 6: "MLA_ERR_SCRATCH_LIMIT"}
    return names.get(status, "MLA_ERR_UNKNOWN")


def _check(status: int, what: str):
    if status != MLA_OK:
        raise MlaError(status, what)


def _ptr(t) -> int:
    if t is None:
        return 0
    return int(t.data_ptr())


_raw = None  # torch._C, once CUDA is up and it gives raw streams


def _stream(stream) -> int:
    global _raw
    if type(stream) is int:
        return stream
    if stream is None:
        if _raw is None:
            import torch
            if not (torch.cuda.is_initialized() and hasattr(torch._C, "_cuda_getCurrentRawStream")):
                return int(torch.cuda.current_stream().cuda_stream)
            _raw = torch._C
        return _raw._cuda_getCurrentRawStream(_raw._cuda_getDevice())  # 0.2 us; the Stream object costs 3
    return int(getattr(stream, "cuda_stream", stream))


_types = None


def _dtypes():
    """(int32, float32, bfloat16) of torch, looked up once."""
    global _types
    if _types is None:
        import torch
        _types = (torch.int32, torch.float32, torch.bfloat16)
    return _types


def mla_status_string(status: int) -> str:
    return load_library().mla_status_string(status).decode()


def mla_get_workspace_size(p: MlaDecodeParams):
    sb, wb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().mla_get_workspace_size(ctypes.byref(p), ctypes.byref(sb), ctypes.byref(wb)),
           "mla_get_workspace_size")
    return sb.value, wb.value


def mla_resolve_num_units(p: MlaDecodeParams) -> int:
    u = ctypes.c_int32()
    _check(load_library().mla_resolve_num_units(ctypes.byref(p), ctypes.byref(u)), "mla_resolve_num_units")
    return u.value


def mla_plan_host(p: MlaDecodeParams, num_units: int, cache_seqlens) -> np.ndarray:
    """Host twin of the split planner; returns the int32 metadata array."""
    seq = np.ascontiguousarray(cache_seqlens, dtype=np.int32)
    nqb = p.batch * p.s_q
    out = np.zeros(8 + 8 * num_units + 2 * nqb, np.int32)
    _check(load_library().mla_plan_host(ctypes.byref(p), num_units, seq.ctypes.data, out.ctypes.data),
           "mla_plan_host")
    return out


def mla_get_scheduler_metadata(p: MlaDecodeParams, cache_seqlens, sched, stream=None):
    _check(load_library().mla_get_scheduler_metadata(ctypes.byref(p), _ptr(cache_seqlens), _ptr(sched),
                                                     _stream(stream)), "mla_get_scheduler_metadata")


def mla_decode(p: MlaDecodeParams, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens, scale: float, out,
               lse, sched, workspace, stream=None):
    _check(load_library().mla_decode(ctypes.byref(p), _ptr(q_nope_absorbed), _ptr(q_rope), _ptr(kv_pages),
                                     _ptr(block_table), _ptr(cache_seqlens), float(scale), _ptr(out), _ptr(lse),
                                     _ptr(sched), _ptr(workspace), _stream(stream)), "mla_decode")


def mla_decode_splitkv(p: MlaDecodeParams, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens,
                       scale: float, out, lse, sched, workspace, stream=None):
    _check(load_library().mla_decode_splitkv(ctypes.byref(p), _ptr(q_nope_absorbed), _ptr(q_rope), _ptr(kv_pages),
                                             _ptr(block_table), _ptr(cache_seqlens), float(scale), _ptr(out),
                                             _ptr(lse), _ptr(sched), _ptr(workspace), _stream(stream)),
           "mla_decode_splitkv")


def mla_combine(p: MlaDecodeParams, out, lse, sched, workspace, stream=None):
    _check(load_library().mla_combine(ctypes.byref(p), _ptr(out), _ptr(lse), _ptr(sched), _ptr(workspace),
                                      _stream(stream)), "mla_combine")


def mla_decode_noalloc(p: MlaDecodeParams, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens,
                       scale: float, out, lse, stream=None):
    """Scheduler metadata + decode with the library's fixed device scratch array
    instead of caller buffers (for callers that cannot allocate device memory)."""
    _check(load_library().mla_decode_noalloc(ctypes.byref(p), _ptr(q_nope_absorbed), _ptr(q_rope), _ptr(kv_pages),
                                             _ptr(block_table), _ptr(cache_seqlens), float(scale), _ptr(out),
                                             _ptr(lse), _stream(stream)), "mla_decode_noalloc")


def mla_quantize_kv_fp8(kv_bf16, kv_fp8, num_tokens: int, stream=None):
    """bf16 cache rows [n, 576] -> 656-byte FP8 rows [n, 656] (codes, tile scales, RoPE)."""
    _check(load_library().mla_quantize_kv_fp8(_ptr(kv_bf16), _ptr(kv_fp8), int(num_tokens), _stream(stream)),
           "mla_quantize_kv_fp8")


def _rows_of(call, t, name, num_tokens, row_bytes, dtypes):
    """Checks a buffer of rows one after another, on the current device."""
    if (t is None or t.dtype not in dtypes or not t.is_contiguous() or num_tokens < 0
            or t.numel() * t.element_size() < num_tokens * row_bytes):
        _refuse(f"{call}: {name}")


def _rows_apart(call, a, b, num_tokens, a_bytes, b_bytes):
    """The rows of two buffers do not meet: other warps read one while a row of the other is written."""
    at, to = a.data_ptr(), b.data_ptr()
    if at < to + num_tokens * b_bytes and to < at + num_tokens * a_bytes:
        _refuse(f"{call}: rows overlap")


def mla_quantize_kv_int4(kv_bf16, kv_int4, num_tokens: int, stream=None):
    """bf16 cache rows [n, 576] -> 416-byte INT4 rows, uint8 [n, 416] (codes, scales, RoPE)."""
    import torch
    _rows_of("mla_quantize_kv_int4", kv_bf16, "kv_bf16", num_tokens, 1152, (torch.bfloat16,))
    _rows_of("mla_quantize_kv_int4", kv_int4, "kv_int4", num_tokens, 416, (torch.uint8, torch.int8))
    if num_tokens == 0:
        return
    _rows_apart("mla_quantize_kv_int4", kv_bf16, kv_int4, num_tokens, 1152, 416)
    _expect_device("mla_quantize_kv_int4", kv_bf16, kv_int4)
    _check(load_library().mla_quantize_kv_int4(_ptr(kv_bf16), _ptr(kv_int4), int(num_tokens), _stream(stream)),
           "mla_quantize_kv_int4")


def mla_dequantize_kv(kv_dtype: int, kv_rows, kv_bf16, num_tokens: int, stream=None):
    """Rows of a cache of any format (MLA_KV_*, a pool's pages hold them one after another; uint8, or bf16 rows as such)
    -> bf16 rows [n, 576]."""
    import torch
    if not 0 <= kv_dtype < 3:
        _refuse("mla_dequantize_kv: kv_dtype")
    rows = (torch.uint8, torch.int8) + ((torch.bfloat16,) if kv_dtype == MLA_KV_BF16 else ())
    _rows_of("mla_dequantize_kv", kv_rows, "kv_rows", num_tokens, _ROW_BYTES[kv_dtype], rows)
    _rows_of("mla_dequantize_kv", kv_bf16, "kv_bf16", num_tokens, 1152, (torch.bfloat16,))
    if num_tokens == 0:
        return
    _rows_apart("mla_dequantize_kv", kv_rows, kv_bf16, num_tokens, _ROW_BYTES[kv_dtype], 1152)
    _expect_device("mla_dequantize_kv", kv_rows, kv_bf16)
    _check(load_library().mla_dequantize_kv(kv_dtype, _ptr(kv_rows), _ptr(kv_bf16), int(num_tokens), _stream(stream)),
           "mla_dequantize_kv")


def mla_quantize_q_fp8(q_nope_absorbed, q_rope, q_fp8, num_rows: int, stream=None):
    """Query rows for an FP8-QK decode: q~ bf16 [n, 512] and q^R bf16 [n, 64] -> 656-byte rows [n, 656]."""
    _check(load_library().mla_quantize_q_fp8(_ptr(q_nope_absorbed), _ptr(q_rope), _ptr(q_fp8), int(num_rows),
                                             _stream(stream)), "mla_quantize_q_fp8")


def mla_absorb_query(q_nope, w_uk, q_absorbed, stream=None):
    """q_absorbed[t, h] = q_nope[t, h] @ w_uk[h]: q_nope bf16 [..., H, d_nope], w_uk bf16 [H, d_nope, 512],
    q_absorbed bf16 [..., H, 512] (leading dims flattened to tokens)."""
    H, d_nope = int(q_nope.shape[-2]), int(q_nope.shape[-1])
    T = int(q_nope.numel() // (H * d_nope))
    _check(load_library().mla_absorb_query(T, H, d_nope, _ptr(q_nope), _ptr(w_uk), _ptr(q_absorbed), _stream(stream)),
           "mla_absorb_query")


def mla_project_output(o_latent, w_uv, out, stream=None):
    """out[t, h] = o_latent[t, h] @ w_uv[h]: o_latent bf16 [..., H, 512], w_uv bf16 [H, 512, d_v],
    out bf16 [..., H, d_v] (leading dims flattened to tokens)."""
    H = int(o_latent.shape[-2])
    T = int(o_latent.numel() // (H * 512))
    d_v = int(w_uv.shape[-1])
    _check(load_library().mla_project_output(T, H, d_v, _ptr(o_latent), _ptr(w_uv), _ptr(out), _stream(stream)),
           "mla_project_output")


def mla_extend_workspace_size(p: MlaExtendParams) -> int:
    n = ctypes.c_size_t()
    _check(load_library().mla_extend_workspace_size(ctypes.byref(p), ctypes.byref(n)), "mla_extend_workspace_size")
    return n.value


def mla_expand_kv(p: MlaExtendParams, kv_pages, block_table, cache_seqlens, w_uk, w_uv, chunk_start: int, k_nope, v,
                  stream=None):
    """k_nope[b, h, j] = w_uk[h] @ c_j and v[b, h, j] = c_j @ w_uv[h] for cache rows j of one chunk:
    k_nope, v bf16 [B, H, chunk_tokens, 128]."""
    _check(load_library().mla_expand_kv(ctypes.byref(p), _ptr(kv_pages), _ptr(block_table), _ptr(cache_seqlens),
                                        _ptr(w_uk), _ptr(w_uv), int(chunk_start), _ptr(k_nope), _ptr(v),
                                        _stream(stream)), "mla_expand_kv")


def mla_extend(p: MlaExtendParams, q_nope, q_rope, kv_pages, block_table, cache_seqlens, w_uk, w_uv, scale: float,
               out, lse, workspace, stream=None):
    """Extend by the expand path, chunk by chunk: out bf16 [B, s_q, H, 128], lse float32 [B, s_q, H]."""
    _check(load_library().mla_extend(ctypes.byref(p), _ptr(q_nope), _ptr(q_rope), _ptr(kv_pages), _ptr(block_table),
                                     _ptr(cache_seqlens), _ptr(w_uk), _ptr(w_uv), float(scale), _ptr(out), _ptr(lse),
                                     _ptr(workspace), _stream(stream)), "mla_extend")


def _bad(t, dtype, shape) -> bool:
    """Not a contiguous tensor of this type and shape.  The library sees pointers alone, so what it cannot check is
    checked here (inline in each call: a step's small operations are bound by the host)."""
    return t is None or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()


def _refuse(what: str, status: int = MLA_ERR_INVALID_ARG):
    raise MlaError(status, what)


def _expect_device(call: str, first, *others):
    """All on the current CUDA device: a pointer of the host or of another device must not reach a kernel."""
    import torch
    d = first.get_device()
    for t in others:
        if t.get_device() != d:
            _refuse(call + ": tensors on different devices")
    if d < 0 or d != torch._C._cuda_getDevice():
        _refuse(call + ": tensors are not on the current CUDA device")


def _expect_pool(call: str, t, p, num_layers: int = 1, layer_stride: int = 0):
    """The pools' pages: large enough for the last layer's last page, rows not strided."""
    pool = p.num_pages * 64 * (_ROW_BYTES[p.kv_dtype] if 0 <= p.kv_dtype < 3 else 1152)
    if (t is None or not t.is_contiguous()
            or t.numel() * t.element_size() < (num_layers - 1) * (layer_stride or pool) + pool):
        _refuse(call + ": kv_pages")


def mla_chunk_workspace_size(p: MlaChunkParams):
    sb, wb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().mla_chunk_workspace_size(ctypes.byref(p), ctypes.byref(sb), ctypes.byref(wb)),
           "mla_chunk_workspace_size")
    return sb.value, wb.value


def mla_chunk_plan_host(p: MlaChunkParams, num_units: int, cu_seqlens, cache_seqlens) -> np.ndarray:
    """Host twin of mla_chunk_schedule; returns the int32 metadata array."""
    cu = np.ascontiguousarray(cu_seqlens, dtype=np.int32)
    seq = np.ascontiguousarray(cache_seqlens, dtype=np.int32)
    if cu.shape != (p.batch + 1,) or seq.shape != (p.batch,):
        raise MlaError(MLA_ERR_INVALID_ARG, "mla_chunk_plan_host")
    q = MlaChunkParams.from_buffer_copy(p)
    q.num_units = num_units
    out = np.zeros(mla_chunk_workspace_size(q)[0] // 4, np.int32)
    _check(load_library().mla_chunk_plan_host(ctypes.byref(p), num_units, cu.ctypes.data, seq.ctypes.data,
                                              out.ctypes.data), "mla_chunk_plan_host")
    return out


def mla_chunk_schedule(p: MlaChunkParams, cu_seqlens, cache_seqlens, sched, stream=None):
    """Work plan of ragged chunks: cu_seqlens int32 [B + 1], cache_seqlens int32 [B] (new tokens included)."""
    i32 = _dtypes()[0]
    if _bad(cu_seqlens, i32, (p.batch + 1,)):
        _refuse("mla_chunk_schedule: cu_seqlens")
    if _bad(cache_seqlens, i32, (p.batch,)):
        _refuse("mla_chunk_schedule: cache_seqlens")
    if sched is None or sched.numel() * sched.element_size() < mla_chunk_workspace_size(p)[0]:
        _refuse("mla_chunk_schedule: sched", MLA_ERR_WORKSPACE)
    _expect_device("mla_chunk_schedule", cu_seqlens, cache_seqlens, sched)
    _check(load_library().mla_chunk_schedule(ctypes.byref(p), cu_seqlens.data_ptr(), cache_seqlens.data_ptr(), sched.data_ptr(),
                                             _stream(stream)), "mla_chunk_schedule")


def mla_chunk_attend(p: MlaChunkParams, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens, scale: float,
                     out, lse, sched, workspace, stream=None):
    """Attention of ragged chunks over the paged cache: q bf16 [T, H, 512] and [T, H, 64], out bf16 [T, H, 512],
    lse float32 [T, H]."""
    sb, wb = mla_chunk_workspace_size(p)
    for name, t, n in (("sched", sched, sb), ("workspace", workspace, wb)):
        if t is None or t.numel() * t.element_size() < n:
            _refuse("mla_chunk_attend: " + name, MLA_ERR_WORKSPACE)
    _attend(p, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens, scale, out, lse, sched, workspace, stream)


def _attend(p, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens, scale, out, lse, sched, workspace, stream):
    T, H, B = p.max_tokens, p.num_heads, p.batch
    i32, f32, bf16 = _dtypes()
    if _bad(q_nope_absorbed, bf16, (T, H, 512)):
        _refuse("mla_chunk_attend: q_nope_absorbed")
    if _bad(q_rope, bf16, (T, H, 64)):
        _refuse("mla_chunk_attend: q_rope")
    if _bad(block_table, i32, (B, p.max_pages_per_seq)):
        _refuse("mla_chunk_attend: block_table")
    if _bad(cache_seqlens, i32, (B,)):
        _refuse("mla_chunk_attend: cache_seqlens")
    if _bad(out, bf16, (T, H, 512)):
        _refuse("mla_chunk_attend: out")
    if _bad(lse, f32, (T, H)):
        _refuse("mla_chunk_attend: lse")
    _expect_pool("mla_chunk_attend", kv_pages, p)
    _expect_device("mla_chunk_attend", q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens, out, lse, sched,
                   workspace)
    _check(load_library().mla_chunk_attend(ctypes.byref(p), _ptr(q_nope_absorbed), _ptr(q_rope), _ptr(kv_pages),
                                           _ptr(block_table), _ptr(cache_seqlens), float(scale), _ptr(out), _ptr(lse),
                                           _ptr(sched), _ptr(workspace), _stream(stream)), "mla_chunk_attend")


def mla_append_kv(p: MlaPoolParams, latent, k_rope, cu_seqlens, cache_seqlens, block_table, kv_pages, stream=None,
                  served=None):
    """Rows of ragged new tokens into the pages: latent bf16 [T, 512] and k_rope bf16 [T, 64], rows of either may be
    strided (the two parts of one [T, 576] array).  With served (int32 [B], from mla_reserve_pages) the tokens of
    sequences that did not get their pages go nowhere."""
    i32, _, bf16 = _dtypes()
    B = p.batch
    for name, t, n in (("latent", latent, 512), ("k_rope", k_rope, 64)):
        if t is None or t.dtype != bf16 or t.dim() != 2 or t.shape[1] != n or t.stride(1) != 1:
            _refuse("mla_append_kv: " + name)
    if k_rope.shape[0] != latent.shape[0]:
        _refuse("mla_append_kv: k_rope")
    if _bad(cu_seqlens, i32, (B + 1,)):
        _refuse("mla_append_kv: cu_seqlens")
    if _bad(cache_seqlens, i32, (B,)):
        _refuse("mla_append_kv: cache_seqlens")
    if _bad(block_table, i32, (B, p.max_pages_per_seq)):
        _refuse("mla_append_kv: block_table")
    if served is not None and _bad(served, i32, (B,)):
        _refuse("mla_append_kv: served")
    _expect_pool("mla_append_kv", kv_pages, p)
    if latent.shape[0] == 0:
        return
    _expect_device("mla_append_kv", latent, k_rope, cu_seqlens, cache_seqlens, block_table, kv_pages)
    # (one row: its stride says nothing)
    ls, rs = (int(t.stride(0)) if t.shape[0] > 1 else n for t, n in ((latent, 512), (k_rope, 64)))
    if served is not None:
        _expect_device("mla_append_kv", served)
        _check(load_library().mla_append_served_kv(ctypes.byref(p), int(latent.shape[0]), latent.data_ptr(), ls, k_rope.data_ptr(), rs,
                                                   cu_seqlens.data_ptr(), cache_seqlens.data_ptr(), block_table.data_ptr(),
                                                   served.data_ptr(), kv_pages.data_ptr(), _stream(stream)), "mla_append_served_kv")
        return
    _check(load_library().mla_append_kv(ctypes.byref(p), int(latent.shape[0]), latent.data_ptr(), ls, k_rope.data_ptr(), rs,
                                        cu_seqlens.data_ptr(), cache_seqlens.data_ptr(), block_table.data_ptr(), kv_pages.data_ptr(),
                                        _stream(stream)), "mla_append_kv")


def mla_rope_table(max_positions: int, theta: float = 10000.0, device="cuda"):
    """The cosines and sines that mla_append_rotated_kv reads, float32 [max_positions, 64]: 32 cosines, then 32 sines, of
    pos * theta ** (-i / 32).  The angles are taken in float64: in float32 those of far positions are off by hundredths."""
    import torch
    pos = torch.arange(max_positions, dtype=torch.float64, device=device)
    angle = pos[:, None] * theta ** (-torch.arange(32, dtype=torch.float64, device=device) / 32.0)
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def _meets(at: int, size: int, first: int, rows: int, stride: int, row_bytes: int) -> bool:
    """Whether [at, at + size) touches one of the rows that start at first, first + stride, ..."""
    if at >= first + (rows - 1) * stride + row_bytes or at + size <= first:
        return False
    if rows == 1 or at <= first or stride < row_bytes:
        return True
    into = (at - first) % stride  # from the last row that starts at or before it
    return into < row_bytes or into + size > stride


def mla_append_rotated_kv(p: MlaPoolParams, latent, k_rope, cos_sin, cu_seqlens, cache_seqlens, block_table, kv_pages,
                          q_rope=None, q_out=None, positions=None, norm_weight=None, norm_eps: float = 1e-6,
                          interleaved: bool = False, served=None, stream=None):
    """mla_append_kv of rows as a model's layer has them: latent bf16 [T, 512] normed on the way where norm_weight (bf16 [512])
    is given, k_rope bf16 [T, 64] rotated by cos_sin (float32 [positions, 64], mla_rope_table), and the queries' q_rope
    bf16 [T, H, 64] (heads and tokens may be strided) rotated into q_out (bf16 [T, H, 64], made if not given).  A
    token's position is its row in its sequence, or positions[t] (int32 [T]).  Returns q_out."""
    i32, f32, bf16 = _dtypes()
    B, call = p.batch, "mla_append_rotated_kv: "
    # (shapes and strides are asked for once each: a step's call is bound by the host)
    if latent is None or latent.dtype is not bf16 or latent.dim() != 2:
        _refuse(call + "latent")
    (T, n), (latent_stride, one) = latent.shape, latent.stride()
    if n != 512 or one != 1:
        _refuse(call + "latent")
    if k_rope is None or k_rope.dtype is not bf16 or k_rope.dim() != 2:
        _refuse(call + "k_rope")
    (n, width), (rope_stride, one) = k_rope.shape, k_rope.stride()
    if n != T or width != 64 or one != 1:
        _refuse(call + "k_rope")
    if cos_sin is None or cos_sin.dtype is not f32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        _refuse(call + "cos_sin")
    num_positions, width = cos_sin.shape
    if width != 64 or num_positions == 0:
        _refuse(call + "cos_sin")
    if _bad(cu_seqlens, i32, (B + 1,)):
        _refuse(call + "cu_seqlens")
    if _bad(cache_seqlens, i32, (B,)):
        _refuse(call + "cache_seqlens")
    if _bad(block_table, i32, (B, p.max_pages_per_seq)):
        _refuse(call + "block_table")
    if positions is not None and _bad(positions, i32, (T,)):
        _refuse(call + "positions")
    if norm_weight is not None and _bad(norm_weight, bf16, (512,)):
        _refuse(call + "norm_weight")
    if served is not None and _bad(served, i32, (B,)):
        _refuse(call + "served")
    H = token_stride = head_stride = q_at = out_at = 0
    if q_rope is not None:
        if q_rope.dtype is not bf16 or q_rope.dim() != 3:
            _refuse(call + "q_rope")
        (n, H, width), (token_stride, head_stride, one) = q_rope.shape, q_rope.stride()
        if n != T or width != 64 or one != 1:
            _refuse(call + "q_rope")
        made = q_out is None
        if made:
            q_out = _new(q_rope, stream, (T, H, 64), bf16)
        elif _bad(q_out, bf16, (T, H, 64)):
            _refuse(call + "q_out")
        if T and H:
            q_at, out_at = q_rope.data_ptr(), q_out.data_ptr()
            if not made:
                # (read and written by the same threads where the two are one, by others where they merely overlap)
                size, last = T * H * 128, (T - 1) * token_stride + (H - 1) * head_stride + 64
                if (q_at < out_at + size and out_at < q_at + 2 * last
                        and not (out_at == q_at and q_rope.is_contiguous())):
                    _refuse(call + "q_out overlaps q_rope")
                if (_meets(out_at, size, latent.data_ptr(), T, 2 * latent_stride, 1024)
                        or _meets(out_at, size, k_rope.data_ptr(), T, 2 * rope_stride, 128)):
                    _refuse(call + "q_out overlaps latent or k_rope")
    elif q_out is not None:
        _refuse(call + "q_out without q_rope")
    _expect_pool("mla_append_rotated_kv", kv_pages, p)
    if T == 0:
        return q_out
    _expect_device("mla_append_rotated_kv", latent, k_rope, cos_sin, cu_seqlens, cache_seqlens, block_table, kv_pages,
                   *[t for t in (positions, norm_weight, served, q_rope, q_out) if t is not None])
    # (one row, or one head: its stride says nothing)
    r = MlaRotateParams(T, latent_stride if T > 1 else 512, rope_stride if T > 1 else 64, token_stride if H and T > 1 else 0,
                        head_stride if H > 1 else 0, H, 1 if interleaved else 0, num_positions, norm_eps)
    _check(load_library().mla_append_rotated_kv(ctypes.byref(p), ctypes.byref(r), latent.data_ptr(), k_rope.data_ptr(), _ptr(norm_weight),
                                                cos_sin.data_ptr(), _ptr(positions), q_at, out_at,
                                                cu_seqlens.data_ptr(), cache_seqlens.data_ptr(), block_table.data_ptr(), _ptr(served),
                                                kv_pages.data_ptr(), _stream(stream)), "mla_append_rotated_kv")
    return q_out


def mla_pool_workspace_size(p: MlaPoolParams, max_forks: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().mla_pool_workspace_size(ctypes.byref(p), int(max_forks), ctypes.byref(n)),
           "mla_pool_workspace_size")
    return n.value


def _expect_tables(call: str, p: MlaPoolParams, block_table, cache_seqlens, ref_counts):
    i32 = _dtypes()[0]
    if _bad(block_table, i32, (p.batch, p.max_pages_per_seq)):
        _refuse(call + ": block_table")
    if _bad(cache_seqlens, i32, (p.batch,)):
        _refuse(call + ": cache_seqlens")
    if _bad(ref_counts, i32, (p.num_pages,)):
        _refuse(call + ": ref_counts")


def _expect_workspace(call: str, p: MlaPoolParams, workspace, forks: int = 0):
    if workspace is None or workspace.numel() * workspace.element_size() < mla_pool_workspace_size(p, forks):
        _refuse(call + ": workspace", MLA_ERR_WORKSPACE)


def _list_of(call: str, name: str, t) -> int:
    """Length of a one-dimensional int32 list."""
    if t is None or t.dim() != 1 or _bad(t, _dtypes()[0], t.shape):
        _refuse(f"{call}: {name}")
    return t.numel()


def mla_copy_pages(p: MlaPoolParams, kv_pages, src_pages, dst_pages, stream=None):
    """Page dst_pages[i] := page src_pages[i] in every layer (int32 [n])."""
    n = _list_of("mla_copy_pages", "src_pages", src_pages)
    if _bad(dst_pages, _dtypes()[0], (n,)):
        _refuse("mla_copy_pages: dst_pages")
    _expect_pool("mla_copy_pages", kv_pages, p, p.num_layers, p.layer_stride)
    if n == 0:
        return
    _expect_device("mla_copy_pages", kv_pages, src_pages, dst_pages)
    _check(load_library().mla_copy_pages(ctypes.byref(p), kv_pages.data_ptr(), src_pages.data_ptr(), dst_pages.data_ptr(), n,
                                         _stream(stream)), "mla_copy_pages")


def mla_fork_sequences(p: MlaPoolParams, kv_pages, parents, children, block_table, cache_seqlens, ref_counts, new_pages,
                       workspace, stream=None):
    """Row children[i] of the table becomes a copy of row parents[i]; new_pages int32 [n] takes the outcomes."""
    _expect_workspace("mla_fork_sequences", p, workspace, 0 if parents is None else parents.numel())
    _fork(p, kv_pages, parents, children, block_table, cache_seqlens, ref_counts, new_pages, workspace, stream)


def _fork(p, kv_pages, parents, children, block_table, cache_seqlens, ref_counts, new_pages, workspace, stream):
    n = _list_of("mla_fork_sequences", "parents", parents)
    i32 = _dtypes()[0]
    if _bad(children, i32, (n,)):
        _refuse("mla_fork_sequences: children")
    if _bad(new_pages, i32, (n,)):
        _refuse("mla_fork_sequences: new_pages")
    _expect_tables("mla_fork_sequences", p, block_table, cache_seqlens, ref_counts)
    _expect_pool("mla_fork_sequences", kv_pages, p, p.num_layers, p.layer_stride)
    if n == 0:
        return
    _expect_device("mla_fork_sequences", kv_pages, parents, children, block_table, cache_seqlens, ref_counts, new_pages,
                   workspace)
    _check(load_library().mla_fork_sequences(ctypes.byref(p), kv_pages.data_ptr(), parents.data_ptr(), children.data_ptr(), n,
                                             block_table.data_ptr(), cache_seqlens.data_ptr(), ref_counts.data_ptr(),
                                             new_pages.data_ptr(), _ptr(workspace), _stream(stream)),
           "mla_fork_sequences")


def mla_reserve_pages(p: MlaPoolParams, num_new, block_table, cache_seqlens, ref_counts, served, workspace, stream=None):
    """Room for num_new[b] more rows of every sequence; served int32 [batch] takes the outcomes."""
    _expect_workspace("mla_reserve_pages", p, workspace)
    _reserve(p, num_new, block_table, cache_seqlens, ref_counts, served, workspace, stream)


def _reserve(p, num_new, block_table, cache_seqlens, ref_counts, served, workspace, stream):
    i32 = _dtypes()[0]
    if _bad(num_new, i32, (p.batch,)):
        _refuse("mla_reserve_pages: num_new")
    if _bad(served, i32, (p.batch,)):
        _refuse("mla_reserve_pages: served")
    _expect_tables("mla_reserve_pages", p, block_table, cache_seqlens, ref_counts)
    _expect_device("mla_reserve_pages", num_new, block_table, cache_seqlens, ref_counts, served, workspace)
    _check(load_library().mla_reserve_pages(ctypes.byref(p), num_new.data_ptr(), block_table.data_ptr(), cache_seqlens.data_ptr(),
                                            ref_counts.data_ptr(), served.data_ptr(), _ptr(workspace), _stream(stream)),
           "mla_reserve_pages")


def mla_free_sequences(p: MlaPoolParams, sequences, block_table, cache_seqlens, ref_counts, stream=None):
    """Ends the sequences (int32 [n], rows of the block table) and gives their pages back."""
    n = _list_of("mla_free_sequences", "sequences", sequences)
    _expect_tables("mla_free_sequences", p, block_table, cache_seqlens, ref_counts)
    if n == 0:
        return
    _expect_device("mla_free_sequences", sequences, block_table, cache_seqlens, ref_counts)
    _check(load_library().mla_free_sequences(ctypes.byref(p), sequences.data_ptr(), n, block_table.data_ptr(),
                                             cache_seqlens.data_ptr(), ref_counts.data_ptr(), _stream(stream)),
           "mla_free_sequences")


def mla_compact_pages(p: MlaPoolParams, kv_pages, block_table, cache_seqlens, ref_counts, num_used, workspace,
                      stream=None):
    """Draws the used pages together at the start of the pools; num_used int32 [1] takes their number."""
    _expect_workspace("mla_compact_pages", p, workspace)
    _compact(p, kv_pages, block_table, cache_seqlens, ref_counts, num_used, workspace, stream)


def _compact(p, kv_pages, block_table, cache_seqlens, ref_counts, num_used, workspace, stream):
    if _bad(num_used, _dtypes()[0], (1,)):
        _refuse("mla_compact_pages: num_used")
    _expect_tables("mla_compact_pages", p, block_table, cache_seqlens, ref_counts)
    _expect_pool("mla_compact_pages", kv_pages, p, p.num_layers, p.layer_stride)
    _expect_device("mla_compact_pages", kv_pages, block_table, cache_seqlens, ref_counts, num_used, workspace)
    _check(load_library().mla_compact_pages(ctypes.byref(p), kv_pages.data_ptr(), block_table.data_ptr(), cache_seqlens.data_ptr(),
                                            ref_counts.data_ptr(), num_used.data_ptr(), _ptr(workspace), _stream(stream)),
           "mla_compact_pages")


def mla_device_error(clear: bool = True) -> int:
    w = ctypes.c_int32()
    _check(load_library().mla_device_error(ctypes.byref(w), int(clear)), "mla_device_error")
    return w.value


def mla_wait_selftest(timeout_us: int, stream=None):
    _check(load_library().mla_wait_selftest(int(timeout_us), _stream(stream)), "mla_wait_selftest")


class Decoder:
    """Convenience wrapper: owns the scheduler-metadata and workspace buffers
    (allocated once through torch) for one problem shape."""

    def __init__(self, p: MlaDecodeParams, device=None):
        import torch
        self.p = p
        self.device = torch.device("cuda" if device is None else device)
        sb, wb = mla_get_workspace_size(p)
        self.num_units = mla_resolve_num_units(p)
        self.sched = torch.empty(sb // 4, dtype=torch.int32, device=self.device)
        self.workspace = torch.empty(max(wb, 256) // 4, dtype=torch.float32, device=self.device)

    def plan(self, cache_seqlens, stream=None):
        mla_get_scheduler_metadata(self.p, cache_seqlens, self.sched, stream)

    def new_outputs(self):
        import torch
        p = self.p
        dt = torch.float32 if p.out_dtype == MLA_OUT_F32 else torch.bfloat16
        out = torch.empty((p.batch, p.s_q, p.num_heads, 512), dtype=dt, device=self.device)
        lse = torch.empty((p.batch, p.s_q, p.num_heads), dtype=torch.float32, device=self.device)
        return out, lse

    def decode(self, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens, scale, out=None, lse=None,
               stream=None):
        if out is None or lse is None:
            out, lse = self.new_outputs()
        mla_decode(self.p, q_nope_absorbed, q_rope, kv_pages, block_table, cache_seqlens, scale, out, lse,
                   self.sched, self.workspace, stream)
        return out, lse


def _new(like, stream, shape=None, dtype=None):
    """A result that `stream` writes, of this tensor's shape and type or those given: its memory comes from that
    stream's pool, not from what the current stream has let go of but may still be using."""
    import torch
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream), device=like.device)
        with torch.cuda.stream(stream):
            return _new(like, None, shape, dtype)
    return torch.empty_like(like) if shape is None else like.new_empty(shape, dtype=dtype)  # (1.3 against 2.6 us)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


_idle_streams = {}


def _idle_stream(index: int):
    """A stream of the library's own (torch's are shared out in turn) on which nothing is ever launched."""
    import torch
    with _lock:
        if index not in _idle_streams:
            handle = ctypes.c_void_p()
            torch.cuda.check_error(int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle))))
            _idle_streams[index] = torch.cuda.ExternalStream(handle.value, device=index)
        return _idle_streams[index]


class _Owner:
    """Buffers that a wrapper's calls use on any stream, in any order.

    torch gives memory that was freed on a stream back to allocations on that stream at once, while its kernels may
    still use it; an allocation for use on another stream must not get such memory.  So the buffers are allocated
    for a stream that runs nothing: all that comes from there was a wrapper's before, and a wrapper's buffers
    are free again only when the streams that it was called on (record_stream) have come to where it was
    dropped.  Streams that torch does not own may be gone by then, and are not waited for: a wrapper used on one is
    kept until its work there is done."""

    def _own(self, *sizes_and_types):
        import torch
        new = lambda: [torch.empty(n, dtype=t, device=self.device) for n, t in sizes_and_types]  # noqa: E731
        self._streams = set()
        if self.device.type != "cuda" or torch.cuda.is_current_stream_capturing():  # (the graph's own memory)
            self._buffers = new()
        else:
            index = self.device.index
            with torch.cuda.stream(_idle_stream(torch.cuda.current_device() if index is None else index)):
                self._buffers = new()
        return self._buffers

    def _on(self, stream) -> int:
        """The handle of the stream of a call, which the buffers are kept for."""
        handle = _stream(stream)
        if handle not in self._streams:
            self._keep_for(stream, handle)
        return handle

    def _keep_for(self, stream, handle):
        import torch
        if self.device.type != "cuda":
            return
        if stream is None:
            stream = torch.cuda.current_stream()
        elif handle == 0:
            stream = torch.cuda.default_stream()
        if isinstance(stream, torch.cuda.Stream) and (handle == 0 or stream.stream_id != handle):  # (not an external one)
            with torch.cuda.stream(stream):
                if torch.cuda.is_current_stream_capturing():
                    return  # (a graph's user keeps the wrapper)
            for t in self._buffers:
                t.record_stream(stream)
        self._streams.add(handle)


class ChunkAttention(_Owner):
    """Convenience wrapper of the chunk attention: owns the plan and the workspace of one problem shape, and a copy of
    its params (`p` reads as a copy too; other params may be set where the buffers hold them)."""

    def __init__(self, p: MlaChunkParams, device=None):
        import torch
        self._p = type(p).from_buffer_copy(p)
        self.device = torch.device("cuda" if device is None else device)
        sb, wb = mla_chunk_workspace_size(self._p)
        self.sched, self.workspace = self._own((sb // 4, torch.int32), (wb, torch.uint8))
        self.seqlens = None

    @property
    def p(self) -> MlaChunkParams:
        return type(self._p).from_buffer_copy(self._p)

    @p.setter
    def p(self, p: MlaChunkParams):
        sb, wb = mla_chunk_workspace_size(p)
        if sb > _nbytes(self.sched) or wb > _nbytes(self.workspace):
            _refuse("ChunkAttention.p: larger than what the wrapper was made for", MLA_ERR_WORKSPACE)
        self._p = type(p).from_buffer_copy(p)

    def plan(self, cu_seqlens, cache_seqlens, stream=None):
        """The plan of a step's lengths; the tensors are read again by attend()."""
        mla_chunk_schedule(self._p, cu_seqlens, cache_seqlens, self.sched, self._on(stream))
        self.seqlens = cache_seqlens

    def attend(self, q_nope_absorbed, q_rope, kv_pages, block_table, scale, out=None, lse=None, stream=None):
        if self.seqlens is None:
            _refuse("ChunkAttention.attend before plan", MLA_ERR_WORKSPACE)
        if out is None:
            out = _new(q_nope_absorbed, stream)
        if lse is None:
            lse = _new(q_nope_absorbed, stream, q_nope_absorbed.shape[:2], _dtypes()[1])
        _attend(self._p, q_nope_absorbed, q_rope, kv_pages, block_table, self.seqlens, scale, out, lse, self.sched,
                self.workspace, self._on(stream))
        return out, lse


class PagePool(_Owner):
    """Convenience wrapper of the page upkeep: owns the workspace of one pool shape, for calls that fork at most
    max_forks sequences, and a copy of its params (`p` reads as a copy too; other params may be set where the
    workspace holds them).  The tables belong to the caller."""

    def __init__(self, p: MlaPoolParams, max_forks: int = 1024, device=None):
        import torch
        self._p = type(p).from_buffer_copy(p)
        self.device = torch.device("cuda" if device is None else device)
        self._max_forks = int(max_forks)
        self.workspace, = self._own((mla_pool_workspace_size(self._p, self._max_forks), torch.uint8))

    @property
    def p(self) -> MlaPoolParams:
        return type(self._p).from_buffer_copy(self._p)

    @p.setter
    def p(self, p: MlaPoolParams):
        if mla_pool_workspace_size(p, self._max_forks) > _nbytes(self.workspace):
            _refuse("PagePool.p: larger than what the wrapper was made for", MLA_ERR_WORKSPACE)
        self._p = type(p).from_buffer_copy(p)

    @property
    def max_forks(self) -> int:
        return self._max_forks

    def new_tables(self):
        """An empty pool's (block_table, cache_seqlens, ref_counts)."""
        import torch
        p, kw = self._p, dict(dtype=torch.int32, device=self.device)
        return (torch.full((p.batch, p.max_pages_per_seq), -1, **kw), torch.zeros(p.batch, **kw),
                torch.zeros(p.num_pages, **kw))

    def copy(self, kv_pages, src_pages, dst_pages, stream=None):
        mla_copy_pages(self._p, kv_pages, src_pages, dst_pages, stream)

    def fork(self, kv_pages, parents, children, block_table, cache_seqlens, ref_counts, stream=None):
        """Returns new_pages int32 [n]: the child's own page, -1 (none needed), -2 (refused), -3 (no page left)."""
        if parents.numel() > self._max_forks:
            _refuse("PagePool.fork: more forks than max_forks", MLA_ERR_WORKSPACE)
        new_pages = _new(parents, stream)
        _fork(self._p, kv_pages, parents, children, block_table, cache_seqlens, ref_counts, new_pages, self.workspace,
              self._on(stream))
        return new_pages

    def reserve(self, num_new, block_table, cache_seqlens, ref_counts, stream=None):
        """Returns served int32 [batch]: 1 (done), 0 (not enough pages), -2 (refused)."""
        served = _new(num_new, stream)
        _reserve(self._p, num_new, block_table, cache_seqlens, ref_counts, served, self.workspace, self._on(stream))
        return served

    def free(self, sequences, block_table, cache_seqlens, ref_counts, stream=None):
        mla_free_sequences(self._p, sequences, block_table, cache_seqlens, ref_counts, stream)

    def compact(self, kv_pages, block_table, cache_seqlens, ref_counts, stream=None):
        """Returns the number of used pages, int32 [1] on the device."""
        used = _new(cache_seqlens, stream, (1,))
        _compact(self._p, kv_pages, block_table, cache_seqlens, ref_counts, used, self.workspace, self._on(stream))
        return used
