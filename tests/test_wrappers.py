"""ChunkAttention and PagePool own what they were made with: params changed afterwards, by the caller or through the
wrapper, never reach a kernel with buffers that are too small for them; and the buffers are no one else's on any
stream, neither when a wrapper is made nor when it is dropped."""
import numpy as np
import pytest

from mla_absorbed_decode_02_gb300 import _lib
from mla_absorbed_decode_02_gb300._lib import MlaChunkParams, MlaError, MlaPoolParams
from mla_absorbed_decode_02_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return _lib.load_library()


def _chunk(**kw):
    base = dict(batch=2, max_tokens=8, num_heads=16, num_pages=300, max_pages_per_seq=150, kv_dtype=_lib.MLA_KV_FP8_E4M3,
                max_kv_tokens=6400, num_units=4)
    base.update(kw)
    return MlaChunkParams.make(**base)


def test_params_changed_after_a_chunk_wrapper_was_made(monkeypatch):
    p = _chunk()
    attn = _lib.ChunkAttention(p, device="cpu")
    room = attn.workspace.numel()
    used = []
    monkeypatch.setattr(_lib, "mla_chunk_schedule", lambda p, *a: used.append(p.max_kv_tokens))
    monkeypatch.setattr(_lib, "_attend", lambda p, *a: used.append(p.max_kv_tokens))
    p.max_kv_tokens = 12800                       # the caller's own, for a wrapper to come
    larger = _lib.ChunkAttention(p, device="cpu")
    attn.p.max_kv_tokens = 12800                  # a copy's
    assert attn.p.max_kv_tokens == 6400 and larger.p.max_kv_tokens == 12800
    import torch
    x = torch.zeros(8, 16, 512, dtype=torch.bfloat16)
    attn.plan(None, x, stream=0)
    attn.attend(x, None, None, None, 1.0, out=x, lse=x, stream=0)
    larger.plan(None, x, stream=0)
    assert used == [6400, 6400, 12800]
    with pytest.raises(MlaError) as e:
        attn.p = p
    assert e.value.status == _lib.MLA_ERR_WORKSPACE
    with pytest.raises(MlaError) as e:
        attn.p = _chunk(max_tokens=80)            # the plan's buffer
    assert e.value.status == _lib.MLA_ERR_WORKSPACE
    attn.p = _chunk(causal=False)                 # what the buffers hold may be set
    assert attn.p.causal == 0 and _lib.mla_chunk_workspace_size(attn.p)[1] == room == attn.workspace.numel()


def test_params_changed_after_a_pool_wrapper_was_made(monkeypatch):
    p = MlaPoolParams.make(batch=4, num_pages=100, max_pages_per_seq=8)
    pool = _lib.PagePool(p, max_forks=8, device="cpu")
    used = []
    for name in ("_fork", "_reserve", "_compact"):
        monkeypatch.setattr(_lib, name, lambda p, *a: used.append((p.num_pages, p.batch)))
    p.num_pages, p.batch = 10000, 4000
    pool.p.num_pages = 10000
    import torch
    ids, lens = torch.zeros(8, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    monkeypatch.setattr(_lib, "_new", lambda like, *a: like)
    pool.fork(None, ids, ids, None, lens, None, stream=0)
    pool.reserve(lens, None, lens, None, stream=0)
    pool.compact(None, None, lens, None, stream=0)
    assert used == [(100, 4)] * 3
    bt, L, ref = pool.new_tables()
    assert bt.shape == (4, 8) and L.shape == (4,) and ref.shape == (100,)
    with pytest.raises(MlaError) as e:
        pool.p = p
    assert e.value.status == _lib.MLA_ERR_WORKSPACE
    with pytest.raises(AttributeError):
        pool.max_forks = 5000
    pool.p = MlaPoolParams.make(batch=4, num_pages=90, max_pages_per_seq=8)
    assert pool.p.num_pages == 90


@pytest.mark.gpu
def test_a_wrapper_refuses_what_its_workspace_does_not_hold():
    """Lengths that only the params of a later, larger wrapper have room for: the first wrapper's plan refuses them
    and its attention writes nothing."""
    import torch
    p = _chunk()
    attn = _lib.ChunkAttention(p)
    p.max_kv_tokens = 12800
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    lens = torch.tensor([64 * 100, 64 * 50], dtype=torch.int32, device="cuda")
    bt = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150)
    pool = torch.zeros(300, 64, 656, dtype=torch.uint8, device="cuda")
    q, qr = torch.zeros(8, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 16, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((8, 16), 7.0, device="cuda")
    attn.plan(cu, lens)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_INVALID_ARG
    attn.attend(q, qr, pool, bt, 0.07, out=out, lse=lse)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_WORKSPACE
    assert (out == 7).all() and (lse == 7).all()
    larger = _lib.ChunkAttention(p)
    larger.plan(cu, lens)
    larger.attend(q, qr, pool, bt, 0.07, out=out, lse=lse)
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    assert (out == 0).all() and np.allclose(lse[7, 0].item(), np.log(64 * 50), atol=1e-5)


# ------------------------------------------------------------------ buffers and streams (GPU)
def _apart(a, b):
    """No byte of a in b: tensors, or (address, bytes)."""
    (p, m), (q, n) = ((x if isinstance(x, tuple) else (x.data_ptr(), x.numel() * x.element_size())) for x in (a, b))
    return p + m <= q or q + n <= p


def _pool_of(pages):
    p = MlaPoolParams.make(8, pages, 4)
    up = _lib.PagePool(p)
    return up, up.new_tables()


def _on(kind, side):
    """How a call is put on a stream: keyword and context."""
    import contextlib

    import torch
    if kind == "current":
        return {}, torch.cuda.stream(side)
    return {"stream": side if kind == "stream" else side.cuda_stream}, contextlib.nullcontext()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["stream", "pointer", "current"])
@pytest.mark.parametrize("pages", [64, 400000])
def test_a_new_wrapper_takes_no_memory_in_use(kind, pages):
    """Memory that the current stream has let go of, but that kernels queued on it still read, does not become the
    workspace of a wrapper that is then used on another stream."""
    import torch
    up, tables = _pool_of(pages)
    new = torch.full((8,), 3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    up.reserve(new, *tables)                     # loads the kernel
    n = up.workspace.numel() // 4
    x = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)              # about a tenth of a second
    y = x * 2
    where = (x.data_ptr(), 4 * n)
    del x                                       # free to the current stream, after y
    other = _lib.PagePool(up.p)
    assert _apart(other.workspace, where)
    kw, on = _on(kind, side)
    with on:
        served = other.reserve(new, *tables, **kw)
    torch.cuda.synchronize()
    assert (y == 10).all() and (served == 1).all() and (tables[1] == 6).all()
    assert _lib.mla_device_error(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["stream", "current"])
def test_a_dropped_wrappers_memory_waits_for_its_streams(kind):
    """The buffers of a wrapper that was dropped while another stream still runs on them go neither to a new wrapper
    nor to a tensor."""
    import torch
    up, tables = _pool_of(300000)
    new = torch.full((8,), 3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    up.reserve(new, *tables)
    torch.cuda.synchronize()
    kw, on = _on(kind, side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    with on:
        served = up.reserve(new, *tables, **kw)
    was, size, p = up.workspace.data_ptr(), up.workspace.numel(), up.p
    del up
    fresh = _lib.PagePool(p)
    assert _apart(fresh.workspace, (was, size))
    with torch.cuda.stream(side):
        tensor = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert _apart(tensor, (was, size))
    fresh.workspace.fill_(255)
    torch.cuda.synchronize()
    assert (served == 1).all() and (tables[1] == 6).all()
    assert _lib.mla_device_error(clear=True) == 0


@pytest.mark.gpu
def test_chunk_wrapper_made_beside_work_in_flight():
    """The same bits from a wrapper made and used on another stream while the current one is busy, and dropped there."""
    import torch
    from test_chunk import SCALE, Problem
    q = Problem([3, 20, 1], [400, 1500, 64], 16, "fp8", seed=31, num_units=30)
    want, want_lse = q.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    outs = []
    for _ in range(3):
        attn = _lib.ChunkAttention(q.p)
        attn.plan(q.d_cu, q.d_L, stream=side)
        outs.append(attn.attend(q.d_q, q.d_qr, q.pool, q.d_bt, SCALE, stream=side))
        del attn
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    for out, lse in outs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("as_pointer", [False, True])
def test_a_stream_that_is_gone_before_the_wrapper(as_pointer):
    """A wrapper called on a stream that torch does not own may be dropped after that stream."""
    import ctypes

    import torch
    up, tables = _pool_of(300000)
    new = torch.full((8,), 3, dtype=torch.int32, device="cuda")
    handle = ctypes.c_void_p()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle))) == 0
    torch.cuda.synchronize()
    served = up.reserve(new, *tables, stream=handle.value if as_pointer else torch.cuda.ExternalStream(handle.value))
    torch.cuda.synchronize()
    assert int(torch.cuda.cudart().cudaStreamDestroy(handle.value)) == 0
    p = up.p
    del up
    again = _lib.PagePool(p)
    assert (again.reserve(new, *tables) == 1).all() and (served == 1).all() and (tables[1] == 6).all()
    assert _lib.mla_device_error(clear=True) == 0
