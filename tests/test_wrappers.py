"""ChunkAttention and PagePool own what they were made with: params changed afterwards, by the caller or through the
wrapper, never reach a kernel with buffers that are too small for them."""
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
    attn.plan(None, x)
    attn.attend(x, None, None, None, 1.0)
    larger.plan(None, x)
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
    pool.fork(None, ids, ids, None, lens, None)
    pool.reserve(lens, None, lens, None)
    pool.compact(None, None, lens, None)
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
