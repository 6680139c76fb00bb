"""Attention of ragged chunks of new tokens over the paged cache (mla_chunk_*): the planner and the
refusals on the CPU, the kernels against the definition in float64 on the GPU.

Tolerances.  Against float64 on the same bf16 inputs (FP8 rows: bf16(code x scale), what they stand
for), with w = softmax weights and A = sum_j w_j |c_j|:
  * a score is a float32 sum of 576 exact products; each partial sum is off by at most 2^-23 of its
    size, so |score error| <= d = scale * 576 * 2^-23 * max_j sum_i |q_i k_ji|;
  * lse moves by at most d, plus 2^-20 (the last logarithm, products and the approximate exponentials
    within their stated 2 ulp) and 2^-23 of its size;
  * each weight is off by at most 2 d (numerator and sum), and by 2^-8 (P in bf16); the output is
    rounded to bf16, 2^-8 of its size at most: |out error| <= 2^-8 |out| + (2^-8 + 2 d + 2^-14) A,
    2^-14 covering float32 accumulation, rescaling and division over at most 2^9 tiles."""
import math

import numpy as np
import pytest

import mla_workloads as mw
from mla_absorbed_decode_02_gb300 import _lib
from mla_absorbed_decode_02_gb300._lib import MlaChunkParams, MlaError
from mla_absorbed_decode_02_gb300.build import build

SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------ planner and refusals (CPU)
@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return _lib.load_library()


def _params(**kw):
    base = dict(batch=3, max_tokens=40, num_heads=16, num_pages=64, max_pages_per_seq=32, num_units=5)
    base.update(kw)
    return MlaChunkParams.make(**base)


def _parse(sched, U):
    cap = sched[2]
    units = sched[16:16 + 16 * U].reshape(U, 16)
    blocks = sched[16 + 16 * U:16 + 16 * U + 8 * cap].reshape(cap, 8)[:sched[3]]
    return units, blocks, sched[16 + 16 * U + 8 * cap:][:8 * sched[7]].reshape(-1, 8)


@pytest.mark.parametrize("H", [1, 7, 16, 64, 96, 128])
@pytest.mark.parametrize("U", [1, 3, 76])
@pytest.mark.parametrize("seed", range(6))
def test_plan_covers_every_tile_once(H, U, seed):
    rng = np.random.default_rng([seed, H, U])
    B = int(rng.integers(1, 20))
    n = rng.integers(0, 40, B) * (rng.random(B) < 0.8)
    L = np.where(rng.random(B) < 0.15, rng.integers(0, 5, B), n + rng.integers(0, 6000, B))
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1]) + int(rng.integers(1, 9))
    p = _params(batch=B, max_tokens=T, num_heads=H, num_units=U, max_pages_per_seq=100)
    sched = _lib.mla_chunk_plan_host(p, U, cu, L)
    tb = max(1, 128 // H)
    assert sched[0] == 0x4D4C4143 and sched[1] == U and sched[6] == tb
    units, blocks, split = _parse(sched, U)
    # every new token in one block, blocks within a sequence; the longest sequences first where they are sorted
    assert sum(b[1] for b in blocks) == cu[-1]
    if len(blocks) > U and sched[9] != 2:
        order = [(-(-(-ln // 256)), seq, tok0) for tok0, _, seq, _, ln, *_ in blocks.tolist()]
        assert order == sorted(order)
    at = 0
    for tok0, ntok, seq, base, ln, nt, splits, off in sorted(blocks.tolist()):
        assert tok0 == at and 1 <= ntok <= tb and cu[seq] <= tok0 and tok0 + ntok <= cu[seq + 1]
        assert ln == L[seq] and base == L[seq] - n[seq] + (tok0 - cu[seq]) + 1
        vis = min(max(base + ntok - 1, 0), ln)
        assert nt == max(1, -(-vis // 256))
        at += ntok
    # units take disjoint stretches that cover all tiles; splits are counted in order
    seen, owner = {k: [] for k in range(len(blocks))}, {}
    for u, rec in enumerate(units):
        if rec[0] < 0:
            continue
        assert np.array_equal(rec[8:], blocks[rec[0]])
        for k in range(rec[0], rec[2] + 1):
            t0 = rec[1] if k == rec[0] else 0
            t1 = rec[3] if k == rec[2] else blocks[k][5]
            assert t0 < t1
            seen[k].append((t0, t1, rec[4] if k == rec[0] else 0))
            owner[k] = u
    slots = 0
    for k, parts in seen.items():
        assert [t for a, b, _ in parts for t in range(a, b)] == list(range(blocks[k][5]))
        assert [s for _, _, s in parts] == list(range(len(parts))) and blocks[k][6] == len(parts)
        if len(parts) > 1:
            assert blocks[k][7] == slots and any(np.array_equal(r, blocks[k]) for r in split)
            slots += len(parts)
    if sched[9] == 2:
        assert slots == 0 and sched[5] == max(sum(3 + 4 * (t1 - t0) for k in seen for t0, t1, _ in seen[k] if owner[k] == u) for u in range(U))
    assert sched[4] == slots <= 2 * max(U - 1, 0) and len(split) == sum(len(v) > 1 for v in seen.values())
    assert sched[8] == sum(-(-int(x) // 64) for x, m in zip(L, n) if m > 0)


def test_plans_of_each_kind():
    """Shares or whole blocks where there are no more blocks than units, blocks dealt in rounds where that costs at
    most 5/4 of stretches (11/10 where the rows fit the L2), stretches else and with more sequences than are sorted."""
    def kind(n, L, H, U):
        cu = np.concatenate([[0], np.cumsum(n)])
        p = _params(batch=len(n), max_tokens=int(cu[-1]), num_heads=H, num_units=U, max_pages_per_seq=200)
        return _lib.mla_chunk_plan_host(p, U, cu, L)[9]
    assert kind([4], [4000], 16, 8) == 1
    assert kind([12] * 24, [8192] * 24, 128, 76) == 2        # 288 blocks: four rounds
    assert kind([4] * 24, [8192] * 24, 128, 76) == 0         # 96 blocks: the second round would be a quarter full
    assert kind([9] * 20, [8192] * 20, 128, 76) == 2         # 1.22 of the stretches, 2560 pages
    assert kind([9] * 20, [2048] * 20, 128, 76) == 0         # 1.12, 640 pages
    assert kind([1] * 1024, [900] * 1024, 128, 76) == 2
    assert kind([1] * 1025, [900] * 1025, 128, 76) == 0
    assert kind([2] * 5, [12000, 300, 300, 300, 300], 128, 8) == 0   # one sequence far longer than the rest


@pytest.mark.parametrize("cu,lens,kw", [
    ([1, 2, 3, 4], [9, 9, 9], {}),                    # does not start at 0
    ([0, 3, 2, 4], [9, 9, 9], {}),                    # decreases
    ([0, 3, 5, 41], [9, 9, 64], {}),                  # past the buffer
    ([0, 1, 2, 3], [9, -1, 9], {}),                   # negative length
    ([0, 1, 2, 3], [9, 9, 32 * 64 + 1], {}),          # past the block table
    ([0, 1, 2, 3], [200, 64, 9], dict(kv_dtype=_lib.MLA_KV_FP8_E4M3, max_kv_tokens=5 * 64)),  # 4 + 1 + 1 pages
])
def test_plan_refuses_lengths(cu, lens, kw):
    with pytest.raises(MlaError) as e:
        _lib.mla_chunk_plan_host(_params(**kw), 5, cu, lens)
    assert e.value.status == _lib.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), _lib.MLA_ERR_INVALID_ARG), (dict(max_tokens=0), _lib.MLA_ERR_INVALID_ARG),
    (dict(num_heads=0), _lib.MLA_ERR_INVALID_ARG), (dict(num_heads=129), _lib.MLA_ERR_UNSUPPORTED),
    (dict(num_pages=0), _lib.MLA_ERR_INVALID_ARG), (dict(page_size=32), _lib.MLA_ERR_UNSUPPORTED),
    (dict(kv_dtype=3), _lib.MLA_ERR_INVALID_ARG), (dict(num_units=-1), _lib.MLA_ERR_INVALID_ARG),
    (dict(kv_dtype=_lib.MLA_KV_FP8_E4M3), _lib.MLA_ERR_INVALID_ARG),   # no room for the expanded rows
    (dict(max_tokens=1 << 25, num_heads=128), _lib.MLA_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 26), _lib.MLA_ERR_UNSUPPORTED), (dict(timeout_us=-1), _lib.MLA_ERR_INVALID_ARG),
])
def test_bad_params(kw, status):
    with pytest.raises(MlaError) as e:
        _lib.mla_chunk_workspace_size(_params(**kw))
    assert e.value.status == status
    p = _params()
    p.reserved[1] = 1
    with pytest.raises(MlaError):
        _lib.mla_chunk_workspace_size(p)


def test_workspace_does_not_grow_with_the_tokens():
    sb, wb = _lib.mla_chunk_workspace_size(_params(num_units=76, max_tokens=8192, num_heads=128))
    assert wb == 2 * 76 * 128 * 513 * 4
    assert sb == 4 * (16 + 16 * 76 + 8 * 8192 + 8 * 76 + 4 + 4 + 8192)
    _, wf = _lib.mla_chunk_workspace_size(_params(num_units=76, kv_dtype=_lib.MLA_KV_FP8_E4M3, max_kv_tokens=1000))
    assert wf == wb + 15 * 64 * 1152


def test_attend_refuses_bad_arguments():
    """Types, shapes and sizes in the binding: nothing is launched.  (Tensors of the host are themselves refused,
    last of all.)"""
    import torch
    p = _params(batch=1, max_tokens=4, num_heads=2, num_pages=2, max_pages_per_seq=2)
    sb, wb = _lib.mla_chunk_workspace_size(p)
    good = dict(q_nope_absorbed=torch.zeros(4, 2, 512, dtype=torch.bfloat16), q_rope=torch.zeros(4, 2, 64, dtype=torch.bfloat16),
                kv_pages=torch.zeros(2, 64, 576, dtype=torch.bfloat16), block_table=torch.zeros(1, 2, dtype=torch.int32),
                cache_seqlens=torch.zeros(1, dtype=torch.int32), scale=SCALE, out=torch.zeros(4, 2, 512, dtype=torch.bfloat16),
                lse=torch.zeros(4, 2), sched=torch.zeros(sb // 4, dtype=torch.int32), workspace=torch.zeros(wb, dtype=torch.uint8))
    bad = [(dict(q_nope_absorbed=good["q_nope_absorbed"].float()), "q_nope_absorbed"), (dict(q_nope_absorbed=good["q_nope_absorbed"][:3]), "q_nope_absorbed"),
           (dict(q_rope=good["q_rope"].transpose(0, 1)), "q_rope"), (dict(kv_pages=good["kv_pages"][:1]), "kv_pages"), (dict(out=good["out"].float()), "out"),
           (dict(lse=good["lse"].T), "lse"), (dict(block_table=good["block_table"].long()), "block_table"),
           (dict(cache_seqlens=torch.zeros(2, dtype=torch.int32)), "cache_seqlens"), (dict(sched=None), "sched"), (dict(workspace=None), "workspace"),
           (dict(sched=good["sched"][1:]), "sched"), (dict(workspace=good["workspace"][1:]), "workspace"), (dict(out=None), "out"), ({}, "device")]
    for b, word in bad:
        with pytest.raises(MlaError, match=word) as e:
            _lib.mla_chunk_attend(p, **{**good, **b}, stream=0)
        assert e.value.status in (_lib.MLA_ERR_INVALID_ARG, _lib.MLA_ERR_WORKSPACE), b
    plan = dict(cu_seqlens=torch.zeros(2, dtype=torch.int32), cache_seqlens=good["cache_seqlens"], sched=good["sched"])
    for b, word in ((dict(cu_seqlens=None), "cu_seqlens"), (dict(cu_seqlens=torch.zeros(1, dtype=torch.int32)), "cu_seqlens"),
                    (dict(cache_seqlens=torch.zeros(1)), "cache_seqlens"), (dict(sched=good["sched"][1:]), "sched"), ({}, "device")):
        with pytest.raises(MlaError, match=word):
            _lib.mla_chunk_schedule(p, **{**plan, **b}, stream=0)


def test_library_refuses_bad_pointers_and_scales():
    """The C entries: null and misaligned pointers, a scale that is not positive and finite."""
    import ctypes
    lib, p = _lib.load_library(), _params(num_units=1)
    buf = ctypes.create_string_buffer(4096)
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    good = [base] * 5 + [SCALE] + [base] * 4 + [0]          # q, q_rope, kv, table, lens | out, lse, sched, workspace, stream
    for k in (0, 1, 2, 3, 4, 6, 7, 8, 9):
        for bad in (0, base + 2):
            args = list(good)
            args[k] = bad
            assert lib.mla_chunk_attend(ctypes.byref(p), *args) == _lib.MLA_ERR_INVALID_ARG, (k, bad)
    for scale in (0.0, -1.0, math.inf, math.nan):
        args = list(good)
        args[5] = scale
        assert lib.mla_chunk_attend(ctypes.byref(p), *args) == _lib.MLA_ERR_INVALID_ARG
    for k in range(3):
        args = [base, base, base, 0]
        args[k] = 0
        assert lib.mla_chunk_schedule(ctypes.byref(p), *args) == _lib.MLA_ERR_INVALID_ARG
    assert lib.mla_chunk_attend(None, *good) == _lib.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------ the kernels (GPU)
class Problem:
    """Seeded inputs on the host and on the GPU: n new tokens and length L for every sequence."""

    def __init__(self, n, L, H, kv="bf16", seed=0, pad=0, extra_pages=3, num_units=0, causal=True, at=None):
        import torch
        rng = np.random.default_rng(seed)
        self.n, self.L, self.H, self.kv, self.causal = np.asarray(n), np.asarray(L), H, kv, causal
        B, need = len(n), -(-self.L // 64)
        self.T = int(self.n.sum()) + pad
        P = int(need.sum()) + extra_pages
        self.pages = rng.permutation(P) if at is None else at + np.arange(P)
        P = P if at is None else at + P
        self.bt = np.full((B, max(1, int(need.max()))), -1, np.int32)
        o = 0
        for b, k in enumerate(need):
            self.bt[b, :k] = self.pages[o:o + k]
            o += k
        bits = lambda *s: mw.to_bf16_bits(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
        self.q, self.qr = bits(max(self.T, 1), H, 512), bits(max(self.T, 1), H, 64)
        self.rows = mw._fill_pool(rng, len(self.pages), kv)   # page self.pages[i] holds rows[i]
        if at is None:
            inv = np.empty(P, np.int64)
            inv[self.pages] = np.arange(P)
            pool = torch.from_numpy(self.rows[inv].view(np.int16 if kv == "bf16" else np.uint8)).cuda()
        else:  # the last pages of a pool that is otherwise never touched
            pool = torch.empty((P,) + self.rows.shape[1:], dtype=torch.int16 if kv == "bf16" else torch.uint8, device="cuda")
            pool[at:] = torch.from_numpy(self.rows.view(np.int16 if kv == "bf16" else np.uint8)).cuda()
        self.pool = pool.view(torch.bfloat16) if kv == "bf16" else pool
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.d_q, self.d_qr = dev(self.q.view(np.int16)).view(torch.bfloat16), dev(self.qr.view(np.int16)).view(torch.bfloat16)
        self.d_cu, self.d_L, self.d_bt = dev(self.cu), dev(self.L.astype(np.int32)), dev(self.bt)
        self.p = MlaChunkParams.make(B, max(self.T, 1), H, P, self.bt.shape[1], causal=causal,
                                     kv_dtype=_lib.MLA_KV_FP8_E4M3 if kv == "fp8" else _lib.MLA_KV_BF16,
                                     max_kv_tokens=max(64, int(need.sum()) * 64), num_units=num_units)

    def latent(self, b):
        """Rows of sequence b in float64: latent and RoPE key."""
        o = int((-(-self.L[:b] // 64)).sum())
        rows = self.rows[o:o + -(-int(self.L[b]) // 64)].reshape(-1, self.rows.shape[-1])[:int(self.L[b])]
        if self.kv == "bf16":
            x = (rows.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
            return x[:, :512], x[:, 512:]
        import oracle
        lat, rope = oracle.fp8_rows_to_f64(rows)
        # the row stands for bf16(code * scale)
        return (mw.to_bf16_bits(lat.astype(np.float32)).astype(np.uint32) << 16).view(np.float32).astype(np.float64), rope

    def reference(self):
        """(out, lse, bound of |out error|, bound of |lse error|), float64."""
        H, T = self.H, int(self.n.sum())
        out, lse = np.zeros((T, H, 512)), np.full((T, H), -np.inf)
        tol_o, tol_l = np.zeros((T, H, 512)), np.zeros((T, H))
        wide = lambda x: (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
        for b in range(len(self.n)):
            c, k = self.latent(b)
            for i in range(int(self.n[b])):
                t = int(self.cu[b]) + i
                seen = max(0, int(self.L[b]) - (int(self.n[b]) - 1 - i if self.causal else 0))
                if seen == 0:
                    continue
                key, q = np.concatenate([c[:seen], k[:seen]], 1), np.concatenate([wide(self.q[t]), wide(self.qr[t])], 1)
                s = SCALE * (q @ key.T)
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(1, keepdims=True)
                w = e / z
                out[t], lse[t] = w @ c[:seen], (m + np.log(z))[:, 0]
                d = SCALE * 576 * 2.0 ** -23 * (np.abs(q) @ np.abs(key).T).max(1)
                tol_l[t] = d + 2.0 ** -20 + 2.0 ** -23 * np.abs(lse[t])
                tol_o[t] = 2.0 ** -8 * np.abs(out[t]) + (2.0 ** -8 + 2 * d[:, None] + 2.0 ** -14) * (w @ np.abs(c[:seen]))
        return out, lse, tol_o, tol_l

    def run(self, attn=None):
        import torch
        attn = attn or _lib.ChunkAttention(self.p)
        out = torch.full((max(self.T, 1), self.H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((max(self.T, 1), self.H), 7.0, device="cuda")
        attn.plan(self.d_cu, self.d_L)
        attn.attend(self.d_q, self.d_qr, self.pool, self.d_bt, SCALE, out=out, lse=lse)
        torch.cuda.synchronize()
        assert _lib.mla_device_error(clear=True) == 0
        return out, lse

    def check(self, attn=None):
        out, lse = self.run(attn)
        T = int(self.n.sum())
        assert (out[T:] == 7).all() and (lse[T:] == 7).all()     # rows behind the last sequence
        o, l = out[:T].double().cpu().numpy(), lse[:T].double().cpu().numpy()
        ref, rl, to, tl = self.reference()
        none = np.isneginf(rl)
        assert np.array_equal(none, np.isneginf(l)) and (o[none] == 0).all()
        assert (np.abs(o - ref) <= to).all(), float((np.abs(o - ref) - to).max())
        assert (np.abs(l[~none] - rl[~none]) <= tl[~none]).all(), float(np.abs(l[~none] - rl[~none]).max())
        return out, lse


RAGGED = [([1], [1]), ([3], [3]), ([5, 0, 2, 9], [5, 77, 2, 300]), ([2, 4, 1], [0, 2, 64]),
          ([1, 17, 8, 1], [256, 257, 513, 640]), ([33, 1], [1100, 191])]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [1, 7, 16, 40, 64, 96, 128])
@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_matches_float64(kv, H, case):
    n, L = RAGGED[case]
    Problem(n, L, H, kv, seed=17 * case + H, pad=case % 3).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,L,H,units,kind", [
    ([2, 2, 3], [300, 520, 700], 128, 2, 2),           # dealt: seven blocks in four rounds
    ([40, 3, 0, 17], [1000, 3, 0, 260], 16, 3, 2),
    ([1] * 11, list(range(0, 1100, 100)), 64, 4, 2),   # one without a key among them
    ([3], [2600], 128, 2, 0),                          # stretches: two rounds would leave a unit idle in the second
    ([1, 1, 1], [5000, 64, 70], 128, 2, 0),
    ([2], [700], 128, 5, 1),                           # shares
])
def test_each_kind_of_plan(kv, n, L, H, units, kind):
    q = Problem(n, L, H, kv, seed=40 + units, num_units=units, pad=1)
    attn = _lib.ChunkAttention(q.p)
    q.check(attn)
    assert int(attn.sched[9]) == kind


@pytest.mark.gpu
@pytest.mark.parametrize("units", [1, 2, 7, 76])
@pytest.mark.parametrize("H,kv", [(16, "bf16"), (128, "fp8")])
def test_units_share_and_split_the_work(units, H, kv):
    """One unit walks every piece; many units split the long sequence and are merged."""
    Problem([3, 1, 10], [700, 3000, 1290], H, kv, seed=units, num_units=units).check()


@pytest.mark.gpu
@pytest.mark.parametrize("units", [3, 9, 40, 76])
def test_the_same_bits_every_time(units):
    """Repeated calls with one plan give the same bits, whatever the plan splits; another plan moves them by no
    more than the rounding of the partials."""
    import torch
    q = Problem([40, 3, 1, 77], [1500, 9000, 12000, 2000], 40, seed=units, num_units=units)
    attn = _lib.ChunkAttention(q.p)
    attn.plan(q.d_cu, q.d_L)
    first = None
    for _ in range(6):
        out, lse = attn.attend(q.d_q, q.d_qr, q.pool, q.d_bt, SCALE)
        torch.cuda.synchronize()
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert _lib.mla_device_error(clear=True) == 0
    one = Problem([40, 3, 1, 77], [1500, 9000, 12000, 2000], 40, seed=units, num_units=1).run()
    assert (first[1] - one[1]).abs().max() <= 2e-6 * one[1].abs().max()
    assert (first[0].float() - one[0].float()).norm() <= 2.0 ** -8 * one[0].float().norm()


@pytest.mark.gpu
def test_without_the_causal_rule():
    Problem([4, 9], [130, 600], 16, seed=3, causal=False).check()


@pytest.mark.gpu
def test_no_new_token_at_all():
    Problem([0, 0], [10, 500], 16, pad=3).check()


@pytest.mark.gpu
def test_pages_past_four_gigabytes():
    """The last pages of a pool of 60,000 (4.4 GB): byte and element offsets past 2^31."""
    Problem([5], [1000], 16, seed=9, at=60000).check()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [8, 128])
@pytest.mark.parametrize("bits", [0x7FC0, 0x7F80, 0xFF80])
def test_rows_that_are_not_finite(H, bits):
    """NaN and infinities past the end reach nobody; in the row of new token 9 of 14 they reach the tokens
    that see it (9..13) and no others, though eight (or sixteen) tokens share a tile."""
    import torch
    n, L = 14, 333
    q = Problem([n], [L], H, seed=21)
    want, want_lse = q.run()
    at = q.pool.view(torch.int16).view(-1, 576)
    page = lambda row: int(q.bt[0, row // 64]) * 64 + row % 64  # noqa: E731
    for row in range(L, -(-L // 64) * 64):
        at[page(row)] = bits - 65536 if bits > 32767 else bits
    got, got_lse = q.run()
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    at[page(L - n + 9), 3:600:5] = bits - 65536 if bits > 32767 else bits
    got, got_lse = q.run()
    assert torch.equal(got[:9], want[:9]) and torch.equal(got_lse[:9], want_lse[:9])
    assert got[9:].isnan().all() and got_lse[9:].isnan().all()


@pytest.mark.gpu
def test_agrees_with_the_decode():
    """One new token a sequence: the decode's operation (its scores carry the exchange's rounding, at most
    2.8e-4 on lse at these inputs)."""
    import torch
    q = Problem([1] * 5, [1, 64, 300, 1000, 2000], 128, seed=5)
    out, lse = q.run()
    p = _lib.MlaDecodeParams.make(5, 1, 128, q.pool.shape[0], q.bt.shape[1])
    dec = _lib.Decoder(p)
    dec.plan(q.d_L)
    o2, l2 = dec.decode(q.d_q.view(5, 1, 128, 512), q.d_qr.view(5, 1, 128, 64), q.pool, q.d_bt, q.d_L, SCALE)
    torch.cuda.synchronize()
    assert (l2[:, 0] - lse).abs().max() <= 3e-4
    assert (o2[:, 0].float() - out.float()).norm() <= 5e-3 * out.float().norm()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_plan_on_the_device_is_the_host_plan(kv):
    import torch
    rng = np.random.default_rng(8)
    for B, H in ((1, 128), (40, 16), (1500, 7), (3000, 128), (30, 128), (40, 128), (300, 64), (1024, 128)):
        n = rng.integers(0, 6, B)
        L = n + rng.integers(0, 3000, B)
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        p = MlaChunkParams.make(B, int(cu[-1]) + 4, H, 16, 64, num_units=76, kv_dtype=1 if kv == "fp8" else 0,
                                max_kv_tokens=64 * 200000)
        sched = torch.zeros(_lib.mla_chunk_workspace_size(p)[0] // 4, dtype=torch.int32, device="cuda")
        _lib.mla_chunk_schedule(p, torch.from_numpy(cu).cuda(), torch.from_numpy(L.astype(np.int32)).cuda(), sched)
        assert np.array_equal(sched.cpu().numpy(), _lib.mla_chunk_plan_host(p, 76, cu, L))


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[-1, 5], [5, 64 * 8 + 1]])
def test_refused_plan_writes_nothing(lens):
    import torch
    q = Problem([2, 3], [100, 500], 16)
    attn = _lib.ChunkAttention(q.p)
    attn.plan(q.d_cu, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_INVALID_ARG
    out = torch.full((5, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 16), 7.0, device="cuda")
    attn.attend(q.d_q, q.d_qr, q.pool, q.d_bt, SCALE, out=out, lse=lse)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_WORKSPACE
    assert (out == 7).all() and (lse == 7).all()
    q.check(attn)                                  # the same buffers serve a good plan afterwards
    other = MlaChunkParams.from_buffer_copy(q.p)   # a plan of other params
    other.causal = 0
    attn.p = other
    attn.attend(q.d_q, q.d_qr, q.pool, q.d_bt, SCALE, out=out, lse=lse)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_WORKSPACE
    assert (out == 7).all() and (lse == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv, change", [("bf16", dict(causal=0)), ("bf16", dict(num_heads=15)), ("bf16", dict(max_tokens=4)),
                                        ("bf16", dict(num_units=9)), ("bf16", dict(max_pages_per_seq=46)), ("fp8", dict(max_kv_tokens=64 * 51)),
                                        ("bf16", dict(batch=1)), ("fp8", dict(kv_dtype=_lib.MLA_KV_BF16))])
def test_plan_of_other_params(kv, change):
    """A plan made for one set of params and used with another writes nothing, whichever of them differs: neither
    the attention nor the merge of the split blocks (there are some) takes an index from it."""
    import ctypes

    import torch
    q = Problem([2, 3], [300, 47 * 64], 16, kv, num_units=8)
    attn = _lib.ChunkAttention(q.p)
    q.check(attn)
    assert int(attn.sched[7]) > 0                  # split blocks
    other = MlaChunkParams.from_buffer_copy(q.p)
    for k, v in change.items():
        assert getattr(q.p, k) != v
        setattr(other, k, v)
    out = torch.full_like(q.d_q, 7.0)
    lse = torch.full(q.d_q.shape[:2], 7.0, device="cuda")
    ptr = lambda *ts: [ctypes.c_void_p(t.data_ptr()) for t in ts]  # noqa: E731
    st = _lib.load_library().mla_chunk_attend(
        ctypes.byref(other), *ptr(q.d_q, q.d_qr, q.pool, q.d_bt, q.d_L), ctypes.c_float(SCALE),
        *ptr(out, lse, attn.sched, _lib.ChunkAttention(q.p).workspace), ctypes.c_void_p(_lib._stream(None)))
    assert st == 0
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_WORKSPACE
    assert (out == 7).all() and (lse == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_captured_and_on_two_streams(kv):
    """Two problems, each with buffers of its own, captured into graphs and replayed at the same time on two
    streams after their inputs changed; the results are those of plain calls, bit for bit."""
    import torch
    qs = [Problem([3, 20, 1], [400, 1500, 64], 16, kv, seed=31, num_units=30),
          Problem([2, 2], [900, 2000], 128, kv, seed=32, num_units=30)]
    want = [q.run() for q in qs]
    state = []
    for q in qs:
        attn, st = _lib.ChunkAttention(q.p), torch.cuda.Stream()
        out, lse = torch.zeros_like(q.d_q), torch.zeros(q.d_q.shape[:2], device="cuda")
        keep = q.d_q.clone()
        q.d_q.zero_()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            attn.plan(q.d_cu, q.d_L)
            attn.attend(q.d_q, q.d_qr, q.pool, q.d_bt, SCALE, out=out, lse=lse)
        q.d_q.copy_(keep)
        state.append((g, st, out, lse, attn))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st, *_ in state:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    for (g, st, out, lse, _), (o, l) in zip(state, want):
        assert torch.equal(out, o) and torch.equal(lse, l)


@pytest.mark.gpu
@pytest.mark.parametrize("H,units", [(16, 1), (128, 0), (128, 9)])
@pytest.mark.parametrize("kv,dim", [("bf16", 7), ("bf16", 300), ("bf16", 515), ("fp8", 515)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("row", [5, 300, 640, 717])
def test_one_score_that_is_not_finite(H, units, kv, dim, value, row):
    """One value of one key: infinite, or finite where its product with the query leaves float32.  Whatever the sign of
    the score, whichever tile the key lies in (three are seen in full by every token, in the last some tokens see
    less), and whether the block is split: the tokens that see the key get NaN, the others keep their bits."""
    import torch
    n, L = 6, 720
    q = Problem([n], [L], H, kv, seed=23, num_units=units)
    sign = torch.where(torch.arange(H, device="cuda") % 2 == 0, 100.0, -100.0).to(torch.bfloat16)   # scores of either sign
    (q.d_q if dim < 512 else q.d_qr)[:, :, dim % 512] = sign
    want, want_lse = q.run()
    assert want.isfinite().all() and want_lse.isfinite().all()
    where = int(q.bt[0, row // 64]) * 64 + row % 64
    if kv == "bf16":
        q.pool.view(-1, 576)[where, dim] = value
    else:
        q.pool.view(-1, 656)[where, 528:].view(torch.bfloat16)[dim - 512] = value
    got, got_lse = q.run()
    first = max(0, row - (L - n))                 # the first token that sees the key
    assert torch.equal(got[:first], want[:first]) and torch.equal(got_lse[:first], want_lse[:first])
    assert got_lse[first:].isnan().all() and got[first:].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,L,H,units", [([4, 9], [130, 600], 128, 0), ([1, 0, 17, 3], [1, 50, 1025, 2], 40, 3), ([5, 2], [3, 0], 128, 2),
                                         ([30, 1], [260, 2000], 7, 9), ([2] * 9, [64 * k + 1 for k in range(9)], 64, 4)])
def test_without_the_causal_rule_everywhere(kv, n, L, H, units):
    """Every new token sees all L_b keys, those of later tokens among them: both row types, several blocks a sequence,
    split and dealt blocks, fewer rows than new tokens."""
    Problem(n, L, H, kv, seed=50 + units, causal=False, pad=2, num_units=units).check()
