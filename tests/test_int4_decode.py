"""Decode over INT4 pages: parameters and plan on the CPU, the kernels against the definition in float64 on the GPU.
The bounds are derived beside int4_util.reference."""
import math

import numpy as np
import pytest

import mla_workloads as mw
from int4_util import SCALE, dequantize_rows, place, random_rows, reference, wide
from mla_absorbed_decode_02_gb300 import _lib
from mla_absorbed_decode_02_gb300._lib import MLA_KV_INT4, MlaDecodeParams, MlaError
from mla_absorbed_decode_02_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return _lib.load_library()


def _params(**kw):
    base = dict(batch=3, s_q=4, num_heads=16, num_pages=20, max_pages_per_seq=9, kv_dtype=MLA_KV_INT4, num_units=7)
    base.update(kw)
    return MlaDecodeParams.make(**base)


# ------------------------------------------------------------------ parameters and plan (CPU)
@pytest.mark.parametrize("kw,status", [
    (dict(qk_fp8=1), _lib.MLA_ERR_INVALID_ARG), (dict(token_group=3), _lib.MLA_ERR_INVALID_ARG), (dict(num_heads=129), _lib.MLA_ERR_UNSUPPORTED),
    (dict(num_heads=33, token_group=2), _lib.MLA_ERR_UNSUPPORTED), (dict(num_heads=17, token_group=4), _lib.MLA_ERR_UNSUPPORTED),
    (dict(page_size=32), _lib.MLA_ERR_UNSUPPORTED),
])
def test_bad_params(kw, status):
    with pytest.raises(MlaError) as e:
        _lib.mla_get_workspace_size(_params(**kw))
    assert e.value.status == status


@pytest.mark.parametrize("H,s_q,group,want", [(16, 4, 0, 4), (16, 8, 0, 4), (8, 8, 0, 8), (20, 4, 0, 2), (20, 3, 0, 3), (21, 6, 0, 3), (32, 8, 0, 2),
                                              (33, 8, 0, 1), (128, 4, 0, 1), (16, 4, 1, 1), (16, 4, 2, 2), (1, 7, 0, 7), (64, 1, 0, 1)])
def test_tokens_share_keys_as_far_as_64_rows_hold_them(H, s_q, group, want):
    p = _params(num_heads=H, s_q=s_q, token_group=group, batch=2)
    plan = _lib.mla_plan_host(p, 7, [100, 300])
    assert plan[5] == want
    assert _lib.mla_get_workspace_size(p)[1] >= (2 * s_q + want * 7) * H * 513 * 4


# ------------------------------------------------------------------ the kernel (GPU)
class Problem:
    def __init__(self, L, H, s_q=1, causal=True, seed=0, units=0, group=0, f32=False, spread=0.0, garbage=True, q_scale=1.0):
        import torch
        rng = np.random.default_rng([seed, H, s_q])
        self.L, self.H, self.s_q, self.causal = np.asarray(L), H, s_q, causal
        B = len(L)
        P, self.bt = place(rng, self.L)
        self.raw = random_rows(rng, P * 64, spread).reshape(P, 64, 416)
        if garbage:  # rows past the sequences' ends and pages that no sequence has: any bits
            used = np.zeros((P, 64), bool)
            for b in range(B):
                for j in range(-(-int(self.L[b]) // 64)):
                    used[self.bt[b, j], :min(64, int(self.L[b]) - 64 * j)] = True
            self.raw[~used] = rng.integers(0, 256, (int((~used).sum()), 416), dtype=np.uint8)
            self.raw[~used, 256:] |= 0xFF  # NaN scales and RoPE values among them
        bits = lambda *s: mw.to_bf16_bits(rng.standard_normal(s, dtype=np.float32) * np.float32(q_scale))  # noqa: E731
        self.q, self.qr = bits(B, s_q, H, 512), bits(B, s_q, H, 64)
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.d_q, self.d_qr = dev(self.q.view(np.int16)).view(torch.bfloat16), dev(self.qr.view(np.int16)).view(torch.bfloat16)
        self.pool, self.d_bt, self.d_L = dev(self.raw), dev(self.bt), dev(self.L.astype(np.int32))
        self.p = MlaDecodeParams.make(B, s_q, H, P, self.bt.shape[1], causal=causal, kv_dtype=MLA_KV_INT4, num_units=units, token_group=group,
                                      out_dtype=_lib.MLA_OUT_F32 if f32 else _lib.MLA_OUT_BF16)

    def rows(self, b):
        return dequantize_rows(self.raw[self.bt[b, :-(-int(self.L[b]) // 64)]])[:int(self.L[b])]

    def run(self, dec=None):
        import torch
        dec = dec or _lib.Decoder(self.p)
        dec.plan(self.d_L)
        out, lse = dec.new_outputs()
        out.fill_(7.0)
        lse.fill_(7.0)
        dec.decode(self.d_q, self.d_qr, self.pool, self.d_bt, self.d_L, SCALE, out=out, lse=lse)
        torch.cuda.synchronize()
        assert _lib.mla_device_error(clear=True) == 0
        return out, lse

    def check(self, dec=None):
        out, lse = self.run(dec)
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(len(self.L)):
            rows = self.rows(b)
            for t in range(self.s_q):
                seen = int(self.L[b]) - (self.s_q - 1 - t if self.causal else 0)
                ref, rl, to, tl = reference(wide(self.q[b, t]).astype(np.float64), wide(self.qr[b, t]).astype(np.float64), rows, seen)
                if seen <= 0:
                    assert (o[b, t] == 0).all() and np.isneginf(l[b, t]).all()
                    continue
                assert (np.abs(o[b, t] - ref) <= to).all(), (b, t, float((np.abs(o[b, t] - ref) - to).max()))
                assert (np.abs(l[b, t] - rl) <= tl).all(), (b, t, float(np.abs(l[b, t] - rl).max()))
        return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 7, 16, 17, 32, 40, 64, 65, 96, 127, 128])
@pytest.mark.parametrize("L", [[1], [64], [65, 3, 0, 128], [129, 127, 500, 1, 257], [1300, 63]])
def test_matches_float64(H, L):
    Problem(L, H, seed=len(L)).check()


@pytest.mark.gpu
@pytest.mark.parametrize("s_q", [2, 3, 4, 8])
@pytest.mark.parametrize("H", [5, 8, 16, 20, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_several_new_tokens(s_q, H, causal):
    """Lengths at the tiles' and pages' borders; some tokens see no key."""
    Problem([8, 2, 64 + s_q - 1, 128, 129, 131, 260, 0], H, s_q=s_q, causal=causal, seed=s_q).check()


@pytest.mark.gpu
@pytest.mark.parametrize("units", [1, 2, 3, 11, 76, 152])
@pytest.mark.parametrize("H,s_q", [(16, 1), (16, 4), (40, 1), (128, 2)])
def test_units_share_and_split_the_work(units, H, s_q):
    Problem([700, 64, 1, 2111, 190], H, s_q=s_q, units=units, seed=units).check()


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("f32", [False, True])
def test_groups_and_float32_outputs(group, f32):
    Problem([70, 333, 5], 16, s_q=4, group=group, f32=f32, seed=group).check()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 128])
def test_scores_that_grow_along_the_keys(H):
    """Values of very different sizes: the running maximum is raised again and again, the output rescaled."""
    q = Problem([3000, 900], H, seed=3, spread=1.5, q_scale=2.0)
    q.check()


@pytest.mark.gpu
def test_long_sequences():
    Problem([40000, 9000, 17], 16, seed=5).check()
    Problem([20000], 128, seed=6).check()


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q", [(16, 1), (16, 4), (128, 3)])
@pytest.mark.parametrize("where", ["scale", "rope"])
@pytest.mark.parametrize("row", [5, 130, 296, 299])
def test_a_key_that_holds_nan(H, s_q, where, row):
    """NaN for the tokens that see the key, and the bits of the others as without it."""
    import torch
    L = [300, 70]
    q = Problem(L, H, s_q=s_q, seed=9)
    before, lse0 = q.run()
    at = q.pool[int(q.bt[0, row // 64]), row % 64]
    (at[256:288] if where == "scale" else at[288:]).view(torch.bfloat16)[7] = math.nan
    out, lse = q.run()
    for t in range(s_q):
        if row < L[0] - (s_q - 1 - t):
            assert torch.isnan(lse[0, t]).all()
            assert torch.isnan(out[0, t]).all()
        else:
            assert torch.equal(out[0, t], before[0, t]) and torch.equal(lse[0, t], lse0[0, t])
    assert torch.equal(out[1], before[1]) and torch.equal(lse[1], lse0[1])


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q", [(16, 4), (128, 3)])
@pytest.mark.parametrize("bits", [0x7C00, 0x7F00, 0x7F80])
@pytest.mark.parametrize("row", [297, 299])
def test_a_scale_that_overflows(H, s_q, bits, row):
    """2^121, the largest binade and infinity: tokens that do not see the key keep their bits."""
    import torch
    L = [300, 70]
    q = Problem(L, H, s_q=s_q, seed=10)
    before, lse0 = q.run()
    q.pool[int(q.bt[0, row // 64]), row % 64][256:288].view(torch.int16)[3] = bits
    out, lse = q.run()
    for t in range(s_q):
        if row < L[0] - (s_q - 1 - t):
            assert torch.isnan(out[0, t]).all() and torch.isnan(lse[0, t]).all()
        else:
            assert torch.equal(out[0, t], before[0, t]) and torch.equal(lse[0, t], lse0[0, t])
    assert torch.equal(out[1], before[1]) and torch.equal(lse[1], lse0[1])


@pytest.mark.gpu
@pytest.mark.parametrize("H,units", [(16, 0), (40, 5), (128, 0)])
def test_the_same_bits_every_time(H, units):
    import torch
    q = Problem([4000, 33, 700], H, s_q=2, units=units, seed=2)
    dec = _lib.Decoder(q.p)
    a = q.run(dec)
    for _ in range(3):
        b = q.run(dec)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_pages_past_four_gigabytes():
    """The last pages of a pool of more than 2^32 bytes that is otherwise never touched."""
    import torch
    q = Problem([200, 130], 16, seed=8)
    first = 165000
    pool = torch.empty(first + q.raw.shape[0], 64, 416, dtype=torch.uint8, device="cuda")
    pool[first:] = q.pool
    want = q.run()
    q.pool, q.d_bt = pool, torch.where(q.d_bt >= 0, q.d_bt + first, q.d_bt)
    q.p.num_pages = pool.shape[0]
    got = q.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_agrees_with_the_decode_of_the_rows_as_bf16():
    """The bf16 decode over the dequantised pool: the same values to both kernels, so within twice the bound."""
    import torch
    q = Problem([500, 64, 1111], 128, s_q=2, seed=12, garbage=False)
    out, lse = q.run()
    rows = torch.empty(q.raw.shape[0], 64, 576, dtype=torch.bfloat16, device="cuda")
    _lib.mla_dequantize_kv(MLA_KV_INT4, q.pool, rows, rows.shape[0] * 64)
    p = MlaDecodeParams.make(3, 2, 128, rows.shape[0], q.bt.shape[1])
    dec = _lib.Decoder(p)
    dec.plan(q.d_L)
    o, l = dec.decode(q.d_q, q.d_qr, rows, q.d_bt, q.d_L, SCALE)
    assert (out.float() - o.float()).norm() <= 5e-3 * o.float().norm() and (lse - l).abs().max() <= 1e-3


@pytest.mark.gpu
def test_captured_and_on_two_streams():
    """Two decoders captured into one graph each, replayed side by side on other streams than they were captured on."""
    import torch
    probs = [Problem([900, 70, 3], 16, seed=20), Problem([64, 2100], 128, s_q=2, seed=21)]
    want, graphs, outs, decs = [q.run() for q in probs], [], [], []
    for q in probs:
        dec = _lib.Decoder(q.p)
        out, lse = dec.new_outputs()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            dec.plan(q.d_L)
            dec.decode(q.d_q, q.d_qr, q.pool, q.d_bt, q.d_L, SCALE, out=out, lse=lse)
        graphs.append(g), outs.append((out, lse)), decs.append(dec)
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.gpu
def test_without_allocation():
    import torch
    q = Problem([900, 70, 3], 40, s_q=2, seed=23)
    want = q.run()
    dec = _lib.Decoder(q.p)
    out, lse = dec.new_outputs()
    _lib.mla_decode_noalloc(q.p, q.d_q, q.d_qr, q.pool, q.d_bt, q.d_L, SCALE, out, lse)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_what_the_device_reports():
    """Pages outside the pool, lengths past the table, metadata of other params: the error word, and other sequences as before."""
    import torch
    q = Problem([200, 130, 64], 16, seed=30)
    want = q.run()
    dec = _lib.Decoder(q.p)
    for bad in (q.p.num_pages, -1, 1 << 30):
        bt = q.d_bt.clone()
        bt[1, 1] = bad
        dec.plan(q.d_L)
        out, lse = dec.decode(q.d_q, q.d_qr, q.pool, bt, q.d_L, SCALE)
        assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_INVALID_ARG
        assert torch.equal(out[0], want[0][0]) and torch.equal(out[2], want[0][2])
    lens = q.d_L.clone()
    lens[1] = q.bt.shape[1] * 64 + 100
    dec.plan(lens)
    out, lse = dec.decode(q.d_q, q.d_qr, q.pool, q.d_bt, lens, SCALE)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_INVALID_ARG
    assert torch.equal(out[0], want[0][0]) and torch.equal(out[2], want[0][2])
    other = _lib.Decoder(MlaDecodeParams.make(3, 1, 16, q.p.num_pages, q.bt.shape[1], kv_dtype=MLA_KV_INT4, num_units=9))
    other.plan(q.d_L)
    dec.sched[:other.sched.numel()] = other.sched
    out, lse = dec.new_outputs()
    out.fill_(7.0)
    dec.decode(q.d_q, q.d_qr, q.pool, q.d_bt, q.d_L, SCALE, out=out, lse=lse)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_WORKSPACE
    assert (out == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q", [(16, 1), (16, 3), (40, 1), (128, 1)])
@pytest.mark.parametrize("units", [5, 0])
def test_nan_in_every_split(H, s_q, units):
    """One key of every tile holds NaN: the merged row is NaN too, and does not look like one that saw no key."""
    import torch
    L = [2000, 1900, 130]
    q = Problem(L, H, s_q=s_q, seed=15, units=units)
    before, lse0 = q.run()
    for j in range(-(-L[0] // 64)):
        q.pool[int(q.bt[0, j]), 3][256:288].view(torch.bfloat16)[j % 16] = math.nan
    out, lse = q.run()
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(out[1:], before[1:]) and torch.equal(lse[1:], lse0[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q", [(16, 1), (20, 2), (128, 1)])
@pytest.mark.parametrize("units", [1, 5, 0])
def test_a_query_that_holds_nan(H, s_q, units):
    """One head of one token: NaN for it, split or not, and the bits of the others as without it."""
    import torch
    q = Problem([2000, 1900, 130], H, s_q=s_q, seed=16, units=units)
    before, lse0 = q.run()
    b, t, h = 1, s_q - 1, H // 2
    q.d_q[b, t, h, 100] = math.nan
    out, lse = q.run()
    assert torch.isnan(out[b, t, h]).all() and torch.isnan(lse[b, t, h])
    out[b, t, h], lse[b, t, h] = before[b, t, h], lse0[b, t, h]
    assert torch.equal(out, before) and torch.equal(lse, lse0)


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q", [(16, 1), (16, 3), (40, 1), (64, 1), (128, 2)])
@pytest.mark.parametrize("bits", [0x7C00, 0x7F00, 0x7F80, 0xFC00, 0xFF80])
@pytest.mark.parametrize("row", [5, 130, 299])
def test_a_scale_that_overflows_where_no_score_would_be_nan(H, s_q, bits, row):
    """Queries that are all positive, so that products with values of one infinity do not cancel to NaN by themselves."""
    import torch
    L = [300, 70]
    q = Problem(L, H, s_q=s_q, seed=17)
    q.d_q.abs_()
    before, lse0 = q.run()
    q.pool[int(q.bt[0, row // 64]), row % 64][256:288].view(torch.int16)[3] = bits - (1 << 16 if bits >> 15 else 0)
    out, lse = q.run()
    for t in range(s_q):
        if row < L[0] - (s_q - 1 - t):
            assert torch.isnan(lse[0, t]).all() and torch.isnan(out[0, t]).all()
        else:
            assert torch.equal(out[0, t], before[0, t]) and torch.equal(lse[0, t], lse0[0, t])
    assert torch.equal(out[1], before[1]) and torch.equal(lse[1], lse0[1])


# ------------------------------------------------------------------ numbers of tokens, heads and rows beyond the ones above
@pytest.mark.parametrize("H,s_q,want", [(16, 5, 1), (16, 7, 1), (10, 7, 1), (32, 3, 1), (12, 5, 5), (9, 7, 7), (16, 6, 3), (20, 6, 3), (40, 2, 1)])
def test_a_group_divides_the_new_tokens(H, s_q, want):
    """Fewer tokens than fit where their number does not divide s_q."""
    assert _lib.mla_plan_host(_params(num_heads=H, s_q=s_q, batch=2), 7, [100, 300])[5] == want


@pytest.mark.gpu
@pytest.mark.parametrize("s_q", [5, 6, 7])
@pytest.mark.parametrize("H", [3, 9, 12, 16, 20, 33, 96])
@pytest.mark.parametrize("causal", [True, False])
def test_odd_numbers_of_new_tokens(s_q, H, causal):
    Problem([8, 3, 64 + s_q - 1, 129, 131, 260, 0], H, s_q=s_q, causal=causal, seed=s_q).check()


def _isolated(L, H, s_q, seed, put, row, units=0):
    """`put` spoils row `row` of the first sequence: NaN for the tokens that see it, and the bits of the others as without it."""
    import torch
    q = Problem(L, H, s_q=s_q, seed=seed, units=units)
    before, lse0 = q.run()
    put(q.pool[int(q.bt[0, row // 64]), row % 64])
    out, lse = q.run()
    for t in range(s_q):
        if row < L[0] - (s_q - 1 - t):
            assert torch.isnan(out[0, t]).all() and torch.isnan(lse[0, t]).all()
        else:
            assert torch.equal(out[0, t], before[0, t]) and torch.equal(lse[0, t], lse0[0, t])
    assert torch.equal(out[1:], before[1:]) and torch.equal(lse[1:], lse0[1:])


# rows of a CTA: 20, 30, 32 (two softmax warpgroups), 40, 48 (three), 64; two CTAs of 33 and of 48
SHARED = [(20, 1), (10, 3), (16, 2), (20, 2), (16, 3), (40, 1), (12, 5), (66, 2), (96, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q", SHARED)
@pytest.mark.parametrize("where", ["scale", "rope"])
@pytest.mark.parametrize("row", [5, 297, 298, 299])
def test_a_key_that_holds_nan_at_every_number_of_rows(H, s_q, where, row):
    import torch

    def put(at):
        (at[256:288] if where == "scale" else at[288:]).view(torch.bfloat16)[7] = math.nan
    _isolated([300, 70], H, s_q, 13, put, row)


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q", SHARED)
@pytest.mark.parametrize("bits", [0x7C00, 0x7F80])
@pytest.mark.parametrize("row", [297, 299])
def test_a_scale_that_overflows_at_every_number_of_rows(H, s_q, bits, row):
    import torch

    def put(at):
        at[256:288].view(torch.int16)[11] = bits
    _isolated([300, 70], H, s_q, 14, put, row)


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q,units", [(16, 1, 0), (16, 3, 5), (40, 1, 0), (128, 2, 0)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, 3e38])
def test_a_query_that_is_not_finite_leaves_the_others(H, s_q, units, value):
    """A head whose scores are infinite or overflow: the other heads of the tile keep their bits, though maxima are exchanged at every tile."""
    import torch
    q = Problem([2000, 700, 130], H, s_q=s_q, seed=18, units=units)
    before, lse0 = q.run()
    b, t, h = 0, s_q // 2, H - 1
    q.d_q[b, t, h, 8:12] = value
    q.d_qr[b, t, h, 5] = -value
    out, lse = q.run()
    assert not torch.isfinite(lse[b, t, h])
    out[b, t, h], lse[b, t, h] = before[b, t, h], lse0[b, t, h]
    assert torch.equal(out, before) and torch.equal(lse, lse0)
