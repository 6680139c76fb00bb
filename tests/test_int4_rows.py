"""INT4 cache rows: the format and its quantiser's arithmetic on the CPU; on the GPU the writer, the way back, the append, the
page upkeep and the chunk attention over such pages."""
import math
from fractions import Fraction

import numpy as np
import pytest

import mla_workloads as mw
from int4_util import SCALE, dequantize_rows, place, quantize_rows, random_rows, reference, wide
from mla_absorbed_decode_02_gb300 import _lib
from mla_absorbed_decode_02_gb300._lib import MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_INT4, MlaChunkParams, MlaError, MlaPoolParams
from mla_absorbed_decode_02_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return _lib.load_library()


# ------------------------------------------------------------------ arithmetic (CPU)
def _round(f, bits):
    """f to `bits` significant bits, ties to even (no under- or overflow)."""
    if f == 0:
        return f
    sign, f = (-1, -f) if f < 0 else (1, f)
    e = f.numerator.bit_length() - f.denominator.bit_length()
    e += (Fraction(2) ** (e + 1) <= f) - (Fraction(2) ** e > f)
    n = f / Fraction(2) ** (e - bits + 1)
    k, rest = n.numerator // n.denominator, n - n.numerator // n.denominator
    return sign * (k + (rest > Fraction(1, 2) or (rest == Fraction(1, 2) and k % 2))) * Fraction(2) ** (e - bits + 1)


def test_quotient_of_every_pair_of_significands():
    """x (8 significant bits) over a scale (4): the corrected reciprocal gives the correctly rounded quotient."""
    for s in range(8, 16):
        r = _round(Fraction(1, s), 24)
        for x in range(128, 256):
            q = _round(x * r, 24)
            assert _round(q + _round(x - q * s, 24) * r, 24) == _round(Fraction(x, s), 24), (x, s)


def test_every_value_is_exact():
    """(128 + n) s - 136 s as one bf16 FMA of bf16 operands: 136 s is a bf16, the result (n - 8) s too."""
    for s in range(8, 16):
        assert _round(Fraction(136 * s), 8) == 136 * s
        for n in range(16):
            assert _round(Fraction((n - 8) * s), 8) == (n - 8) * s and 128 + n < 256


def test_rows_by_hand():
    """One row's bytes, written out: the place of each code, the scale's rounding, the RoPE values."""
    x = np.zeros((1, 512), np.float32)
    x[0, :8] = [7, -7, 1, -1, 3.5, 0.5, 1.5, -0.5]      # scale 1; ties go to even
    x[0, 32] = 8                                        # 8 / 7 = 1.1428.. -> 1.25 (four bits: 1.125 is less)
    x[0, 33] = -3
    row = quantize_rows(x, np.arange(64, dtype=np.uint16)[None])[0]
    codes = {0: 15, 2: 9, 4: 12, 6: 10, 1: 1, 3: 7, 5: 8, 7: 8}
    word = sum(c << (4 * (d // 2) + 16 * (d % 2)) for d, c in codes.items())
    assert row[:4].view(np.uint32)[0] == word and row[4:8].view(np.uint32)[0] == 0x88888888
    assert row[256:260].view(np.uint16).tolist() == [0x3F80, 0x3FA0] and row[260:262].view(np.uint16)[0] == 0x3F80
    back = dequantize_rows(row)[0]
    assert back[:8].tolist() == [7, -7, 1, -1, 4, 0, 2, 0] and back[32:34].tolist() == [7.5, -2.5] and (back[40:512] == 0).all()
    assert np.array_equal(row[288:].view(np.uint16), np.arange(64))


def test_error_of_a_row():
    """Half a step at most, scale / 2, and a scale is at most 9/8 of amax / 7 (the next four-bit number)."""
    rng = np.random.default_rng(0)
    x = wide(mw.to_bf16_bits(rng.standard_normal((200, 512), dtype=np.float32) * np.exp(4 * rng.standard_normal((200, 1))).astype(np.float32)))
    back = dequantize_rows(quantize_rows(x, np.zeros((200, 64), np.uint16)))[:, :512]
    top = np.abs(x).reshape(200, 16, 32).max(-1).repeat(32, 1)
    assert (np.abs(back - x) <= top / 7 * 9 / 8 / 2 * (1 + 2 ** -20)).all()


def test_calls_refuse_bad_arguments():
    import ctypes
    import torch
    x, rows = torch.zeros(4, 576, dtype=torch.bfloat16), torch.zeros(4, 416, dtype=torch.uint8)
    for call, args in ((_lib.mla_quantize_kv_int4, (None, rows, 4)), (_lib.mla_quantize_kv_int4, (x, None, 4)), (_lib.mla_quantize_kv_int4, (x, rows, -1)),
                       (_lib.mla_quantize_kv_int4, (x[:3], rows, 4)), (_lib.mla_quantize_kv_int4, (x, rows[:3], 4)), (_lib.mla_quantize_kv_int4, (x.T, rows, 4)),
                       (_lib.mla_dequantize_kv, (3, rows, x, 4)), (_lib.mla_dequantize_kv, (-1, rows, x, 4)), (_lib.mla_dequantize_kv, (MLA_KV_INT4, rows[:3], x, 4)),
                       (_lib.mla_dequantize_kv, (MLA_KV_FP8_E4M3, rows, x, 4)), (_lib.mla_dequantize_kv, (MLA_KV_INT4, rows, x[:2], 4)),
                       (_lib.mla_dequantize_kv, (MLA_KV_INT4, rows, x, 4)), (_lib.mla_quantize_kv_int4, (x, rows, 4))):   # (host tensors, last)
        with pytest.raises(MlaError) as e:
            call(*args, stream=0)
        assert e.value.status == _lib.MLA_ERR_INVALID_ARG
    _lib.mla_quantize_kv_int4(x, rows, 0, stream=0)
    _lib.mla_dequantize_kv(MLA_KV_INT4, rows, x, 0, stream=0)
    lib = _lib.load_library()
    buf = ctypes.create_string_buffer(4096)
    g = (ctypes.addressof(buf) + 255) // 256 * 256
    for a in ((0, g, 1), (g, 0, 1), (g + 8, g, 1), (g, g + 8, 1), (g, g, -1)):
        assert lib.mla_quantize_kv_int4(*a, 0) == _lib.MLA_ERR_INVALID_ARG
        assert lib.mla_dequantize_kv(MLA_KV_INT4, *a, 0) == _lib.MLA_ERR_INVALID_ARG
    assert lib.mla_dequantize_kv(7, g, g, 1, 0) == _lib.MLA_ERR_INVALID_ARG


def test_params_take_the_format():
    p = MlaPoolParams.make(2, 10, 5, kv_dtype=MLA_KV_INT4, layer_stride=10 * 64 * 416)
    assert _lib.mla_pool_workspace_size(p, 4) > 0
    with pytest.raises(MlaError):
        _lib.mla_pool_workspace_size(MlaPoolParams.make(2, 10, 5, kv_dtype=MLA_KV_INT4, layer_stride=10 * 64 * 416 - 16), 4)
    with pytest.raises(MlaError):   # no room for the expanded rows
        _lib.mla_chunk_workspace_size(MlaChunkParams.make(1, 4, 16, 4, 4, kv_dtype=MLA_KV_INT4, num_units=3))
    kw = dict(num_units=3, max_kv_tokens=1000)
    assert (_lib.mla_chunk_workspace_size(MlaChunkParams.make(1, 4, 16, 4, 4, kv_dtype=MLA_KV_INT4, **kw))
            == _lib.mla_chunk_workspace_size(MlaChunkParams.make(1, 4, 16, 4, 4, kv_dtype=MLA_KV_FP8_E4M3, **kw)))


# ------------------------------------------------------------------ the writer and the way back (GPU)
def _write(x_bits):
    import torch
    x = torch.from_numpy(np.ascontiguousarray(x_bits).view(np.int16)).cuda().view(torch.bfloat16)
    out = torch.full((len(x) + 1, 416), 0xA5, dtype=torch.uint8, device="cuda")
    _lib.mla_quantize_kv_int4(x, out, len(x))
    assert (out[-1] == 0xA5).all()
    return out[:-1]


@pytest.mark.gpu
def test_writer_at_every_border():
    """Groups whose largest value is a hold the bf16 values on, just above and just below every border between two codes; scales
    over the whole float32 range, tiny, huge and zero among them."""
    rng = np.random.default_rng(1)
    groups = []
    for a in np.concatenate([np.exp2(rng.uniform(-130, 126, 600)), [0.0, 1.0, 7.0, 8.0, 2.0 ** -126, 2.0 ** -133, 9.2e-41, 3e38, 7 * 2.0 ** 119, 7 * 2.0 ** 119 * 1.01]]):
        top = wide(mw.to_bf16_bits(np.float32([a])))[0]
        s = max(float(((np.float32(top) / np.float32(7)).view(np.uint32) + np.uint32(0xFFFFF) & np.uint32(0xFFF00000)).view(np.float32)), 2.0 ** -126)
        with np.errstate(over="ignore"):
            bits = mw.to_bf16_bits(np.float32((np.arange(7) + 0.5) * s)).astype(np.int64)
        near = np.concatenate([bits - 1, bits, bits + 1, bits])
        x = wide(np.clip(near, 0, 0x7F7F).astype(np.uint16)) * rng.choice([-1, 1], 28).astype(np.float32)
        groups.append(np.concatenate([np.clip(x, -top, top), [top, 0, -top, -0.0]]).astype(np.float32))
    x = np.stack(groups)
    x = np.concatenate([x, np.zeros((-len(x) % 16, 32), np.float32)]).reshape(-1, 512)
    bits = mw.to_bf16_bits(np.concatenate([x, rng.standard_normal((len(x), 64), dtype=np.float32)], 1))
    want = quantize_rows(wide(bits[:, :512]), bits[:, 512:])
    got = _write(bits).cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:10]


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 7, 8, 4099])
def test_writer_and_way_back(n):
    import torch
    rng = np.random.default_rng(n)
    x = rng.standard_normal((n, 576), dtype=np.float32) * np.exp(5 * rng.standard_normal((n, 1))).astype(np.float32)
    bits = mw.to_bf16_bits(x)
    rows = _write(bits)
    assert np.array_equal(rows.cpu().numpy(), quantize_rows(wide(bits[:, :512]), bits[:, 512:]))
    back = torch.full((n + 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    _lib.mla_dequantize_kv(MLA_KV_INT4, rows, back, n)
    assert (back[n] == 7).all() and np.array_equal(back[:n].double().cpu().numpy(), dequantize_rows(rows.cpu().numpy()))
    # again from what was read back: the values are those of codes under a scale as large at most, so they stay
    again = torch.empty_like(rows)
    _lib.mla_quantize_kv_int4(back[:n].contiguous(), again, n)
    twice = torch.empty_like(back)
    _lib.mla_dequantize_kv(MLA_KV_INT4, again, twice, n)
    assert (twice[:n].double() - back[:n].double()).abs().max() <= back[:n, :512].double().abs().max() / 7 * 9 / 16
    # the other formats
    bf = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    out = torch.empty_like(bf)
    _lib.mla_dequantize_kv(MLA_KV_BF16, bf, out, n)
    assert torch.equal(out, bf)
    raw = torch.empty(n, 656, dtype=torch.uint8, device="cuda")
    _lib.mla_quantize_kv_fp8(bf, raw, n)
    _lib.mla_dequantize_kv(MLA_KV_FP8_E4M3, raw, out, n)
    import oracle
    lat, rope = oracle.fp8_rows_to_f64(raw.cpu().numpy())
    assert np.array_equal(out[:, :512].float().cpu().numpy(), wide(mw.to_bf16_bits(lat.astype(np.float32)))) and np.array_equal(out[:, 512:].double().cpu().numpy(), rope)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 3.3e38])
def test_values_that_are_not_finite(value):
    """All 32 of the group read back as NaN, the others as without it, the RoPE bits as they are."""
    import torch
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((3, 576), dtype=np.float32)).cuda().to(torch.bfloat16)
    y = x.clone()
    y[1, 70] = value
    y[2, 512 + 9] = value
    rows, plain = torch.empty(3, 416, dtype=torch.uint8, device="cuda"), torch.empty(3, 416, dtype=torch.uint8, device="cuda")
    _lib.mla_quantize_kv_int4(y, rows, 3)
    _lib.mla_quantize_kv_int4(x, plain, 3)
    a, b = torch.empty(3, 576, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 576, dtype=torch.bfloat16, device="cuda")
    _lib.mla_dequantize_kv(MLA_KV_INT4, rows, a, 3)
    _lib.mla_dequantize_kv(MLA_KV_INT4, plain, b, 3)
    assert torch.isnan(a[1, 64:96]).all()
    a[1, 64:96] = b[1, 64:96]
    assert torch.equal(a[2, 521:522].view(torch.int16), y[2, 521:522].view(torch.int16))
    a[2, 521] = b[2, 521]
    assert torch.equal(a, b)


# ------------------------------------------------------------------ append and upkeep (GPU)
def _ragged(n, L, seed, pad=0):
    import torch
    rng = np.random.default_rng(seed)
    n, L = np.asarray(n), np.asarray(L)
    P, bt = place(rng, L)
    T = int(n.sum()) + pad
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn(T, 576, device="cuda", generator=g) * torch.rand(T, 1, device="cuda", generator=g) * 30).to(torch.bfloat16)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    cu = np.concatenate([[0], np.cumsum(n)])
    at = [(int(bt[b, q // 64]), q % 64) for b in range(len(n)) for q in range(int(L[b] - n[b]), int(L[b]))]
    pool = torch.randint(0, 256, (P, 64, 416), device="cuda", generator=g, dtype=torch.uint8)
    return MlaPoolParams.make(len(n), P, bt.shape[1], kv_dtype=MLA_KV_INT4), x, dev(cu), dev(L), dev(bt), pool, at


@pytest.mark.gpu
@pytest.mark.parametrize("served", [False, True])
@pytest.mark.parametrize("n,L,pad", [([1], [1], 0), ([0, 3, 0, 0, 70, 1], [9, 3, 0, 64, 200, 129], 5), ([1] * 33, list(range(1, 34)), 0),
                                     ([2, 0] * 700, [100, 7] * 700, 1)])
def test_append_writes_the_rows(n, L, pad, served):
    import torch
    p, x, cu, lens, bt, pool, at = _ragged(n, L, seed=len(n), pad=pad)
    want = pool.clone()
    raw = torch.empty(len(x), 416, dtype=torch.uint8, device="cuda")
    _lib.mla_quantize_kv_int4(x, raw, len(x))
    took = torch.ones(len(n), dtype=torch.int32, device="cuda")
    if served:
        took[1::3] = 0
    keep = torch.repeat_interleave(took.cpu(), torch.tensor(n)).bool().numpy()
    pg, r = (np.array(v) for v in zip(*at))
    want[pg[keep], r[keep]] = raw[:len(at)][torch.from_numpy(keep).cuda()]
    _lib.mla_append_kv(p, x[:, :512], x[:, 512:], cu, lens, bt, pool, served=took if served else None)
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    assert torch.equal(pool, want)


@pytest.mark.gpu
def test_upkeep_moves_the_pages():
    """Copy, fork, free and compact on pages of this size, in two layers with a gap between them."""
    import torch
    P, B, M = 40, 6, 8
    stride = P * 64 * 416 + 4096
    pool = torch.randint(0, 256, (2 * stride - 4096,), dtype=torch.uint8, device="cuda")
    layer = lambda i: pool[i * stride:i * stride + P * 64 * 416].view(P, 64, 416)  # noqa: E731
    keeper = _lib.PagePool(MlaPoolParams.make(B, P, M, kv_dtype=MLA_KV_INT4, num_layers=2, layer_stride=stride))
    bt, lens, ref = keeper.new_tables()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    assert keeper.reserve(i32(100, 0, 300, 64, 0, 0), bt, lens, ref).tolist() == [1] * 6
    rows = lambda b, i: layer(i)[bt[b, :-(-int(lens[b]) // 64)].long()].reshape(-1, 416)[:int(lens[b])].clone()  # noqa: E731
    held = {b: [rows(b, i) for i in (0, 1)] for b in (0, 2, 3)}
    assert keeper.fork(pool, i32(0, 2, 3), i32(1, 4, 5), bt, lens, ref)[2] == -1
    for child, parent in ((1, 0), (4, 2), (5, 3)):
        assert all(torch.equal(rows(child, i), held[parent][i]) for i in (0, 1))
    keeper.free(i32(0, 3), bt, lens, ref)
    used = keeper.compact(pool, bt, lens, ref)
    assert int(used) == int((ref > 0).sum()) and (ref[:int(used)] > 0).all()
    for b, parent in ((1, 0), (2, 2), (4, 2), (5, 3)):
        assert all(torch.equal(rows(b, i), held[parent][i]) for i in (0, 1))
    before = [layer(i).clone() for i in (0, 1)]
    keeper.copy(pool, i32(3, 0), i32(38, 39))
    for i in (0, 1):
        before[i][38], before[i][39] = before[i][3], before[i][0]
        assert torch.equal(layer(i), before[i])
    assert _lib.mla_device_error(clear=True) == 0


# ------------------------------------------------------------------ chunk attention (GPU)
def _chunk(n, L, H, seed, pad=0, units=0, causal=True):
    """Runs the chunk attention and compares it with the definition on the rows' exact values."""
    import torch
    rng = np.random.default_rng([seed, H])
    n, L = np.asarray(n), np.asarray(L)
    P, bt = place(rng, L)
    T = int(n.sum()) + pad
    raw = random_rows(rng, P * 64).reshape(P, 64, 416)
    for b in range(len(L)):  # past the end: any bits
        if L[b] % 64:
            raw[bt[b, L[b] // 64], L[b] % 64:] = 0xFF
    bits = lambda *s: mw.to_bf16_bits(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    q, qr = bits(max(T, 1), H, 512), bits(max(T, 1), H, 64)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    p = MlaChunkParams.make(len(n), max(T, 1), H, P, bt.shape[1], causal=causal, kv_dtype=MLA_KV_INT4, num_units=units,
                            max_kv_tokens=max(64, int((-(-L // 64)).sum()) * 64))
    attn = _lib.ChunkAttention(p)
    out, lse = torch.full((max(T, 1), H, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((max(T, 1), H), 7.0, device="cuda")
    attn.plan(dev(cu), dev(L.astype(np.int32)))
    attn.attend(dev(q.view(np.int16)).view(torch.bfloat16), dev(qr.view(np.int16)).view(torch.bfloat16), dev(raw), dev(bt), SCALE, out=out, lse=lse)
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    T = int(n.sum())
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(n)):
        rows = dequantize_rows(raw[bt[b, :-(-int(L[b]) // 64)]])[:int(L[b])] if L[b] else np.zeros((0, 576))
        for i in range(int(n[b])):
            t = int(cu[b]) + i
            ref, rl, to, tl = reference(wide(q[t]).astype(np.float64), wide(qr[t]).astype(np.float64), rows, int(L[b]) - (int(n[b]) - 1 - i if causal else 0))
            none = np.isneginf(rl)
            assert np.array_equal(none, np.isneginf(l[t])) and (np.abs(o[t] - ref) <= to).all() and (np.abs(l[t] - rl)[~none] <= tl[~none]).all(), (b, i)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 16, 40, 128])
@pytest.mark.parametrize("n,L", [([1], [1]), ([5, 0, 2, 9], [5, 77, 2, 300]), ([2, 4, 1], [0, 2, 64]), ([1, 17, 8, 1], [256, 257, 513, 640])])
def test_chunk_attention(n, L, H):
    _chunk(n, L, H, seed=len(n), pad=len(n) % 3)


@pytest.mark.gpu
def test_chunk_attention_in_other_ways():
    _chunk([3, 1], [2600, 130], 128, seed=1, units=2)
    _chunk([4, 9], [130, 600], 16, seed=2, causal=False)
    _chunk([0, 0], [70, 5], 16, seed=3, pad=2)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [0x7C00, 0x7F00, 0x7F80, 0x7FC0, 0xFC00, 0xFF80])
def test_scales_that_overflow_read_back_as_nan(bits):
    """All 32 values of the group, whatever their codes; the largest scale below them is still exact."""
    import torch
    rng = np.random.default_rng(22)
    raw = random_rows(rng, 9)
    raw[4, 256:288].view(np.uint16)[5] = bits
    raw[6, 256:288].view(np.uint16)[2] = 0x7BF0
    raw[6, :256].view(np.uint32)[8:12] = 0x08080808 | 0x10111111    # (codes whose values a float32 holds: -8 .. 1 times 1.875 2^120)
    out = torch.empty(9, 576, dtype=torch.bfloat16, device="cuda")
    _lib.mla_dequantize_kv(MLA_KV_INT4, torch.from_numpy(raw).cuda(), out, 9)
    got = out.double().cpu().numpy()
    assert np.isnan(got[4, 160:192]).all()
    raw[4, 256:288].view(np.uint16)[5] = 0x3F80
    want = dequantize_rows(raw)
    got[4, 160:192] = want[4, 160:192]
    assert np.array_equal(got, want)


@pytest.mark.gpu
def test_chunks_over_a_scale_that_overflows():
    """The tokens that see the key get NaN, the others keep their bits; all queries positive."""
    import torch
    rng = np.random.default_rng(23)
    P, bt = place(rng, np.array([300, 70]))
    raw = random_rows(rng, P * 64).reshape(P, 64, 416)
    g = torch.Generator("cuda").manual_seed(23)
    q, qr = (torch.randn(9, 16, d, device="cuda", generator=g).abs().to(torch.bfloat16) for d in (512, 64))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    attn = _lib.ChunkAttention(MlaChunkParams.make(2, 9, 16, P, bt.shape[1], kv_dtype=MLA_KV_INT4, max_kv_tokens=(5 + 2) * 64))
    attn.plan(i32(0, 6, 9), i32(300, 70))
    table = torch.from_numpy(bt).cuda()
    before, lse0 = attn.attend(q, qr, torch.from_numpy(raw).cuda(), table, SCALE)
    for row in (40, 296):
        bad = raw.copy()
        bad[bt[0, row // 64], row % 64, 256:288].view(np.uint16)[9] = 0x7C00
        out, lse = attn.attend(q, qr, torch.from_numpy(bad).cuda(), table, SCALE)
        sees = [t for t in range(6) if row <= 294 + t]
        keep = [t for t in range(9) if t not in sees]
        assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
        assert torch.equal(out[keep], before[keep]) and torch.equal(lse[keep], lse0[keep])
    assert _lib.mla_device_error(clear=True) == 0


def test_calls_refuse_other_types():
    """bf16 rows that are no bf16, packed rows that are no bytes."""
    import torch
    x, rows = torch.zeros(4, 576, dtype=torch.bfloat16), torch.zeros(4, 416, dtype=torch.uint8)
    q, d = _lib.mla_quantize_kv_int4, _lib.mla_dequantize_kv
    for call, args, name in ((q, (x.float(), rows, 4), "kv_bf16"), (q, (x.half(), rows, 4), "kv_bf16"), (q, (x.view(torch.uint8), rows, 4), "kv_bf16"),
                             (q, (x, torch.zeros(4, 208, dtype=torch.int16), 4), "kv_int4"), (q, (x, torch.zeros(4, 416, dtype=torch.bfloat16), 4), "kv_int4"),
                             (d, (MLA_KV_INT4, rows, x.float(), 4), "kv_bf16"), (d, (MLA_KV_FP8_E4M3, torch.zeros(4, 656, dtype=torch.uint8), x.half(), 4), "kv_bf16"),
                             (d, (MLA_KV_INT4, torch.zeros(4, 416), x, 4), "kv_rows"), (d, (MLA_KV_FP8_E4M3, torch.zeros(4, 328, dtype=torch.int16), x, 4), "kv_rows"),
                             (d, (MLA_KV_BF16, x.half(), x, 4), "kv_rows"), (d, (MLA_KV_BF16, x.float(), x, 4), "kv_rows")):
        with pytest.raises(MlaError, match=name) as e:
            call(*args, stream=0)
        assert e.value.status == _lib.MLA_ERR_INVALID_ARG
    for kv, t in ((MLA_KV_BF16, x.clone()), (MLA_KV_BF16, torch.zeros(4, 1152, dtype=torch.uint8)), (MLA_KV_INT4, rows)):
        with pytest.raises(MlaError, match="device"):      # (taken, but for lying on the host)
            d(kv, t, x, 4, stream=0)


def test_calls_refuse_rows_written_over_others():
    import torch
    buf = torch.zeros(4 * 1152 + 4 * 656, dtype=torch.uint8)
    wide_rows = buf[:4 * 1152].view(torch.bfloat16).view(4, 576)
    for at in (0, 416, 4 * 1152 - 16):
        with pytest.raises(MlaError, match="overlap"):
            _lib.mla_quantize_kv_int4(wide_rows, buf[at:at + 4 * 416], 4, stream=0)
        with pytest.raises(MlaError, match="overlap"):
            _lib.mla_dequantize_kv(MLA_KV_INT4, buf[at:at + 4 * 416], wide_rows, 4, stream=0)
    with pytest.raises(MlaError, match="overlap"):
        _lib.mla_dequantize_kv(MLA_KV_BF16, wide_rows, wide_rows, 4, stream=0)
    with pytest.raises(MlaError, match="device"):          # side by side
        _lib.mla_quantize_kv_int4(wide_rows, buf[4 * 1152:], 4, stream=0)
    with pytest.raises(MlaError, match="device"):          # (rows past num_tokens are not touched)
        _lib.mla_dequantize_kv(MLA_KV_INT4, buf[2 * 1152:], wide_rows, 2, stream=0)


# ------------------------------------------------------------------ bounds of every group, scales past the largest, types
@pytest.mark.gpu
def test_quantised_again():
    """Rows of very different sizes, read back and written again: the bytes are those of the definition on the values read, and each
    group of 32 moves by half a step of its own new scale at most."""
    import torch
    rng = np.random.default_rng(21)
    n = 999
    x = rng.standard_normal((n, 576), dtype=np.float32) * np.exp(5 * rng.standard_normal((n, 1))).astype(np.float32)
    rows = _write(mw.to_bf16_bits(x))
    back = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    _lib.mla_dequantize_kv(MLA_KV_INT4, rows, back, n)
    again, twice = torch.empty_like(rows), torch.empty_like(back)
    _lib.mla_quantize_kv_int4(back, again, n)
    _lib.mla_dequantize_kv(MLA_KV_INT4, again, twice, n)
    bits = back.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(again.cpu().numpy(), quantize_rows(wide(bits[:, :512]), bits[:, 512:]))
    step = wide(again[:, 256:288].contiguous().cpu().numpy().view(np.uint16)).astype(np.float64).repeat(32, 1)
    assert (np.abs((twice[:, :512].double() - back[:, :512].double()).cpu().numpy()) <= step / 2).all()
    assert torch.equal(twice[:, 512:], back[:, 512:])
