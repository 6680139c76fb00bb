"""The append of unrotated rows: refusals on the CPU; on the GPU the rows, the keys' and the queries' rotation and the norm
against float64, and a run of all of it with the decode.

Tolerances.  A rotated value is x c - y s in float32 (two roundings and the table's own, 2^-24 each) rounded to bf16 once:
|error| <= 2^-8 |value| + 2^-22 (|x| + |y|).  A normed value is x r w with r from a float32 sum of 512 squares (each
addition off by 2^-24 of a sum that only grows, through a tree of 16 and 5 steps: 2^-19 in all), a reciprocal root within 2 ulp and
two products, rounded to bf16 once: |error| <= 2^-8 |value| + 2^-17 |value|.  Where rows are quantised, what is compared is the bytes
that the writer gives for the normed rows this library appends to bf16 pages."""
import ctypes
import math

import numpy as np
import pytest

from int4_util import SCALE, place
from mla_absorbed_decode_02_gb300 import _lib
from mla_absorbed_decode_02_gb300._lib import MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_INT4, MlaError, MlaPoolParams, MlaRotateParams
from mla_absorbed_decode_02_gb300.build import build

ROW = {MLA_KV_BF16: 1152, MLA_KV_FP8_E4M3: 656, MLA_KV_INT4: 416}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return _lib.load_library()


# ------------------------------------------------------------------ refusals (CPU)
def _good(T=4, H=3, B=2):
    import torch
    p = MlaPoolParams.make(B, 6, 3, kv_dtype=MLA_KV_INT4)
    x, q = torch.zeros(T, 576, dtype=torch.bfloat16), torch.zeros(T, H, 192, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    args = [p, x[:, :512], x[:, 512:], torch.zeros(50, 64), i32(B + 1), i32(B), i32(B, 3), torch.zeros(6, 64, 416, dtype=torch.uint8)]
    return args, dict(q_rope=q[..., 128:], q_out=torch.zeros(T, H, 64, dtype=torch.bfloat16), positions=i32(T), norm_weight=torch.zeros(512, dtype=torch.bfloat16),
                      served=i32(B))


def test_calls_refuse_bad_arguments():
    import torch
    args, kw = _good()
    bad = [({1: args[1][:, :500]}, {}), ({1: args[1].float()}, {}), ({2: args[2][:2]}, {}), ({2: None}, {}), ({3: args[3][:, :32]}, {}), ({3: args[3].double()}, {}),
           ({3: args[3][:0]}, {}), ({4: args[4][:2]}, {}), ({5: args[5].long()}, {}), ({6: args[6].T}, {}), ({7: args[7][:5]}, {}), ({7: None}, {}),
           ({}, dict(q_rope=kw["q_rope"][:2])), ({}, dict(q_rope=kw["q_rope"][..., :32])), ({}, dict(q_rope=kw["q_rope"].float())), ({}, dict(q_out=kw["q_out"][:, :2])),
           ({}, dict(q_out=kw["q_rope"])), ({}, dict(q_rope=None)), ({}, dict(positions=kw["positions"][:3])), ({}, dict(positions=kw["positions"].long())),
           ({}, dict(norm_weight=kw["norm_weight"][:100])), ({}, dict(norm_weight=kw["norm_weight"].float())), ({}, dict(served=kw["served"][:1])),
           ({}, dict(norm_eps=-1.0)), ({}, dict(norm_eps=math.nan))]
    for at, over in bad:
        with pytest.raises(MlaError) as e:
            _lib.mla_append_rotated_kv(*[at.get(i, a) for i, a in enumerate(args)], **dict(kw, **over), stream=0)
        assert e.value.status == _lib.MLA_ERR_INVALID_ARG, (at.keys(), over.keys())
    # q_out over a part of the queries that it is made from
    both = torch.zeros(8, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(MlaError, match="overlaps"):
        _lib.mla_append_rotated_kv(*args, **dict(kw, q_rope=both[:4], q_out=both[1:5]), stream=0)
    with pytest.raises(MlaError, match="device"):   # tensors of the host, last of all
        _lib.mla_append_rotated_kv(*args, **kw, stream=0)
    # nothing to do: no launch
    args, kw = _good(T=0)
    assert _lib.mla_append_rotated_kv(*args, **kw, stream=0).shape == (0, 3, 64)


def test_library_refuses_bad_pointers_and_strides():
    lib = _lib.load_library()
    p = MlaPoolParams.make(2, 6, 3, kv_dtype=MLA_KV_INT4)
    buf = ctypes.create_string_buffer(4096)
    g = (ctypes.addressof(buf) + 255) // 256 * 256
    good = dict(max_tokens=4, latent_stride=576, rope_stride=576, q_token_stride=576, q_head_stride=192, num_heads=3, interleaved=0, max_positions=9, norm_eps=1e-6)
    make = lambda **kw: MlaRotateParams(*[dict(good, **kw)[n] for n, _ in MlaRotateParams._fields_[:-1]])  # noqa: E731
    ptrs = [g] * 12
    call = lambda r, a: lib.mla_append_rotated_kv(ctypes.byref(p), ctypes.byref(r) if r else None, *a, 0)  # noqa: E731
    # latent, k_rope, norm_weight, cos_sin, positions, q_rope, q_out, cu, lens, table, served, pages
    for k in range(12):
        for bad in ((0,) if k not in (2, 4, 10) else ()) + (g + 2,):
            assert call(make(), ptrs[:k] + [bad] + ptrs[k + 1:]) == _lib.MLA_ERR_INVALID_ARG, (k, bad - g)
    for kw in (dict(max_tokens=-1), dict(latent_stride=504), dict(latent_stride=580), dict(rope_stride=56), dict(rope_stride=66), dict(q_token_stride=4),
               dict(q_head_stride=-8), dict(num_heads=-1), dict(interleaved=2), dict(max_positions=0), dict(norm_eps=-1.0), dict(norm_eps=math.inf)):
        assert call(make(**kw), ptrs) == _lib.MLA_ERR_INVALID_ARG, kw
    assert call(make(num_heads=70000), ptrs) == _lib.MLA_ERR_UNSUPPORTED
    assert call(None, ptrs) == _lib.MLA_ERR_INVALID_ARG
    r = make()
    r.reserved[1] = 1
    assert call(r, ptrs) == _lib.MLA_ERR_INVALID_ARG
    assert call(make(max_tokens=0), ptrs) == _lib.MLA_OK


def test_the_table():
    """Far positions: a float32 angle would be off by hundredths."""
    t = _lib.mla_rope_table(200001, device="cpu").double().numpy()
    for pos in (0, 1, 77, 131071, 200000):
        for i in (0, 1, 13, 31):
            a = pos * 10000.0 ** (-i / 32)
            assert abs(t[pos, i] - math.cos(a)) < 2 ** -24 + 1e-9 and abs(t[pos, 32 + i] - math.sin(a)) < 2 ** -24 + 1e-9
    assert _lib.mla_rope_table(4, theta=500.0, device="cpu").shape == (4, 64)


# ------------------------------------------------------------------ the kernel (GPU)
class Case:
    def __init__(self, n, L, H, kv, seed=0, pad=0, strided=True, sigma=1.0):
        import torch
        rng = np.random.default_rng(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.n, self.L, self.H, self.kv = np.asarray(n), np.asarray(L), H, kv
        P, self.bt = place(rng, self.L)
        self.T, self.rows = int(self.n.sum()), int(self.n.sum()) + pad
        bf = lambda *s: (torch.randn(*s, device="cuda", generator=g) * sigma).to(torch.bfloat16)  # noqa: E731
        x = bf(max(self.rows, 1), 576)[:self.rows]
        self.lat, self.rope = (x[:, :512], x[:, 512:]) if strided else (x[:, :512].contiguous(), x[:, 512:].contiguous())
        q = bf(max(self.rows, 1), H, 192 if strided else 64)[:self.rows]
        self.q = q[..., 128:] if strided else q
        self.weight = (1 + 0.2 * torch.randn(512, device="cuda", generator=g)).to(torch.bfloat16)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        self.cu, self.lens, self.table = dev(np.concatenate([[0], np.cumsum(self.n)])), dev(self.L), dev(self.bt)
        self.pool = torch.randint(0, 256, (P, 64, ROW[kv]), device="cuda", generator=g, dtype=torch.uint8)
        self.p = MlaPoolParams.make(len(n), P, self.bt.shape[1], kv_dtype=kv)
        self.seq = np.repeat(np.arange(len(n)), self.n)
        self.row = np.concatenate([np.arange(l - k, l) for k, l in zip(self.n, self.L)]).astype(np.int64) if self.T else np.zeros(0, np.int64)
        self.at = (self.bt[self.seq, self.row // 64], self.row % 64)

    def call(self, **kw):
        import torch
        kw.setdefault("cos_sin", _lib.mla_rope_table(int(self.L.max()) + 1))
        out = torch.full((self.rows, self.H, 64), 7.0, dtype=torch.bfloat16, device="cuda") if self.H else None
        got = _lib.mla_append_rotated_kv(self.p, self.lat, self.rope, kw.pop("cos_sin"), self.cu, self.lens, self.table, self.pool,
                                         q_rope=self.q if self.H else None, q_out=kw.pop("q_out", out), **kw)
        torch.cuda.synchronize()
        return got


def _turned(x, pos, interleaved, theta=10000.0):
    """(float64 rotation of x [..., 64] at positions [T], |x| + |y| of each value's pair)."""
    x = x.double().cpu().numpy()
    a = pos[:, None] * theta ** (-np.arange(32) / 32.0)
    c, s = np.cos(a), np.sin(a)
    if x.ndim == 3:
        c, s = c[:, None], s[:, None]
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y, z, w = u * c - v * s, v * c + u * s, np.abs(u) + np.abs(v)
    join = (lambda a, b: np.stack([a, b], -1).reshape(x.shape)) if interleaved else (lambda a, b: np.concatenate([a, b], -1))
    return join(y, z), join(w, w)


def _near(got, ref, size):
    got = got.double().cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * size).all(), float(np.abs(got - ref).max())


RAGGED = [([1], [1], 0), ([3, 0, 2, 9], [3, 77, 130, 300], 2), ([1] * 40, list(range(60, 100)), 1), ([70, 1, 0, 130], [70, 64, 5, 700], 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_INT4])
@pytest.mark.parametrize("H", [0, 1, 7, 16, 40, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_rows_and_queries(kv, H, interleaved, case):
    import torch
    n, L, pad = RAGGED[case]
    s = Case(n, L, H, kv, seed=case + H, pad=pad, strided=case != 1)
    before = s.pool.clone()
    q = s.call(interleaved=interleaved)
    assert _lib.mla_device_error(clear=True) == 0
    pg, r = (torch.from_numpy(np.asarray(v, np.int64)).cuda() for v in s.at)
    raw = s.pool[pg, r]
    _near(raw[:, ROW[kv] - 128:].contiguous().view(torch.bfloat16), *_turned(s.rope[:s.T], s.row, interleaved))
    if H:
        _near(q[:s.T], *_turned(s.q[:s.T], s.row, interleaved))
        assert (q[s.T:] == 7).all()
    # the latent as the writer of its format has it; everything else as it was
    want = torch.cat([s.lat[:s.T], s.rope[:s.T]], 1).contiguous()
    if kv == MLA_KV_BF16:
        want = want.view(torch.uint8)
    else:
        out = torch.empty(s.T, ROW[kv], dtype=torch.uint8, device="cuda")
        (_lib.mla_quantize_kv_fp8 if kv == MLA_KV_FP8_E4M3 else _lib.mla_quantize_kv_int4)(want, out, s.T)
        want = out
    assert torch.equal(raw[:, :ROW[kv] - 128], want[:, :ROW[kv] - 128])
    before[pg, r] = raw
    assert torch.equal(s.pool, before)


@pytest.mark.gpu
@pytest.mark.parametrize("sigma", [1e-3, 1.0, 300.0])
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_INT4])
def test_norm(kv, sigma):
    import torch
    n, L = [5, 0, 33, 1], [5, 9, 200, 64]
    s = Case(n, L, 16, MLA_KV_BF16, seed=3, sigma=sigma)
    s.call(norm_weight=s.weight, norm_eps=1e-6)
    pg, r = (torch.from_numpy(np.asarray(v, np.int64)).cuda() for v in s.at)
    normed = s.pool[pg, r].contiguous().view(torch.bfloat16)
    x = s.lat.double().cpu().numpy()
    ref = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6) * s.weight.double().cpu().numpy()
    assert (np.abs(normed[:, :512].double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(ref)).all()
    if kv == MLA_KV_BF16:
        return
    t = Case(n, L, 16, kv, seed=3, sigma=sigma)
    t.call(norm_weight=t.weight, norm_eps=1e-6)
    want = torch.empty(s.T, ROW[kv], dtype=torch.uint8, device="cuda")
    (_lib.mla_quantize_kv_fp8 if kv == MLA_KV_FP8_E4M3 else _lib.mla_quantize_kv_int4)(normed.contiguous(), want, s.T)
    pg, r = (torch.from_numpy(np.asarray(v, np.int64)).cuda() for v in t.at)
    assert torch.equal(t.pool[pg, r], want)
    assert _lib.mla_device_error(clear=True) == 0


@pytest.mark.gpu
def test_positions_of_the_callers_own_and_in_place():
    """Positions far out and in any order; queries rotated where they are."""
    import torch
    s = Case([6, 4], [10, 70], 20, MLA_KV_INT4, seed=5, strided=False)
    pos = np.array([0, 199999, 5, 5, 131072, 7, 1, 65536, 3, 100000])
    q0 = s.q.clone()
    table = _lib.mla_rope_table(200000)
    got = s.call(cos_sin=table, positions=torch.from_numpy(pos.astype(np.int32)).cuda(), q_out=s.q)
    assert got.data_ptr() == s.q.data_ptr() and _lib.mla_device_error(clear=True) == 0
    _near(got, *_turned(q0, pos, False))
    pg, r = (torch.from_numpy(np.asarray(v, np.int64)).cuda() for v in s.at)
    _near(s.pool[pg, r][:, 288:].contiguous().view(torch.bfloat16), *_turned(s.rope, pos, False))


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [2, 33, 700])
def test_tokens_that_are_not_served(batch):
    import torch
    rng = np.random.default_rng(batch)
    n, past = rng.integers(0, 4, batch), rng.integers(4, 90, batch)
    n[0] = 2
    s = Case(n, past + n, 16, MLA_KV_INT4, seed=batch)
    served = rng.integers(0, 2, batch).astype(np.int32)
    served[:2] = [1, 0]
    before = s.pool.clone()
    q = s.call(served=torch.from_numpy(served).cuda())
    assert _lib.mla_device_error(clear=True) == 0
    on = torch.from_numpy(served[s.seq] == 1).cuda()
    assert (q[~on] == 7).all() and not (q[on] == 7).all(-1).any()
    pg, r = (torch.from_numpy(np.asarray(v, np.int64)).cuda() for v in s.at)
    assert torch.equal(s.pool[pg[~on], r[~on]], before[pg[~on], r[~on]])
    _near(s.pool[pg[on], r[on]][:, 288:].contiguous().view(torch.bfloat16), *_turned(s.rope[on], s.row[on.cpu().numpy()], False))


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "row", "position", "table"])
def test_tokens_that_cannot_be_placed(what):
    """A page outside the pool, a row past the block table, a position outside the table: reported, the token left out, the
    others as without it."""
    import torch
    s, w = (Case([2, 1, 3], [66, 40, 192], 16, MLA_KV_INT4, seed=7) for _ in range(2))
    want_q = w.call()
    kw = {}
    if what == "page":
        s.table[0, 1] = s.p.num_pages
        lost = [0, 1]
    elif what == "row":
        s.lens[2] += 1  # rows 190 .. 192: the last one lies past the table
        lost = [5]
    elif what == "position":
        pos = torch.from_numpy(s.row.astype(np.int32)).cuda()
        pos[2] = -1
        kw["positions"], lost = pos, [2]
    else:
        kw["cos_sin"], lost = _lib.mla_rope_table(65), [1, 3, 4, 5]
    q = s.call(**kw)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_INVALID_ARG
    keep = [t for t in range(6) if t not in lost]
    assert (q[lost] == 7).all()
    if what == "row":
        keep = [0, 1, 2]
    assert torch.equal(q[keep], want_q[keep])
    pg, r = (torch.from_numpy(np.asarray(v, np.int64)).cuda() for v in s.at)
    assert torch.equal(s.pool[pg[keep], r[keep]], w.pool[pg[keep], r[keep]])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_INT4])
def test_a_step_of_a_layer(kv):
    """reserve, append with rotation, decode, captured into a graph on another stream and replayed: what the calls give one by
    one, and what plain rows give that were rotated beforehand."""
    import torch
    B, H, M, P = 5, 16, 6, 40
    pp = MlaPoolParams.make(B, P, M, kv_dtype=kv)
    keeper = _lib.PagePool(pp)
    g = torch.Generator("cuda").manual_seed(1)
    bf = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    table, weight = _lib.mla_rope_table(M * 64), bf(512) * 0.1 + 1
    first, more = [100, 7, 64, 0, 250], [1] * B
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = lambda n: i32(np.concatenate([[0], np.cumsum(n)]).tolist())  # noqa: E731
    x0, x1, qn, qr = bf(sum(first), 576), bf(B, 576), bf(B, 1, H, 512), bf(B, H, 192)[..., 128:]
    cu0, cu1, n0, n1 = cu(first), cu(more), i32(first), i32(more)

    def start():
        bt, lens, ref = keeper.new_tables()
        pool = torch.zeros(P, 64, ROW[kv], dtype=torch.uint8, device="cuda")
        served = keeper.reserve(n0, bt, lens, ref)
        _lib.mla_append_rotated_kv(pp, x0[:, :512], x0[:, 512:], table, cu0, lens, bt, pool, norm_weight=weight, interleaved=True, served=served)
        return bt, lens, ref, pool

    dec = _lib.Decoder(_lib.MlaDecodeParams.make(B, 1, H, P, M, kv_dtype=kv, out_dtype=_lib.MLA_OUT_F32))
    out, lse = dec.new_outputs()
    q = torch.empty(B, H, 64, dtype=torch.bfloat16, device="cuda")

    def step(bt, lens, ref, pool):
        served = keeper.reserve(n1, bt, lens, ref)
        _lib.mla_append_rotated_kv(pp, x1[:, :512], x1[:, 512:], table, cu1, lens, bt, pool, q_rope=qr, q_out=q, norm_weight=weight, interleaved=True,
                                   served=served)
        dec.plan(lens)
        dec.decode(qn, q.view(B, 1, H, 64), pool, bt, lens, SCALE, out=out, lse=lse)

    state = start()
    step(*state)
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    want = [t.clone() for t in (out, lse, q, *state)]
    # plain rows that were normed and rotated beforehand
    state = start()
    keeper.reserve(n1, *state[:3])
    x = x1[:, :512].float()
    lat = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * weight.float()).to(torch.bfloat16)
    rope = torch.from_numpy(_turned(x1[:, 512:], np.array(first), True)[0]).cuda().to(torch.bfloat16)
    _lib.mla_append_kv(pp, lat, rope, cu1, state[1], state[0], state[3])
    dec.plan(state[1])
    turned = torch.from_numpy(_turned(qr, np.array(first), True)[0]).cuda().to(torch.bfloat16)
    o, l = dec.decode(qn, turned.view(B, 1, H, 64), state[3], state[0], state[1], SCALE)
    assert (o - want[0]).norm() <= 1e-2 * o.norm() and (l - want[1]).abs().max() <= 1e-2
    # captured
    state = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(*state)
    for t, v in zip(state, start()):
        t.copy_(v)
    out.zero_(), q.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    for t, v in zip((out, lse, q, *state), want):
        assert torch.equal(t, v)


def test_queries_are_not_written_over_the_rows():
    """q_out over latent or k_rope, which other warps read in the same launch; a place between strided rows is nobody's."""
    import torch
    args, kw = _good()
    x = torch.zeros(4, 2048, dtype=torch.bfloat16)
    args[1], args[2] = x[:, :512], x[:, 512:576]
    flat = x.view(-1)
    one = lambda at, T=4: flat[at:at + T * 192].view(T, 3, 64)  # noqa: E731
    for at in (0, 64, 504, 512, 568, 1984, 2048 * 3 + 512 - 8):
        with pytest.raises(MlaError, match="overlaps"):
            _lib.mla_append_rotated_kv(*args, **dict(kw, q_out=one(at)), stream=0)
    for at in (576, 2048 - 768, 2048 * 3 + 576):
        with pytest.raises(MlaError, match="device"):
            _lib.mla_append_rotated_kv(*args, **dict(kw, q_out=one(at)), stream=0)


def test_where_a_buffer_meets_strided_rows():
    rng = np.random.default_rng(4)
    hits = 0
    for _ in range(4000):
        rows, width, gap, first, size = (int(v) for v in rng.integers([1, 1, 0, 0, 1], [6, 9, 12, 40, 20]))
        at = int(rng.integers(0, 110))
        want = any(at < first + i * (width + gap) + width and first + i * (width + gap) < at + size for i in range(rows))
        assert _lib._meets(at, size, first, rows, width + gap, width) == want, (at, size, first, rows, width, gap)
        hits += want
    assert 500 < hits < 3500


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 64, 1000, 10000])
@pytest.mark.parametrize("sigma", [1e-3, 1.0, 300.0])
def test_the_norms_last_bit(T, sigma):
    """The squares are summed in a fixed order, four neighbours at a time: over the rows' quarters, over the four, then over the lanes.
    A norm in elementary float32 operations in that order has the same bits, and so has one over torch's mean of a row."""
    import torch
    s = Case([T], [T], 0, MLA_KV_BF16, seed=T, sigma=sigma)
    s.call(norm_weight=s.weight, norm_eps=1e-6)
    assert _lib.mla_device_error(clear=True) == 0
    pg, r = (torch.from_numpy(np.asarray(v, np.int64)).cuda() for v in s.at)
    got = s.pool[pg, r].contiguous().view(torch.bfloat16)[:, :512]
    x = s.lat.float()
    sq = x.square().view(T, 4, 32, 4)                       # quarter, lane, neighbour (a bf16's square is exact in float32)
    part = sq[:, 0]
    for k in (1, 2, 3):
        part = part + sq[:, k]
    lane = ((part[..., 0] + part[..., 1]) + part[..., 2]) + part[..., 3]
    while lane.shape[1] > 1:
        lane = lane[:, 0::2] + lane[:, 1::2]
    for mean in (lane / 512, x.square().mean(1, keepdim=True)):
        want = (x * torch.rsqrt(mean + 1e-6) * s.weight.float()).to(torch.bfloat16)
        assert torch.equal(got, want), int((got != want).any(1).sum())
