"""The paged cache's upkeep (append, copy, fork, reserve, free, compact): refusals on the CPU, the kernels
against a plain model of the tables on the GPU, and a serving run of all of them with the attention.

Everything here moves bytes or counts, so results are compared for equality; the FP8 rows that append
writes are those of mla_quantize_kv_fp8, byte for byte."""
import math

import numpy as np
import pytest

from mla_absorbed_decode_02_gb300 import _lib
from mla_absorbed_decode_02_gb300._lib import MLA_KV_BF16, MLA_KV_FP8_E4M3, MlaError, MlaPoolParams
from mla_absorbed_decode_02_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return _lib.load_library()


def _params(**kw):
    base = dict(batch=6, num_pages=32, max_pages_per_seq=8, kv_dtype=MLA_KV_FP8_E4M3, num_layers=2)
    base.update(kw)
    return MlaPoolParams.make(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), _lib.MLA_ERR_INVALID_ARG), (dict(num_pages=0), _lib.MLA_ERR_INVALID_ARG),
    (dict(max_pages_per_seq=0), _lib.MLA_ERR_INVALID_ARG), (dict(num_layers=0), _lib.MLA_ERR_INVALID_ARG),
    (dict(num_layers=20000), _lib.MLA_ERR_UNSUPPORTED), (dict(kv_dtype=5), _lib.MLA_ERR_INVALID_ARG),
    (dict(page_size=16), _lib.MLA_ERR_UNSUPPORTED), (dict(layer_stride=-16), _lib.MLA_ERR_INVALID_ARG),
    (dict(layer_stride=32 * 64 * 656 - 16), _lib.MLA_ERR_INVALID_ARG), (dict(layer_stride=32 * 64 * 656 + 8), _lib.MLA_ERR_INVALID_ARG),
    (dict(num_pages=1 << 26), _lib.MLA_ERR_UNSUPPORTED),
])
def test_bad_params(kw, status):
    with pytest.raises(MlaError) as e:
        _lib.mla_pool_workspace_size(_params(**kw), 4)
    assert e.value.status == status


def test_workspace_and_reserved():
    assert _lib.mla_pool_workspace_size(_params(), 0) % 256 == 0
    assert _lib.mla_pool_workspace_size(_params(num_pages=1000), 0) >= 4 * (4 + 1000 + 2 * 501)
    assert _lib.mla_pool_workspace_size(_params(), 5000) >= 4 * (2 * 5000 + 6)
    with pytest.raises(MlaError):
        _lib.mla_pool_workspace_size(_params(), -1)
    p = _params()
    p.reserved[3] = 1
    with pytest.raises(MlaError):
        _lib.mla_pool_workspace_size(p, 0)


def test_calls_refuse_bad_arguments():
    """Wrong types, shapes, short pools and workspaces: an error before anything is launched."""
    import torch
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    p = _params(num_layers=2)
    pool, bt, lens, ref, ws = torch.zeros(2, 32, 64, 656, dtype=torch.uint8), i32(6, 8), i32(6), i32(32), torch.zeros(8192, dtype=torch.uint8)
    three = i32(3)
    bad = [
        (_lib.mla_copy_pages, (p, pool[:1], three, three)), (_lib.mla_copy_pages, (p, pool, three, three[:2])),
        (_lib.mla_copy_pages, (p, pool, three.long(), three)), (_lib.mla_copy_pages, (p, None, three, three)),
        (_lib.mla_fork_sequences, (p, pool, three, three, bt[:5], lens, ref, three, ws)),
        (_lib.mla_fork_sequences, (p, pool, three, three, bt, lens, ref[:9], three, ws)),
        (_lib.mla_fork_sequences, (p, pool, three, three, bt, lens, ref, three[:1], ws)),
        (_lib.mla_fork_sequences, (p, pool, i32(5000), i32(5000), bt, lens, ref, i32(5000), ws)),  # workspace too small
        (_lib.mla_fork_sequences, (p, pool, three, three, bt, lens, ref, three, None)),
        (_lib.mla_reserve_pages, (p, three, bt, lens, ref, lens, ws)), (_lib.mla_reserve_pages, (p, lens, bt, lens, ref, three, ws)),
        (_lib.mla_reserve_pages, (p, lens, bt.T, lens, ref, lens, ws)),
        (_lib.mla_free_sequences, (p, three.float(), bt, lens, ref)), (_lib.mla_free_sequences, (p, three, bt, i32(7), ref)),
        (_lib.mla_compact_pages, (p, pool, bt, lens, ref, None, ws)), (_lib.mla_compact_pages, (p, pool, bt, lens, ref, i32(1), ws[:100])),
    ]
    x = torch.zeros(4, 576, dtype=torch.bfloat16)
    q = _params(num_layers=1)
    good = [q, x[:, :512], x[:, 512:], i32(7), lens, bt, pool]
    for at, v in ((1, x[:, :500]), (1, x[:, :512].float()), (2, x[:2, 512:]), (2, None), (3, i32(6)), (4, None), (5, bt.long()), (6, pool[0, :5])):
        bad.append((_lib.mla_append_kv, tuple(v if k == at else a for k, a in enumerate(good))))
    for call, args in bad:
        with pytest.raises(MlaError) as e:
            call(*args, stream=0)
        assert e.value.status in (_lib.MLA_ERR_INVALID_ARG, _lib.MLA_ERR_WORKSPACE), call
    # tensors of the host are refused, last of all
    for call, args in ((_lib.mla_copy_pages, (p, pool, three, three)), (_lib.mla_fork_sequences, (p, pool, three, three, bt, lens, ref, three, ws)),
                       (_lib.mla_reserve_pages, (p, lens, bt, lens, ref, lens, ws)), (_lib.mla_free_sequences, (p, three, bt, lens, ref)),
                       (_lib.mla_compact_pages, (p, pool, bt, lens, ref, i32(1), ws)), (_lib.mla_append_kv, tuple(good))):
        with pytest.raises(MlaError, match="device"):
            call(*args, stream=0)
    # nothing to do: no launch
    _lib.mla_copy_pages(p, pool, i32(0), i32(0), stream=0)
    _lib.mla_fork_sequences(p, pool, i32(0), i32(0), bt, lens, ref, i32(0), ws, stream=0)
    _lib.mla_free_sequences(p, i32(0), bt, lens, ref, stream=0)
    _lib.mla_append_kv(q, x[:0, :512], x[:0, 512:], i32(7), lens, bt, pool, stream=0)


def test_library_refuses_bad_pointers_and_strides():
    """The C entries themselves: null and misaligned pointers, negative counts, row strides that the 16-byte
    accesses cannot take."""
    import ctypes
    lib, p = _lib.load_library(), ctypes.byref(_params())
    buf = ctypes.create_string_buffer(4096)
    g = (ctypes.addressof(buf) + 255) // 256 * 256
    calls = {"mla_append_kv": [4, g, 576, g, 576, g, g, g, g, 0], "mla_copy_pages": [g, g, g, 2, 0],
             "mla_fork_sequences": [g, g, g, 2, g, g, g, g, g, 0], "mla_reserve_pages": [g, g, g, g, g, g, 0],
             "mla_free_sequences": [g, 2, g, g, g, 0], "mla_compact_pages": [g, g, g, g, g, g, 0]}
    for name, args in calls.items():
        for k, v in enumerate(args[:-1]):
            for bad in ((0, g + 2) if v == g else (-1,)):
                a = list(args)
                a[k] = bad
                assert getattr(lib, name)(p, *a) == _lib.MLA_ERR_INVALID_ARG, (name, k, bad)
        assert getattr(lib, name)(None, *args) == _lib.MLA_ERR_INVALID_ARG
    for k, stride in ((2, 511), (2, 516), (4, 63), (4, 70)):
        a = list(calls["mla_append_kv"])
        a[k] = stride
        assert lib.mla_append_kv(p, *a) == _lib.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------ a plain model of the pool
class Model:
    """The pool's tables and bytes on the host, with the documented rules written as loops."""

    def __init__(self, p, pool):
        self.p, self.pool = p, pool.copy()
        self.bt = np.full((p.batch, p.max_pages_per_seq), -1, np.int32)
        self.L, self.ref = np.zeros(p.batch, np.int32), np.zeros(p.num_pages, np.int32)

    def free_pages(self):
        return [int(x) for x in np.nonzero(self.ref == 0)[0]]

    def reserve(self, n):
        served, left, short = [], self.free_pages(), False
        for b in range(self.p.batch):
            if n[b] < 0 or self.L[b] < 0 or int(self.L[b]) + int(n[b]) > 64 * self.p.max_pages_per_seq:
                served.append(-2)
                continue
            a, e = -(-int(self.L[b]) // 64), -(-(int(self.L[b]) + int(n[b])) // 64)
            if e - a > 0 and (short or e - a > len(left)):
                short = True
                served.append(0)
                continue
            for j in range(a, e):
                self.bt[b, j] = left.pop(0)
                self.ref[self.bt[b, j]] = 1
            self.L[b] += n[b]
            served.append(1)
        return served

    def fork(self, parents, children):
        L0, bt0, out, left, named = self.L.copy(), self.bt.copy(), [], self.free_pages(), set()
        for a, c in zip(parents, children):
            B = self.p.batch
            if not (0 <= a < B and 0 <= c < B) or L0[c] != 0 or c in named or not 0 <= L0[a] <= 64 * self.p.max_pages_per_seq:
                out.append(-2)
                continue
            named.add(c)
            full, rows = divmod(int(L0[a]), 64)
            own = -1
            if rows:
                if not left:
                    out.append(-3)
                    continue
                own = left.pop(0)
                self.pool[:, own, :rows] = self.pool[:, bt0[a, full], :rows]
                self.ref[own] = 1
            self.bt[c] = -1
            for j in range(full):
                self.bt[c, j] = bt0[a, j]
                self.ref[bt0[a, j]] += 1
            if rows:
                self.bt[c, full] = own
            self.L[c] = L0[a]
            out.append(own)
        return out

    def free(self, ids):
        for b in ids:
            for j in range(-(-int(self.L[b]) // 64)):
                self.ref[self.bt[b, j]] -= 1
                self.bt[b, j] = -1
            self.L[b] = 0

    def compact(self):
        used = int((self.ref != 0).sum())
        for s, d in zip([q for q in range(used, self.p.num_pages) if self.ref[q]], [q for q in range(used) if not self.ref[q]]):
            self.pool[:, d] = self.pool[:, s]
            self.ref[d], self.ref[s] = self.ref[s], 0
            for b in range(self.p.batch):
                row = self.bt[b, :-(-int(self.L[b]) // 64)]
                row[row == s] = d
        return used

    def copy(self, src, dst):
        for s, d in zip(src, dst):
            self.pool[:, d] = self.pool[:, s]


class Both:
    """The model and the device, driven together."""

    def __init__(self, seed=0, gap=0, **kw):
        import torch
        self.p = _params(**kw)
        row = 1152 if self.p.kv_dtype == MLA_KV_BF16 else 656
        layer = self.p.num_pages * 64 * row
        if gap:
            self.p.layer_stride = layer + gap
        rng = np.random.default_rng(seed)
        self.flat = rng.integers(0, 256, self.p.num_layers * (layer + gap), dtype=np.uint8)
        view = self.flat.reshape(self.p.num_layers, -1)[:, :layer].reshape(self.p.num_layers, self.p.num_pages, 64, row)
        self.m = Model(self.p, view)
        self.d = torch.from_numpy(self.flat.copy()).cuda()
        self.dview = self.d.view(self.p.num_layers, -1)[:, :layer].view(self.p.num_layers, self.p.num_pages, 64, row)
        self.gap = self.d.view(self.p.num_layers, -1)[:, layer:].clone()
        self.pool = _lib.PagePool(self.p, max_forks=64)
        self.bt, self.L, self.ref = self.pool.new_tables()

    def dev(self, x):
        import torch
        return torch.tensor(list(x), dtype=torch.int32, device="cuda")

    def tables(self):
        return self.bt, self.L, self.ref

    def reserve(self, n):
        got = self.pool.reserve(self.dev(n), *self.tables())
        assert got.tolist() == self.m.reserve(n)

    def fork(self, parents, children):
        got = self.pool.fork(self.d, self.dev(parents), self.dev(children), *self.tables())
        assert got.tolist() == self.m.fork(parents, children)

    def free(self, ids):
        self.pool.free(self.dev(ids), *self.tables())
        self.m.free(ids)

    def compact(self):
        assert self.pool.compact(self.d, *self.tables()).tolist() == [self.m.compact()]

    def copy(self, src, dst):
        self.pool.copy(self.d, self.dev(src), self.dev(dst))
        self.m.copy(src, dst)

    def check(self, error=0):
        assert _lib.mla_device_error(clear=True) == error
        assert np.array_equal(self.bt.cpu().numpy(), self.m.bt)
        assert np.array_equal(self.L.cpu().numpy(), self.m.L)
        assert np.array_equal(self.ref.cpu().numpy(), self.m.ref)
        assert np.array_equal(self.dview.cpu().numpy(), self.m.pool)
        # the counts are those of the table
        held = self.m.bt[self.m.bt >= 0]
        assert np.array_equal(np.bincount(held, minlength=self.p.num_pages), self.m.ref)
        assert (self.d.view(self.p.num_layers, -1)[:, self.p.num_pages * 64 * (1152 if self.p.kv_dtype == MLA_KV_BF16 else 656):]
                == self.gap).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_FP8_E4M3])
@pytest.mark.parametrize("gap", [0, 4096])
def test_a_pool_through_its_life(kv, gap):
    s = Both(seed=kv, gap=gap, kv_dtype=kv, num_layers=3)
    s.reserve([64, 1, 0, 130, 0, 65])
    s.check()
    s.fork([0, 1, 3], [2, 4, 4])                  # 0 ends on a page boundary; the second name of 4 is refused
    s.check(error=_lib.MLA_ERR_INVALID_ARG)
    s.free([3, 0, 3])                             # named twice
    s.check()
    s.compact()
    s.check()
    s.reserve([3, 63, 64, 200, 0, 1])
    s.fork([], [])
    s.check()
    s.free(range(6))
    s.check()
    s.compact()
    s.check()
    assert (s.ref == 0).all() and (s.bt == -1).all()


@pytest.mark.gpu
def test_forks_that_cannot_be():
    s = Both(num_pages=6)
    s.reserve([70, 10, 0, 0, 0, 0])               # pages 0, 1 | 2; three are free
    s.fork([0, 9, 0, 0, -1, 2, 0, 1], [0, 2, 7, 2, 3, 3, 4, 5])   # busy child, rows out of range, an empty parent
    s.check(error=_lib.MLA_ERR_INVALID_ARG)
    s.free([4])
    s.fork([0, 0], [3, 4])                        # 3 is empty (a fork of nothing); one page is left, then none
    s.check()
    s.free([2])
    s.fork([0, 1], [2, 4])
    s.check()


@pytest.mark.gpu
def test_reserve_when_pages_run_out():
    s = Both(num_pages=7, batch=8)
    s.reserve([64, 65, 0, 1, 0, 0, 10, 0])        # 5 pages
    s.check()
    s.reserve([64, -1, 30, 64, 64 * 9, 0, 20, 1])  # 0: one page, 2: the last one, 3 fails, 6 needs none, 7 fails
    s.check(error=_lib.MLA_ERR_INVALID_ARG)


@pytest.mark.gpu
@pytest.mark.parametrize("pages,batch", [(4096, 40), (4097, 1500), (20000, 2050)])
def test_many_pages_and_sequences(pages, batch):
    """More than one round of every scan: over 4096 pages, over 1024 sequences and forks."""
    rng = np.random.default_rng(pages)
    s = Both(num_pages=pages, batch=batch, num_layers=1, max_pages_per_seq=16)
    s.pool = _lib.PagePool(s.p, max_forks=batch)
    live = batch // 2
    s.reserve([int(x) for x in rng.integers(0, 120, live)] + [0] * (batch - live))
    s.free([int(x) for x in rng.permutation(live)[: live // 3]])
    kids = [b for b in range(batch) if s.m.L[b] == 0][: batch // 2]
    s.fork([int(x) for x in rng.integers(0, live, len(kids))], kids)
    s.reserve([int(x) for x in rng.integers(0, 130, batch)])
    s.free([int(x) for x in rng.permutation(batch)[: batch // 3]])
    s.compact()
    s.check()


@pytest.mark.gpu
def test_copy_and_pages_out_of_range():
    s = Both(num_layers=2)
    s.copy([0, 5, 7, 9], [1, 6, 7, 31])
    s.check()
    s.pool.copy(s.d, s.dev([3, 32, -1]), s.dev([-2, 4, 8]))       # every pair refused
    s.check(error=_lib.MLA_ERR_INVALID_ARG)
    s.pool.free(s.dev([6, -1]), *s.tables())
    s.check(error=_lib.MLA_ERR_INVALID_ARG)
    s.reserve([10, 70, 0, 0, 0, 0])
    for wrong in (-3, 64 * 8 + 1):                 # lengths that cannot be: nothing is touched
        s.L[0] = s.m.L[0] = wrong
        s.pool.free(s.dev([0]), *s.tables())
        s.pool.compact(s.d, *s.tables())
        assert s.pool.reserve(s.dev([1] * 6), *s.tables()).tolist() == s.m.reserve([1] * 6)
        assert s.pool.fork(s.d, s.dev([0]), s.dev([5]), *s.tables()).tolist() == [-2]
        s.check(error=_lib.MLA_ERR_INVALID_ARG)


# ------------------------------------------------------------------ append
def _append_case(kv, n, L, seed, pad=0, strided=True):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    n, L = np.asarray(n), np.asarray(L)
    need = -(-L // 64)
    P = int(need.sum()) + 2
    perm = np.random.default_rng(seed).permutation(P)
    bt = np.full((len(n), max(1, int(need.max()))), -1, np.int32)
    o = 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[o:o + k]
        o += k
    T = int(n.sum()) + pad
    x = (torch.randn(T, 576, device="cuda", generator=g) * torch.rand(T, 1, device="cuda", generator=g) * 30).to(torch.bfloat16)
    row = 1152 if kv == MLA_KV_BF16 else 656
    pool = torch.randint(0, 256, (P, 64, row), device="cuda", generator=g, dtype=torch.uint8)
    lat, rope = (x[:, :512], x[:, 512:]) if strided else (x[:, :512].contiguous(), x[:, 512:].contiguous())
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    p = MlaPoolParams.make(len(n), P, bt.shape[1], kv_dtype=kv)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    at = [(int(bt[b, q // 64]), q % 64) for b in range(len(n)) for q in range(int(L[b] - n[b]), int(L[b]))]
    return p, lat, rope, dev(cu), dev(L), dev(bt), pool, at, x


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_FP8_E4M3])
@pytest.mark.parametrize("n,L,pad", [([1], [1], 0), ([0, 3, 0, 0, 70, 1], [9, 3, 0, 64, 200, 129], 5), ([1] * 33, list(range(1, 34)), 0),
                                     ([2, 0] * 700, [100, 7] * 700, 1), ([0, 0], [5, 5], 3)])
def test_append_writes_the_rows(kv, n, L, pad):
    import torch
    p, lat, rope, cu, lens, bt, pool, at, x = _append_case(kv, n, L, seed=len(n) + kv, pad=pad, strided=len(n) != 33)
    want = pool.clone()
    if at:
        rows = x[:len(at)]
        if kv == MLA_KV_BF16:
            raw = rows.view(torch.uint8)
        else:
            raw = torch.empty(len(at), 656, dtype=torch.uint8, device="cuda")
            _lib.mla_quantize_kv_fp8(rows.contiguous(), raw, len(at))
        pg, r = (torch.tensor(v, device="cuda") for v in zip(*at))
        want[pg, r] = raw
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, pool)
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    assert torch.equal(pool, want)


@pytest.mark.gpu
def test_append_of_values_that_are_not_finite():
    """bf16 bits are kept; in an FP8 tile a NaN reads back as NaN, an infinity makes its tile NaN, and the other
    tiles keep their bytes."""
    import torch
    p, lat, rope, cu, lens, bt, pool, at, x = _append_case(MLA_KV_FP8_E4M3, [3], [10], seed=4)
    want = pool.clone()
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, want)
    x[0, 130], x[1, 300] = float("nan"), float("inf")
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, pool)
    torch.cuda.synchronize()
    value = lambda row: row[:512].view(torch.float8_e4m3fn).float() * row[512:528].view(torch.float32).repeat_interleave(128)  # noqa: E731
    a, b, c = (pool[pg, r] for pg, r in at)
    wa, wb, wc = (want[pg, r] for pg, r in at)
    assert value(a)[130].isnan() and value(a).isnan().sum() == 1
    assert value(b)[256:384].isnan().all() and value(b).isnan().sum() == 128
    assert torch.equal(c, wc) and torch.equal(a[256:512], wa[256:512]) and torch.equal(b[:256], wb[:256])


@pytest.mark.gpu
def test_append_outside_the_table_is_refused():
    import torch
    p, lat, rope, cu, lens, bt, pool, at, x = _append_case(MLA_KV_BF16, [4, 2, 3], [4, 2, 3], seed=6)
    want = pool.clone()
    pg, r = (torch.tensor(v, device="cuda") for v in zip(*at[4:6]))
    want[pg, r] = x[4:6].view(torch.uint8)
    lens[0] = 2                                   # the first two of its four tokens would lie before row 0
    want[at[2][0], 0], want[at[2][0], 1] = x[2].view(torch.uint8), x[3].view(torch.uint8)
    bt[2, 0] = p.num_pages                        # no such page
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, pool)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_INVALID_ARG
    assert torch.equal(pool, want)


@pytest.mark.gpu
def test_append_of_tokens_before_the_first_sequence_is_refused():
    """cu[0] past 0: the tokens before it belong to no sequence and go nowhere; the others are written."""
    import torch
    p, lat, rope, cu, lens, bt, pool, at, x = _append_case(MLA_KV_BF16, [3, 2], [9, 2], seed=8)
    want = pool.clone()
    cu[0], lens[0] = 2, 7                         # one token is left of the first three: row 6
    want[at[0][0], 6] = x[2].view(torch.uint8)
    pg, r = (torch.tensor(v, device="cuda") for v in zip(*at[3:]))
    want[pg, r] = x[3:5].view(torch.uint8)
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, pool)
    assert _lib.mla_device_error(clear=True) == _lib.MLA_ERR_INVALID_ARG
    assert torch.equal(pool, want)


@pytest.mark.gpu
@pytest.mark.parametrize("as_pointer", [False, True])
def test_results_for_another_stream(as_pointer):
    """A call on another stream takes no memory for its result that kernels waiting on the current stream still read."""
    import torch
    p = MlaPoolParams.make(8, 64, 4)
    up = _lib.PagePool(p)
    bt, lens, ref = up.new_tables()
    new = torch.full((8,), 3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    _lib.mla_reserve_pages(p, new, bt, lens, ref, torch.empty_like(new), up.workspace)   # loads the kernel
    torch.cuda.synchronize()
    x = torch.full((8,), 5, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)              # about a tenth of a second
    y = x * 2
    where = x.data_ptr()
    del x                                       # its memory is free to the current stream, after y
    served = up.reserve(new, bt, lens, ref, stream=side.cuda_stream if as_pointer else side)
    assert served.data_ptr() != where
    torch.cuda.synchronize()
    assert (y == 10).all() and (served == 1).all() and (lens == 6).all()
    assert _lib.mla_device_error(clear=True) == 0


# ------------------------------------------------------------------ together
@pytest.mark.gpu
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_FP8_E4M3])
def test_a_serving_run(kv):
    """Prompts arrive, are forked, go on separately, one ends, the pool is compacted and the rest goes on: after
    every step the attention over the shared pages equals, bit for bit, the attention over a private pool that
    holds each sequence's rows alone."""
    import torch
    B, H, P, M = 6, 16, 40, 8
    g = torch.Generator("cuda").manual_seed(kv)
    p = MlaPoolParams.make(B, P, M, kv_dtype=kv)
    up = _lib.PagePool(p)
    bt, L, ref = up.new_tables()
    row = (576, torch.bfloat16) if kv == MLA_KV_BF16 else (656, torch.uint8)
    pool = torch.zeros(P, 64, row[0], dtype=row[1], device="cuda")
    alone_pool = torch.zeros(B * M, 64, row[0], dtype=row[1], device="cuda")
    alone_bt = torch.arange(B * M, dtype=torch.int32, device="cuda").view(B, M)
    held = [torch.zeros(0, 576, dtype=torch.bfloat16, device="cuda") for _ in range(B)]   # the model: rows of each sequence
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(n):
        T = sum(n)
        x = torch.randn(T, 576, device="cuda", generator=g).to(torch.bfloat16)
        q = torch.randn(T, H, 512, device="cuda", generator=g).to(torch.bfloat16)
        qr = torch.randn(T, H, 64, device="cuda", generator=g).to(torch.bfloat16)
        cu = dev([0] + list(np.cumsum(n)))
        assert (up.reserve(dev(n), bt, L, ref) == 1).all()
        _lib.mla_append_kv(p, x[:, :512], x[:, 512:], cu, L, bt, pool)
        o = 0
        for b, k in enumerate(n):
            held[b] = torch.cat([held[b], x[o:o + k]])
            o += k
        assert L.tolist() == [len(h) for h in held]
        outs = []
        rows = torch.cat([h for h in held])
        all_cu = dev([0] + list(np.cumsum([len(h) for h in held])))
        _lib.mla_append_kv(MlaPoolParams.make(B, B * M, M, kv_dtype=kv), rows[:, :512], rows[:, 512:], all_cu, L, alone_bt, alone_pool)
        for pages, table in ((pool, bt), (alone_pool, alone_bt)):
            attn = _lib.ChunkAttention(_lib.MlaChunkParams.make(B, T, H, pages.shape[0], M, kv_dtype=kv, max_kv_tokens=B * M * 64))
            attn.plan(cu, L)
            outs.append(attn.attend(q, qr, pages, table, 192 ** -0.5))
        torch.cuda.synchronize()
        assert _lib.mla_device_error(clear=True) == 0
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        assert outs[0][0].isfinite().all()

    step([100, 64, 0, 0, 0, 7])
    assert up.fork(pool, dev([0, 0, 1]), dev([2, 3, 4]), bt, L, ref).tolist()[2] == -1
    for a, c in ((0, 2), (0, 3), (1, 4)):
        held[c] = held[a].clone()
    step([1, 1, 30, 2, 64, 100])
    up.free(dev([0, 5]), bt, L, ref)
    held[0] = held[5] = held[0][:0]
    used = int(up.compact(pool, bt, L, ref))
    assert used == int((ref > 0).sum()) and (ref[:used] > 0).all() and int(bt.max()) == used - 1
    step([3, 70, 1, 5, 0, 66])
    step([1, 1, 1, 1, 1, 1])


@pytest.mark.gpu
def test_upkeep_captured_on_another_stream():
    """fork, reserve, free and compact captured into one graph on a side stream give what plain calls give."""
    import torch
    def drive(s):
        s.pool.free(ids, *s.tables())
        a = s.pool.fork(s.d, par, chi, *s.tables())
        b = s.pool.reserve(new, *s.tables())
        c = s.pool.compact(s.d, *s.tables())
        return a, b, c

    s, t = Both(seed=5, num_layers=2), Both(seed=5, num_layers=2)
    ids, par, chi, new = s.dev([1]), s.dev([0, 3]), s.dev([1, 2]), s.dev([0, 0, 0, 0, 5, 60])
    for x in (s, t):
        x.reserve([100, 70, 0, 130, 0, 30])
    want = drive(s)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        got = drive(t)
    with torch.cuda.stream(side):
        g.replay()
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    for a, b in zip(want + s.tables() + (s.d,), got + t.tables() + (t.d,)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ steps whose pages run out
def test_append_refuses_a_bad_served():
    import ctypes

    import torch
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    p, x = _params(num_layers=1), torch.zeros(4, 576, dtype=torch.bfloat16)
    good = (p, x[:, :512], x[:, 512:], i32(7), i32(6), i32(6, 8), torch.zeros(32, 64, 656, dtype=torch.uint8))
    for served in (i32(5), i32(7), i32(6).long(), i32(12)[::2], i32(6, 1)):
        with pytest.raises(MlaError, match="served") as e:
            _lib.mla_append_kv(*good, stream=0, served=served)
        assert e.value.status == _lib.MLA_ERR_INVALID_ARG
    with pytest.raises(MlaError, match="device"):
        _lib.mla_append_kv(*good, stream=0, served=i32(6))
    buf = ctypes.create_string_buffer(4096)
    g = (ctypes.addressof(buf) + 255) // 256 * 256
    args = [4, g, 576, g, 576, g, g, g, g, g, 0]       # ... block_table, served, kv_pages, stream
    for k, v in enumerate(args[:-1]):
        for bad in ((0, g + 2) if v == g else (-1,)):
            a = list(args)
            a[k] = bad
            assert _lib.load_library().mla_append_served_kv(ctypes.byref(p), *a) == _lib.MLA_ERR_INVALID_ARG, (k, bad)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_FP8_E4M3])
@pytest.mark.parametrize("batch", [1, 31, 32, 33, 700, 2100])
def test_append_leaves_out_what_is_not_served(kv, batch):
    """Only tokens of sequences whose `served` is 1 are written, for every depth of the search; the lengths and
    pages of the others are not looked at."""
    import torch
    rng = np.random.default_rng(batch)
    n = rng.integers(0, 4, batch)
    n[-1] = 2
    served = rng.choice([1, 1, 0, -2], batch)
    served[-1] = 0 if batch == 1 else 1
    p, lat, rope, cu, lens, bt, pool, at, x = _append_case(kv, n, n + rng.integers(0, 100, batch), seed=batch + kv, pad=3)
    want = pool.clone()
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, want)
    d_served = torch.from_numpy(served.astype(np.int32)).cuda()
    plain = pool.clone()
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, plain, served=torch.ones_like(d_served))
    assert torch.equal(plain, want)
    skipped = [a for a, b in zip(at, np.repeat(np.arange(batch), n)) if served[b] != 1]
    if skipped:
        pg, r = (torch.tensor(v, device="cuda") for v in zip(*skipped))
        want[pg, r] = pool[pg, r]
    lens[d_served == -2], bt[d_served == 0] = -5, -1     # neither is read
    _lib.mla_append_kv(p, lat, rope, cu, lens, bt, pool, served=d_served)
    torch.cuda.synchronize()
    assert _lib.mla_device_error(clear=True) == 0
    assert torch.equal(pool, want)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [MLA_KV_BF16, MLA_KV_FP8_E4M3])
def test_a_step_whose_pages_run_out(kv):
    """reserve, append and attention of one step with its token buffers as they were laid out: the sequence that gets
    no page keeps its rows, and those that share pages with it keep theirs; the others' results are those of a pool
    with pages enough."""
    import torch
    B, H, M = 4, 16, 4
    g = torch.Generator("cuda").manual_seed(kv)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    row = (576, torch.bfloat16) if kv == MLA_KV_BF16 else (656, torch.uint8)
    first, second = [128, 0, 70, 5], [3, 9, 100, 30]
    token = lambda n, w: torch.randn(n, *w, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    x1, x2, q, qr = token(203, (576,)), token(142, (576,)), token(142, (H, 512)), token(142, (H, 64))
    cu1, cu2 = dev([0, 128, 128, 198, 203]), dev([0, 3, 12, 112, 142])
    got = {}
    for P in (16, 6):
        p = MlaPoolParams.make(B, P, M, kv_dtype=kv)
        up = _lib.PagePool(p)
        t = up.new_tables()
        bt, L, ref = t
        pool = torch.zeros(P, 64, row[0], dtype=row[1], device="cuda")
        served = up.reserve(dev(first), *t)
        _lib.mla_append_kv(p, x1[:, :512], x1[:, 512:], cu1, L, bt, pool, served=served)
        assert up.fork(pool, dev([0]), dev([1]), *t).tolist() == [-1]    # 1 shares both pages of 0; 5 pages are held
        before = pool.clone()
        served = up.reserve(dev(second), *t)                             # of six pages one is left: 0's
        assert served.tolist() == ([1] * 4 if P == 16 else [1, 0, 0, 1])
        attn = _lib.ChunkAttention(_lib.MlaChunkParams.make(B, 142, H, P, M, kv_dtype=kv, max_kv_tokens=B * M * 64))
        attn.plan(cu2, L)
        _lib.mla_append_kv(p, x2[:, :512], x2[:, 512:], cu2, L, bt, pool, served=served)
        out, lse = attn.attend(q, qr, pool, bt, 192 ** -0.5)
        torch.cuda.synchronize()
        assert _lib.mla_device_error(clear=True) == 0
        got[P] = out, lse
        if P == 6:
            assert L.tolist() == [131, 128, 70, 35]
            for b, rows in ((0, 128), (1, 128), (2, 70), (3, 5)):         # what was cached before the step
                held = bt[b, :-(-rows // 64)].long()
                assert torch.equal(pool[held].flatten(0, 1)[:rows], before[held].flatten(0, 1)[:rows])
    for b in (0, 3):
        for a, e in zip(got[16], got[6]):
            assert torch.equal(a[cu2[b]:cu2[b + 1]], e[cu2[b]:cu2[b + 1]])
