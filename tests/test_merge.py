"""The merge of split partials (mla_combine) alone: partials of any kind put into the workspace, among them such as a row with NaN
leaves.

Tolerance.  out = sum_i w_i o_i with w_i = exp(lse_i - lse), in float32.  lse = M + ln S: the exponentials (2 ulp each) and their sum are
off by (n + 4) 2^-23 relative, so ln S by as much plus 2^-22 |ln S|, and the sum with M by 2^-24 |lse|; with n <= 160 splits and |lse| <= 16 that is
below 2^-15.  A weight's exponent has lse's error and the rounding of a difference of at most 32: 2^-14 in all.  The products and their sum add
n 2^-24.  |out error| <= 2^-13 sum_i w_i |o_i| covers all of it."""
import numpy as np
import pytest

from mla_absorbed_decode_02_gb300 import _lib
from mla_absorbed_decode_02_gb300._lib import MlaDecodeParams
from mla_absorbed_decode_02_gb300.build import build

KINDS = ["numbers", "one NaN", "all NaN", "no keys", "NaN and no keys", "numbers and no keys"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return _lib.load_library()


# (units, lengths): 1 + ceil(units / query blocks) splits are expected, which picks the 4, 8, 16 or 32 column slices
@pytest.mark.gpu
@pytest.mark.parametrize("units,L", [(3, [3000, 2500]), (20, [3000, 2500, 70]), (40, [6000, 4000, 1]), (152, [20000])])
@pytest.mark.parametrize("H", [1, 17, 40])
def test_partials_of_any_kind(units, L, H):
    """A row in which some split has NaN is NaN, in out and lse; one whose splits saw no key gets 0 and -inf; all others are the
    weighted sum, with the same bits whatever their neighbours hold."""
    import torch
    B = len(L)
    p = MlaDecodeParams.make(B, 1, H, 64, 400, num_units=units, out_dtype=_lib.MLA_OUT_F32)
    dec = _lib.Decoder(p)
    dec.plan(torch.tensor(L, dtype=torch.int32, device="cuda"))
    sched = dec.sched.cpu().numpy()
    ns, off = sched[8 + 8 * units:][:B], sched[8 + 8 * units + B:][:B]
    assert (ns > 1).any()
    slots = B + units
    rng = np.random.default_rng([units, H])
    o, lse = rng.standard_normal((slots, H, 512)).astype(np.float32), rng.uniform(-8, 8, (slots, H)).astype(np.float32)
    plain = lse.copy()
    kind = rng.integers(0, len(KINDS), (B, H))
    if H >= len(KINDS):
        kind[:, :len(KINDS)] = np.arange(len(KINDS))
    for b in np.flatnonzero(ns > 1):
        for h in range(H):
            x, name = lse[off[b]:off[b] + ns[b], h], KINDS[kind[b, h]]
            some = rng.permutation(len(x))[:max(1, len(x) // 2)]
            if name == "one NaN":
                x[rng.integers(len(x))] = np.nan
            elif name == "all NaN":
                x[:] = np.nan
            elif name == "no keys":
                x[:] = -np.inf
            elif name == "NaN and no keys":
                x[:] = np.nan
                x[some] = -np.inf
            elif name == "numbers and no keys":
                x[some] = -np.inf
            o[off[b]:off[b] + ns[b], h][np.isneginf(x)] = 0    # (what a split without keys writes)
    at = slots * H * 512
    at_lse = (at * 4 + 255) // 256 * 64

    def merge(parts):
        dec.workspace[:at] = torch.from_numpy(o).cuda().flatten()
        dec.workspace[at_lse:at_lse + slots * H] = torch.from_numpy(parts).cuda().flatten()
        out, total = dec.new_outputs()
        out.fill_(7.0), total.fill_(7.0)
        _lib.mla_combine(p, out, total, dec.sched, dec.workspace)
        torch.cuda.synchronize()
        assert _lib.mla_device_error(clear=True) == 0
        return out[:, 0].cpu().numpy(), total[:, 0].cpu().numpy()

    out, total = merge(lse)
    finite_out, finite_total = merge(plain)
    for b in range(B):
        if ns[b] < 2:
            assert (out[b] == 7).all() and (total[b] == 7).all()     # (the decode's own)
            continue
        for h in range(H):
            x, v = lse[off[b]:off[b] + ns[b], h].astype(np.float64), o[off[b]:off[b] + ns[b], h].astype(np.float64)
            if np.isnan(x).any():
                assert np.isnan(total[b, h]) and np.isnan(out[b, h]).all(), (b, h, KINDS[kind[b, h]])
            elif np.isneginf(x).all():
                assert np.isneginf(total[b, h]) and (out[b, h] == 0).all()
            else:
                want = x.max() + np.log(np.exp(x - x.max()).sum())
                w = np.exp(x - want)[:, None]
                assert abs(total[b, h] - want) <= 2.0 ** -15
                assert (np.abs(out[b, h] - (w * v).sum(0)) <= 2.0 ** -13 * (w * np.abs(v)).sum(0)).all()
            if KINDS[kind[b, h]] == "numbers":
                assert np.array_equal(out[b, h], finite_out[b, h]) and total[b, h] == finite_total[b, h]
