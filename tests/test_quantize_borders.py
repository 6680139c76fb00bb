"""The cache quantiser at the borders between two E4M3 codes: quotients on, just above and just below every
border, tiny ones, and scales over the whole float32 range, byte for byte as IEEE division and rounding to
nearest even give them."""
import numpy as np
import pytest

import mla_workloads as mw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_absorbed_decode_02_gb300.build import build
    build()


def test_every_border():
    """Tiles whose largest value is a (so scale = a / 448) hold the bf16 values around border * scale."""
    import torch
    from mla_absorbed_decode_02_gb300 import mla_quantize_kv_fp8
    rng = np.random.default_rng(1)
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()  # 0 .. 448
    borders = (codes[1:] + codes[:-1]) / 2
    tiles = []
    for a in np.concatenate([np.exp2(rng.uniform(-126, 120, 300)), [1.0, 448.0, 7.0, 2.0 ** -100, 3e-39, 9.2e-41, 3e38]]):
        top = (mw.to_bf16_bits(np.float32([a])).astype(np.uint32) << 16).view(np.float32)[0]
        x = np.zeros((2, 128), np.float32)
        with np.errstate(over="ignore"):
            near = (borders.astype(np.float64) * (float(top) / 448.0)).astype(np.float32)
        bits = mw.to_bf16_bits(near).astype(np.int64)
        for row, shift in ((0, 0), (1, rng.integers(-1, 2, 126))):
            x[row, :126] = (np.clip(bits + shift, 0, 0x7F7F).astype(np.uint32) << 16).view(np.float32) * rng.choice([-1, 1], 126)
            x[row, 126] = top
        x[:, :126] = np.clip(x[:, :126], -top, top)
        tiles.append(x)
    tiles = np.concatenate(tiles)
    tiles = tiles[:len(tiles) // 4 * 4].reshape(-1, 512)
    bits = mw.to_bf16_bits(np.concatenate([tiles, np.zeros((len(tiles), 64), np.float32)], 1))
    ref = mw.quantize_fp8_rows((bits[:, :512].astype(np.uint32) << 16).view(np.float32), bits[:, 512:])
    out = torch.empty((len(bits), 656), dtype=torch.uint8, device="cuda")
    mla_quantize_kv_fp8(torch.from_numpy(bits.view(np.int16)).cuda(), out, len(bits))
    got = out.cpu().numpy()
    assert np.array_equal(got, ref), np.argwhere(got != ref)[:10]


def test_many_random_rows():
    """Two million values: the reciprocal's path and the division's agree with the definition on all of them."""
    import torch
    from mla_absorbed_decode_02_gb300 import mla_quantize_kv_fp8
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(4096, 576, generator=g) * torch.exp(torch.randn(4096, 1, generator=g) * 4)).to(torch.bfloat16)
    bits = x.view(torch.int16).numpy().view(np.uint16)
    ref = mw.quantize_fp8_rows(x[:, :512].float().numpy(), bits[:, 512:])
    out = torch.empty((4096, 656), dtype=torch.uint8, device="cuda")
    mla_quantize_kv_fp8(x.cuda(), out, 4096)
    assert np.array_equal(out.cpu().numpy(), ref)
