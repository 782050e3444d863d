"""4-bit rows read back with scales of the caller's own."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import fp4_ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BITS = {"f16": (11, -24, 2.0 ** 16), "bf16": (8, -133, 2.0 ** 128), "f32": (24, -149, 2.0 ** 128)}


def rounded(v, dtype):
    """float64 values to the nearest of the type (ties to even), as float64."""
    digits, least, over = BITS[dtype]
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - digits, least))
    with np.errstate(invalid="ignore"):
        r = np.rint(v / step) * step
        return np.where(np.abs(r) >= over, np.copysign(np.inf, r), r)


def read_back(codes, unit, scale, block, byte, dtype):
    """Bytes of codes' values (with signs) and scale bytes, read back with the rows' scales, and what they stand for."""
    rows, cols = codes.shape
    sign = np.signbit(codes).astype(np.uint8) * 8
    nibble = np.searchsorted(fp4_ref.CODES, np.abs(codes)).astype(np.uint8) + sign
    q = nibble[:, 0::2] + nibble[:, 1::2] * 16
    tiles = fp4_ref.tiles(byte)
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    got = ms.dequantize_rows_fp4(dev(q), dev(tiles), dev(scale.astype(np.float32)), block=block, out_dtype=DT[dtype])
    want = rounded(codes * np.repeat(unit, block, axis=1) * scale.astype(np.float64)[:, None], dtype)  # 30 bits: exact
    return got.double().cpu().numpy(), want


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_rounded_once(dtype, block):
    """Row scales that are no powers of two, among them such that a product in fp32 falls on a 16-bit border."""
    rng = np.random.default_rng(block)
    rows, cols = 6000, 64
    codes = rng.choice(fp4_ref.CODES, size=(rows, cols)) * rng.choice([-1.0, 1.0], size=(rows, cols))
    codes[:, 0] = rng.choice(fp4_ref.CODES[1:], size=rows)
    if block == 16:
        byte = rng.integers(8, 127, size=(rows, cols // block)).astype(np.uint8)  # without NaN
        unit = torch.from_numpy(byte).view(torch.float8_e4m3fn).double().numpy()
    else:
        byte = rng.integers(120, 135, size=(rows, cols // block)).astype(np.uint8)
        unit = np.ldexp(1.0, byte.astype(np.int64) - 127)
    # borders between neighbours of the 16-bit types
    digits = BITS["bf16" if dtype == "f32" else dtype][0]
    border = (2 * rng.integers(2 ** (digits - 1), 2 ** digits, size=rows) + 1) * 2.0 ** -digits
    scale = (border / (codes[:, 0] * unit[:, 0])).astype(np.float32)
    step = rng.integers(-1, 2, size=rows)
    scale = np.where(step == 0, scale, np.nextafter(scale, np.where(step > 0, np.inf, -np.inf).astype(np.float32)))
    scale[::5] = -scale[::5]
    scale[::7] *= np.float32(2.0 ** -20)  # f16: subnormal values
    got, want = read_back(codes, unit, scale, block, byte, dtype)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_scales_at_the_ends_of_the_range(dtype):
    """E8M0 bytes whose product with a code leaves fp32's range, with row scales that bring it back; subnormal row scales."""
    rng = np.random.default_rng(3)
    rows, cols = 400, 96
    codes = rng.choice(fp4_ref.CODES, size=(rows, cols)) * rng.choice([-1.0, 1.0], size=(rows, cols))
    byte = rng.integers(248, 255, size=(rows, 3)).astype(np.uint8)
    byte[200:] = rng.integers(0, 8, size=(200, 3))
    byte[::10, 1] = 127
    scale = np.float32(2.0) ** rng.integers(-140, 0, size=rows).astype(np.float32)
    scale[1::2] *= rng.uniform(1, 2, size=rows // 2).astype(np.float32)
    scale[200:] = (np.float32(2.0) ** rng.integers(-20, 127, size=200) * rng.uniform(1, 1.9, size=200)).astype(np.float32)
    scale[390:] = 0
    got, want = read_back(codes, np.ldexp(1.0, byte.astype(np.int64) - 127), scale, 32, byte, dtype)
    assert np.array_equal(got, want)
    byte = rng.integers(0, 127, size=(rows, 6)).astype(np.uint8)
    scale = np.ldexp(rng.uniform(1, 2, size=rows), rng.integers(-149, 128, size=rows)).astype(np.float32)
    scale[np.isinf(scale)] = 1
    unit = torch.from_numpy(byte).view(torch.float8_e4m3fn).double().numpy()
    got, want = read_back(codes, unit, scale, 16, byte, dtype)
    assert np.array_equal(got, want)
