"""4-bit rows in calls of more rows than the grids hold at once: the same bytes
and values as in calls of few rows, for every group of threads a row may have."""
import pytest
import torch

import maxsim_scoring_gb300 as ms

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# columns, and rows: more than 152 * 8 blocks of 256 threads quantise at a time (two rows in flight), and more than 152 * 16
# read back (four rows), with a part of a tile of 128 rows at the end
SIZES = [(30, 1400003), (64, 700001), (120, 350011), (250, 175003), (500, 88001), (1000, 44003), (1500, 25001), (2000, 22003),
         (2900, 13001), (4000, 11003), (8000, 5501), (16000, 2701), (16400, 2605)]


@pytest.mark.parametrize("cols,rows", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("aligned", [True, False])
def test_rows_as_in_small_calls(cols, rows, dtype, block, aligned):
    g = torch.Generator(device="cuda").manual_seed(rows)
    width = -(-cols // 16) * 16 if aligned else cols + 1 - cols % 2  # odd strides: rows of every phase
    x = torch.empty(rows, width, device="cuda", dtype=DT[dtype]).normal_(generator=g)
    x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda").float()).to(x.dtype)
    x = x[:, :cols]
    q, b, s = ms.quantize_rows_fp4(x, block=block)
    y = ms.dequantize_rows_fp4(q, b, s, block=block, cols=cols, out_dtype=DT[dtype])
    # a single round of either grid
    few = max(128, 152 * 8 * 16 // -(-cols // 16) // 128 * 128)
    for r in range(0, rows, few):
        e = min(rows, r + few)
        part = ms.quantize_rows_fp4(x[r:e], block=block)
        assert torch.equal(part[0], q[r:e]) and torch.equal(part[1], b[r // 128:-(-e // 128)])
        assert part[2] is None or torch.equal(part[2], s[r:e])
        assert torch.equal(ms.dequantize_rows_fp4(*part, block=block, cols=cols, out_dtype=DT[dtype]), y[r:e])
    # what all rows must show: errors of at most half a step of a code, or the cut at 6 (of at most 8 in blocks of 32)
    off = (y.float() - x.float()).abs().amax(dim=1)
    top = x.float().abs().amax(dim=1)
    assert (off <= top * 0.26).all() and (off[top > 0] > 0).float().mean() > 0.9
    assert ms.device_status() == 0
