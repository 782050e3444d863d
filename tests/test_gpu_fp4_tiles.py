"""The 4-bit product through every tile kernel, several tiles for each pair of
SMs: block scales of several sizes and sums that are exact in fp32."""
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests.fp4_shapes import PLANS

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def operand(g, rows, K, block):
    """(bytes, block scales, row scales) and their values in float64: block scales of 0.5, 1 and 2, row scales of 2^-3 to 2^3.

    Products are multiples of 1/16, and of a sum of K = 4096 of them at most 36 * 4 * 4096 * 16 < 2^24."""
    code = torch.randint(0, 16, (rows, K), generator=g, device="cuda", dtype=torch.uint8)
    q = code[:, 0::2] + code[:, 1::2] * 16
    blocks, words = K // block, -(-K // (4 * block))
    e = torch.randint(-1, 2, (rows, blocks), generator=g, device="cuda")
    byte = (e + 127 if block == 32 else 56 + 8 * e).to(torch.uint8)  # E8M0, or E4M3
    full = torch.zeros(-(-rows // 128) * 128, 4 * words, dtype=torch.uint8, device="cuda")
    full[:rows, :blocks] = byte
    tiles = full.view(-1, 4, 32, words, 4).permute(0, 3, 2, 1, 4).contiguous()  # [row tile, word, r % 32, r / 32 % 4, block % 4]
    s = torch.exp2(torch.randint(-3, 4, (rows,), generator=g, device="cuda").float())
    v = CODES.cuda()[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0).double()
    v = v * torch.exp2(e.double()).repeat_interleave(block, dim=1)
    return (q, tiles, s), v


@pytest.mark.parametrize("M,N,K", list(PLANS))
@pytest.mark.parametrize("block", [16, 32])
def test_exact_products(M, N, K, block):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, xv = operand(g, M, K, block)
    w, wv = operand(g, N, K, block)
    bias = torch.randint(-9, 10, (N,), generator=g, device="cuda").float()
    scaled = (xv @ wv.t()) * (x[2].double()[:, None] * w[2].double())
    for with_bias in (False, True):
        want = (scaled + bias.double() if with_bias else scaled).float()
        for dtype in ("f32", "bf16", "f16"):
            # rows in front and behind stay as they are
            buf = torch.full((M + 16, N), 7.0, dtype=DT[dtype], device="cuda")
            y = ms.linear_fp4(*x, *w, bias if with_bias else None, block=block, out_dtype=DT[dtype], out=buf[8:8 + M])
            off = (y != want.to(DT[dtype])).nonzero()
            assert not len(off), f"{dtype}: {len(off)} of {y.numel()} differ, first at {off[0].tolist()}"
            assert (buf[:8] == 7).all() and (buf[8 + M:] == 7).all()
    assert ms.device_status() == 0


@pytest.mark.parametrize("M,N,K", [(8200, 2050, 800), (9000, 1704, 320), (2050, 8200, 800)])
def test_wide_products_are_repeatable_and_replay(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (ms.quantize_rows_fp4(torch.randn(r, K, generator=g, device="cuda")) for r in (M, N))
    want = ms.linear_fp4(*x, *w)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ms.linear_fp4(*x, *w, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert torch.equal(ms.linear_fp4(*x, *w), want)


@pytest.mark.parametrize("M,N,K", [(8200, 2056, 800), (2050, 8200, 800), (9000, 1700, 320), (1700, 9000, 320)])
def test_nan_scales_reach_their_rows_alone(M, N, K):
    """A NaN block scale (block 32) or row scale: its row or column, in tiles of 128 and 256 columns."""
    g = torch.Generator(device="cuda").manual_seed(2)
    for block in (16, 32):
        (q, b, s), _ = operand(g, M, K, block)
        w, _ = operand(g, N, K, block)
        want = ms.linear_fp4(q, b, s, *w, block=block, out_dtype=torch.float32)
        s2, b2 = s.clone(), b.clone()
        s2[M - 1] = float("nan")
        row = 300  # tile 2, word 0, row 12 of 32, second quarter
        b2[row // 128, 0, row % 32, row // 32 % 4, 1] = 255 if block == 32 else 127
        got = ms.linear_fp4(q, b2, s2, *w, block=block, out_dtype=torch.float32)
        assert got[M - 1].isnan().all() and got[row].isnan().all()
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[[row, M - 1]] = False
        assert torch.equal(got[keep], want[keep])
