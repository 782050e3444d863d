"""Sums of the INT8 linear beyond 2^24, where float32 no longer holds every
integer: f32 outputs and sliced products are the exact sum rounded once, in
every kernel and whatever the number of tokens; 16-bit outputs stay within
what one float32 accumulator may lose."""
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import head_ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def codes(g, rows, K, low, high):
    return torch.randint(low, high + 1, (rows, K), generator=g, device="cuda", dtype=torch.int8)


def operands(kind, M, N, K, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(M * 7 + N * 3 + K + seed)
    if kind == "random":
        return codes(g, M, K, -128, 127), codes(g, N, K, -128, 127)
    if kind == "small":                        # |x w| <= 64: sums of magnitudes stay below 2^24 up to the largest K
        return codes(g, M, K, -8, 8), codes(g, N, K, -8, 8)
    if kind == "extreme":                      # every product 2^14
        x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        return x, torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    x, w = codes(g, M, K, 90, 127), codes(g, N, K, 90, 127)
    if kind == "turning":                      # up to the middle of K, and down again
        w[:, K // 2:] *= -1
    return x, w


def product(x, w, dtype):
    one_m, one_n = torch.ones(len(x), device="cuda"), torch.ones(len(w), device="cuda")
    y = ms.linear_int8(x, one_m, w, one_n, out_dtype=DT[dtype])
    assert ms.device_status() == 0
    return y


def exact(x, w):
    return x.double() @ w.double().t()         # every partial sum below 2^53


# Few tokens and small products; tiles of 64, 128 and 256 columns, both ways round, with rows on and off their
# 16-byte boundaries, weights kept in shared memory, K of one part, of two and of more, a part of its own size last;
# K cut into slices of one part and of several, both ways round, N a multiple of four and not.
SHAPES = [(5, 40, 20000), (300, 1500, 640), (2000, 1500, 1024), (9000, 2000, 1024), (2000, 9000, 1024), (20000, 64, 1024),
          (999, 1537, 1111), (9000, 600, 1100), (600, 9000, 1100), (9000, 601, 1152), (1300, 900, 4096), (5000, 2000, 2048),
          (20000, 64, 2048), (20000, 50, 2048), (20000, 128, 2000), (9000, 60, 2112), (9000, 61, 3201), (60, 9000, 2112),
          (300, 121, 9000), (700, 300, 16384), (700, 301, 16384), (2500, 302, 9000), (300, 301, 16384), (130, 300, 131071),
          (300, 130, 131071), (2000, 20, 131071), (2, 20, 131071)]
SLICED = SHAPES[18:26]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["random", "one_signed", "turning", "extreme"])
def test_f32_sums_are_exact(M, N, K, kind):
    x, w = operands(kind, M, N, K)
    assert torch.equal(product(x, w, "f32"), exact(x, w).float())


@pytest.mark.parametrize("M,N,K", SLICED)
@pytest.mark.parametrize("dtype,kind", [("bf16", "one_signed"), ("bf16", "turning"), ("f16", "small")])
def test_sliced_16_bit_sums_are_exact(M, N, K, dtype, kind):
    x, w = operands(kind, M, N, K)
    assert torch.equal(product(x, w, dtype), exact(x, w).float().to(DT[dtype]))


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_sums_below_2_24_are_exact_at_any_length(M, N, K, dtype):
    # sums of magnitudes below 2^24: a block of K that is left out or taken twice cannot hide in a tolerance
    x, w = operands("small", M, N, K)
    assert torch.equal(product(x, w, dtype), exact(x, w).float().to(DT[dtype]))


@pytest.mark.parametrize("M,N,K", [(2000, 1500, 4096), (1500, 2000, 4096), (5000, 2000, 2048), (20000, 64, 2048), (20000, 128, 2000),
                                   (9000, 60, 2112), (60, 9000, 2112), (1300, 900, 16384)])
@pytest.mark.parametrize("kind", ["one_signed", "turning"])
def test_16_bit_sums_of_one_accumulator(M, N, K, kind):
    # each step of 16 products may lose a unit of the last place (2^-23) of the largest partial sum
    x, w = operands(kind, M, N, K)
    y, ref = product(x, w, "bf16").double(), exact(x, w)
    half = K // 2 if kind == "turning" else K
    largest = exact(x[:, :half], w[:, :half]).abs()
    loss = (K + 15) // 16 * 2.0 ** -23 * largest
    assert ((y - ref).abs() <= loss + head_ref.ROUND["bf16"] * (ref.abs() + loss)).all()


@pytest.mark.parametrize("M,N,K", [(3000, 1537, 1111), (300, 3000, 4096), (2000, 128, 2048), (700, 301, 16384)])
@pytest.mark.parametrize("kind", ["random", "one_signed"])
def test_a_token_alone_and_among_others(M, N, K, kind):
    # the same bits from the kernel for few tokens and from the one for many
    x, w = operands(kind, M, N, K)
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    xs, ws = (torch.rand(n, generator=g, device="cuda") for n in (M, N))
    bias = torch.randn(N, generator=g, device="cuda")
    full = ms.linear_int8(x, xs, w, ws, bias, out_dtype=torch.float32)
    for rows in (slice(0, 1), slice(7, 12), slice(M - 16, M)):
        assert torch.equal(ms.linear_int8(x[rows], xs[rows], w, ws, bias, out_dtype=torch.float32), full[rows])
