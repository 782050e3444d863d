"""The 4-bit product with row scales far from 1 and from one another, exact: the
sums are small whole numbers, and every rounding that is left is restated in 64 bits."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import fp4_ref
from tests.test_gpu_fp4_rows import DT, rounded

pytestmark = pytest.mark.gpu
# tiles of 64, 128 and 256 columns; one of many stages shared by the pairs of a cluster
SHAPES = [(60, 200, 96), (200, 60, 96), (1, 300, 2048), (4000, 1000, 64), (1000, 4000, 64), (2560, 1024, 2048), (1024, 2560, 2048), (2560, 1027, 2048)]


def codes(seed, rows, K):
    """(bytes, block scales of 1, values) of random 4-bit rows in blocks of 32; the first rows are zero."""
    rng = np.random.default_rng(seed)
    v = rng.choice(fp4_ref.CODES, size=(rows, K)) * rng.choice([-1.0, 1.0], size=(rows, K))
    v[:2] = 0
    nibble = np.searchsorted(fp4_ref.CODES, np.abs(v)).astype(np.uint8) + np.signbit(v).astype(np.uint8) * 8
    q = torch.from_numpy(nibble[:, 0::2] + nibble[:, 1::2] * 16).cuda()
    unit = torch.full(((rows + 127) // 128, (K + 127) // 128, 32, 4, 4), 127, dtype=torch.uint8, device="cuda")
    return q, unit, torch.from_numpy(v).cuda()


def digits24(v):
    """Nearest values of 24 bits, of any exponent."""
    _, e = np.frexp(v)
    return np.ldexp(np.rint(np.ldexp(v, 24 - e)), e - 24)


def expected(x, w, sx, sw, dtype):
    dot = (x @ w.T).cpu().numpy()
    with np.errstate(over="ignore"):
        y = rounded(dot * digits24(sx.astype(np.float64)[:, None] * sw.astype(np.float64)), "f32")
        return y if dtype == "f32" else rounded(y, dtype)


def product(M, N, K, sx, sw, dtype, bias=None):
    (qx, ux, x), (qw, uw, w) = codes(M + K, M, K), codes(N, N, K)
    dev = lambda s: torch.from_numpy(s).cuda()  # noqa: E731
    y = ms.linear_fp4(qx, ux, dev(sx), qw, uw, dev(sw), None if bias is None else dev(bias), block=32, out_dtype=DT[dtype])
    return y, x, w


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["near", "opposite", "any"])
def test_far_scales(M, N, K, dtype, kind):
    rng = np.random.default_rng(M * 3 + N)
    reach = {"near": (-10, 10, -10, 10), "opposite": (60, 126, -126, -60), "any": (-126, 127, -126, 127)}[kind]
    sx = np.ldexp(rng.uniform(1, 2, size=M), rng.integers(reach[0], reach[1], size=M)).astype(np.float32)
    sw = np.ldexp(rng.uniform(1, 2, size=N), rng.integers(reach[2], reach[3], size=N)).astype(np.float32)
    if kind == "any":
        sx[::3] = np.ldexp(1.0, rng.integers(-126, 20, size=len(sx[::3]))).astype(np.float32)  # as the quantisation gives them
        sx[5::50], sw[7::50], sw[1::9] = 0, 2.0 ** -149, -sw[1::9]
        sx[4::50] = 2.0 ** -140 * 1.3
    y, x, w = product(M, N, K, sx, sw, dtype)
    assert np.array_equal(y.double().cpu().numpy(), expected(x, w, sx, sw, dtype))


@pytest.mark.parametrize("M,N,K", SHAPES[:2] + SHAPES[3:])
def test_bias_beside_far_scales(M, N, K):
    rng = np.random.default_rng(N)
    sx, sw = np.full(M, 2.0 ** 90, np.float32), np.full(N, 2.0 ** -91, np.float32)
    sx[3::4] = 2.0 ** -126
    bias = rng.integers(-9, 9, size=N).astype(np.float32)
    for out in ("f32", "bf16"):
        y, x, w = product(M, N, K, sx, sw, out, bias)
        dot = (x @ w.T).cpu().numpy()
        want = dot * 0.5 * (sx > 1)[:, None] + bias  # what is left of the small rows is far below a rounding of the bias, but where that is 0
        want = np.where((sx <= 1)[:, None] & (bias == 0), dot * 2.0 ** -126 * 2.0 ** -91, want)
        assert np.array_equal(y.double().cpu().numpy(), rounded(rounded(want, "f32"), out))


def test_either_operand_first():
    """The same bits whichever operand has more rows."""
    for M, N, K in SHAPES[3:]:
        rng = np.random.default_rng(K)
        sx, sw = (np.ldexp(rng.uniform(1, 2, size=n), rng.integers(-9, 9, size=n)).astype(np.float32) for n in (M, N))
        (qx, ux, _), (qw, uw, _) = codes(1, M, K), codes(2, N, K)
        a, b = (qx, ux, torch.from_numpy(sx).cuda()), (qw, uw, torch.from_numpy(sw).cuda())
        one, two = (ms.linear_fp4(*p, *q, block=32, out_dtype=torch.float32) for p, q in ((a, b), (b, a)))
        assert torch.equal(one, two.t())


def test_infinite_and_nan_scales():
    (qx, ux, x), (qw, uw, w) = codes(1, 40, 64), codes(2, 30, 64)
    sx, sw = torch.ones(40, device="cuda"), torch.ones(30, device="cuda")
    sx[3], sx[4], sw[5], sx[9], sw[9] = float("nan"), float("inf"), float("nan"), 2.0 ** 100, 2.0 ** -100
    y = ms.linear_fp4(qx, ux, sx, qw, uw, sw, block=32, out_dtype=torch.float32).double()
    want = (x @ w.t()) * (sx.double()[:, None] * sw.double())
    assert torch.equal(y.isnan(), want.isnan()) and y[3].isnan().all() and y[:, 5].isnan().all()
    assert torch.equal(y.nan_to_num(nan=0.0, posinf=1e300, neginf=-1e300), want.float().double().nan_to_num(nan=0.0, posinf=1e300, neginf=-1e300))
