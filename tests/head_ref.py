"""Plain references of the token head's operators (numpy, float64 and exact
integers), and the error bounds that the GPU tests hold the kernels to."""
import numpy as np

U = 2.0 ** -24                                             # unit roundoff of float32
ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": U}   # of the output types
TINY = {"f16": 2.0 ** -25, "bf16": 0.0, "f32": 0.0}        # half of f16's smallest subnormal
FLT_MIN = np.float32(2.0 ** -126)


def philox4x32_10(block, seed, offset):
    """uint32 words [n, 4] for the counters (block low, block high, offset low, offset high)."""
    mask = np.uint64(0xFFFFFFFF)
    block = np.asarray(block, dtype=np.uint64)
    c = [block & mask, block >> np.uint64(32), np.full_like(block, offset & 0xFFFFFFFF),
         np.full_like(block, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & mask,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1).astype(np.uint32)


def keep_mask(rows, cols, p, seed, offset):
    n = rows * cols
    words = philox4x32_10(np.arange((n + 7) // 8), seed, offset)
    halves = np.stack([words & 0xFFFF, words >> 16], axis=-1).reshape(-1)[:n]
    return (halves >= round(p * 65536)).reshape(rows, cols)


def dropout(x, p, seed, offset, residual=None):
    """(y, bound) in float64 for x [rows, cols] in float64."""
    t = round(p * 65536)
    keep = keep_mask(*x.shape, p, seed, offset)
    kept = np.zeros_like(x)
    kept[keep] = x[keep] * (65536.0 / (65536 - t)) if t < 65536 else 0.0
    y = kept if residual is None else kept + residual
    # the scale and the product are rounded, then the sum
    with np.errstate(invalid="ignore"):
        return y, 3 * U * np.abs(kept) + U * np.abs(y)


def quantize(x, normalize):
    """(q int8, scale float64, relative bound of scale) for float32 x [rows, cols]; q in the definition's float32."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    bad = ~np.isfinite(x).all(axis=1)
    xf = np.where(bad[:, None], np.float32(0), x)
    a = np.abs(xf).max(axis=1) if cols else np.zeros(rows, np.float32)
    s = np.maximum((a * (np.float32(1) / np.float32(127))).astype(np.float32), FLT_MIN)
    y = (xf / s[:, None]).astype(np.float32)
    q = np.clip(np.rint(y), -127, 127).astype(np.int8)
    scale, rel = s.astype(np.float64), np.full(rows, 2 * U)
    if normalize:
        norm = np.sqrt((xf.astype(np.float64) ** 2).sum(axis=1)) / np.maximum(a.astype(np.float64) / 127, 2.0 ** -126)
        scale = np.where(norm > 0, 1.0 / np.where(norm > 0, norm, 1.0), float(FLT_MIN))
        # squares of quotients with 4 roundings each, a sum of cols terms, root and reciprocal
        rel = np.full(rows, (cols / 2 + 12) * U)
    scale[bad] = np.nan
    return q, scale, rel


def linear(x, xs, w, ws, bias):
    """(y float64, bound before the output's rounding) for int8 x, w and float32 scales."""
    xi, wi = x.astype(np.float64), w.astype(np.float64)   # every sum below 2^53: exact
    dot = xi @ wi.T
    y = dot * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    # conversion of the sum, two scale products, the bias
    err = 4 * U * np.abs(y)
    # sums beyond 2^24 may lose a unit of the last place in each 16-wide step
    mag = np.abs(xi) @ np.abs(wi).T
    steps = (x.shape[1] + 15) // 16
    scale = xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    err += np.where(mag >= 2.0 ** 24, steps * 2 * U * mag * scale, 0.0)
    if bias is not None:
        y = y + bias.astype(np.float64)
        err += U * np.abs(y)
    return y, err


def within(got, ref, bound, dtype):
    """Asserts |got - ref| <= bound + the rounding of dtype; NaN and infinities in the same places."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    tol = (bound + ROUND[dtype] * (np.abs(ref) + bound) + TINY[dtype])[fine]
    err = np.abs(got[fine] - ref[fine])
    assert np.all(err <= tol), f"{(err > tol).sum()} of {err.size} values off, worst by {(err / np.maximum(tol, 1e-300)).max():.3g} of the bound"
