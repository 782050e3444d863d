"""Plain reference of the 4-bit floating-point rows (numpy, float64: every
quotient that is rounded here is exact or decided by exact comparisons), and
the bound that the products are held to."""
import numpy as np

CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# E4M3: exponent bias 7, subnormals of 2^-9, 127 is NaN
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)])


def nearest(v, table):
    """Indices of the table's values nearest to v >= 0; the even index of two as near. The comparisons are exact for
    v of up to 40 bits."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    up, down = table[hi] - v, v - table[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def round_quotient(x, d, table):
    """Indices of the table's values nearest to x / d >= 0, decided by x against d times the table's midpoints (products
    and sums of few bits, exact in float64): ties to the even index."""
    mid = (table[1:] + table[:-1]) / 2
    i = np.zeros(x.shape, dtype=np.int64)
    for k, m in enumerate(mid):
        edge = d * m
        i = np.where((x > edge) | ((x == edge) & (k % 2 == 1)), k + 1, i)
    return i


def quantize(x, block):
    """(q uint8 [rows, ceil(cols / 32) * 16], scale bytes [rows, blocks], row scales or None) of float64 x [rows, cols]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    width = (cols + 31) // 32 * 32
    y = np.zeros((rows, width))
    y[:, :cols] = x
    blocks = width // block
    y = y.reshape(rows, blocks, block)
    bad = ~np.isfinite(y)
    fine = np.where(bad, 0.0, y)
    a = np.abs(fine).max(axis=2, initial=0.0)
    if block == 32:
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), -200).astype(np.int64)
        e = np.where(2.0 ** (e + 1) <= a, e + 1, np.where(2.0 ** e > a, np.where(a > 0, e - 1, e), e))
        byte = np.maximum(e - 2, -127) + 127
        unit = np.exp2(byte - 127.0)
        lost = bad.any(axis=2)
        byte = np.where(lost, 255, byte)
        row = None
    else:
        lost_row = bad.any(axis=(1, 2))
        s = np.full(rows, 2.0 ** -126)
        most = a.max(axis=1, initial=0.0)
        while (most > 2688 * s).any():
            s = np.where(most > 2688 * s, 2 * s, s)
        s = np.where(lost_row, 1.0, s)
        byte = np.maximum(round_quotient(a, 6 * s[:, None], E4M3), 1)
        lost = np.repeat(lost_row[:, None], blocks, axis=1)
        byte = np.where(lost, 1, byte)
        unit = E4M3[byte] * s[:, None]
        row = np.where(lost_row, np.nan, s).astype(np.float32)
    code = round_quotient(np.abs(fine), unit[:, :, None] * np.ones(block), CODES)
    code = code + 8 * np.signbit(fine)
    code = np.where(lost[:, :, None], 0, code).reshape(rows, width).astype(np.uint8)
    byte = byte[:, :(cols + block - 1) // block]  # the padding of a row's last piece has no scale
    return code[:, 0::2] | code[:, 1::2] << 4, byte.astype(np.uint8), row


def tiles(byte):
    """Scale bytes [rows, blocks] in tiles [rows / 128, blocks / 4, 32, 4, 4], zeros where there is none."""
    rows, blocks = byte.shape
    R, W = (rows + 127) // 128, (blocks + 3) // 4
    out = np.zeros((R, W, 32, 4, 4), dtype=np.uint8)
    for r in range(rows):
        for b in range(blocks):
            out[r // 128, b // 4, r % 32, r // 32 % 4, b % 4] = byte[r, b]
    return out


def values(q, byte, block):
    """[rows, columns] in float64, without the row scales."""
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1)
    v = CODES[code & 7] * np.where(code > 7, -1.0, 1.0)
    if block == 16:
        unit = np.append(E4M3, np.nan)[byte]
    else:
        unit = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    unit = np.pad(unit, ((0, 0), (0, v.shape[1] // block - unit.shape[1])))
    return v * np.repeat(unit, block, axis=1)


def linear(x, w, xs, ws, bias):
    """(y, bound before the output's rounding) for float64 x [M, K], w [N, K] and row scales.

    The matrix units add the products of 64 columns and the sum so far at a time,
    aligned to the largest and cut at no fewer than 24 bits: each of the 65
    addends loses at most 2^-23 of the sum of absolute products, so all steps
    together at most 65 / 64 * K * 2^-23 of it; parts that are added later lose
    less. Then two scales and a bias, each rounded."""
    U = 2.0 ** -24
    with np.errstate(invalid="ignore"):
        y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        err = (x.shape[1] + 64) * 65 / 64 * 2 * U * mag
        s = (np.ones(len(x)) if xs is None else xs.astype(np.float64))[:, None] * (
            np.ones(len(w)) if ws is None else ws.astype(np.float64))[None, :]
        y, err = y * s, err * np.abs(s)
        err = err + 2 * U * (np.abs(y) + err)
        if bias is not None:
            y = y + bias.astype(np.float64)
            err = err + U * (np.abs(y) + err)
    return y, err
