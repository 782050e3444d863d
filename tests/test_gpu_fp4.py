"""4-bit floating-point rows on the GPU: codes and scales bit for bit against the
definition, the reading back, the product within derived bounds and bit for bit
where every sum is exact."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import fp4_ref, head_ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def rows_of(seed, rows, cols, dtype, pad=0, offset=0):
    """[rows, cols] with rows of many sizes, as a slice of a wider buffer that starts `offset` elements in."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g) * torch.exp2(torch.randint(-9, 8, (rows, 1), generator=g).float())
    x[:, ::13] *= 30
    x[:, 5::29] = 0
    flat = torch.zeros(offset + x.numel(), dtype=DT[dtype])
    flat[offset:] = x.to(DT[dtype]).reshape(-1)
    return flat.cuda()[offset:].view(rows, cols + pad)[:, :cols]


def check_quantized(x, block, got):
    q, byte, row = fp4_ref.quantize(x.double().cpu().numpy(), block)
    for name, a, b in (("codes", got[0].cpu().numpy(), q), ("block scales", got[1].cpu().numpy(), fp4_ref.tiles(byte))):
        assert a.shape == b.shape
        off = np.argwhere(a != b)
        assert not len(off), f"{len(off)} {name} of {a.size} differ, first at {off[0]}: {a[tuple(off[0])]}, {b[tuple(off[0])]}"
    if block == 16:
        same = np.array_equal(got[2].cpu().numpy(), row, equal_nan=True)
        assert same, "row scales"
    else:
        assert got[2] is None
    return q, byte, row


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,offset", [
    (1, 1, 0, 0), (3, 15, 1, 0), (5, 16, 0, 0), (130, 17, 15, 0), (129, 31, 1, 3), (128, 32, 0, 0), (7, 33, 0, 1), (260, 100, 28, 0),
    (33, 128, 0, 0), (9, 129, 0, 5), (20, 500, 12, 0), (6, 512, 0, 16), (5, 1000, 0, 0), (4, 1024, 0, 0), (3, 1111, 5, 0),
    (2, 2048, 0, 0), (3, 4095, 1, 0), (2, 5000, 0, 1), (2, 16384, 0, 0), (1, 16400, 0, 0), (2, 20001, 0, 7)])
def test_quantize(block, dtype, rows, cols, pad, offset):
    x = rows_of(rows * 7919 + cols, rows, cols, dtype, pad, offset)
    got = ms.quantize_rows_fp4(x, block=block)
    q, byte, row = check_quantized(x, block, got)
    want = fp4_ref.values(q, byte, block)[:, :cols]
    if row is not None:
        want = want * row.astype(np.float64)[:, None]
    for out in DT:  # exact wherever the exponents reach: rounded once in any case
        y = ms.dequantize_rows_fp4(*got, block=block, cols=cols, out_dtype=DT[out])
        assert y.shape == x.shape
        same = torch.equal(y.double().cpu(), torch.from_numpy(want).to(DT[out]).double())
        assert same, out
    whole = ms.dequantize_rows_fp4(*got, block=block, out_dtype=torch.float32)
    assert whole.shape == (rows, 2 * q.shape[1]) and not whole[:, cols:].any()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(5, 17), (40, 33), (9, 127), (6, 530), (3, 1030), (2, 4500)])
def test_dequantize_into_rows_anywhere(dtype, rows, cols):
    """Rows of every phase in a wider buffer: what is around them stays."""
    x = rows_of(cols, rows, cols, "f32")
    got = ms.quantize_rows_fp4(x, block=32)
    want = ms.dequantize_rows_fp4(*got, block=32, cols=cols, out_dtype=DT[dtype])
    lib, e = ms._native.lib(), DT[dtype].itemsize
    for offset in range(9):
        for ld in (cols, cols + 3):
            buf = torch.full((offset + rows * ld + 9,), 7.0, dtype=DT[dtype], device="cuda")
            rc = lib.maxsim_dequantize_rows_fp4(got[0].data_ptr(), got[0].shape[1], got[1].data_ptr(), None, rows, cols, 32,
                                                {2: 0, 4: 2}[e], buf.data_ptr() + offset * e, ld, torch.cuda.current_stream().cuda_stream)
            assert rc == 0
            body = buf[offset:offset + rows * ld].view(rows, ld)
            same = torch.equal(body[:, :cols], want)
            assert same and (body[:, cols:] == 7).all() and (buf[:offset] == 7).all() and (buf[offset + rows * ld:] == 7).all()


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_borders(block):
    """Every border between two codes, the values next to it, and ties, for every scale mantissa."""
    rows = []
    for m in range(8):
        top = 6.0 * (1 + m / 8) * 2.0 ** 3
        edges = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * ((1 + m / 8) * 2.0 ** 3 if block == 16 else 8.0)
        e = edges.astype(np.float32)
        for v in (e, np.nextafter(e, np.float32(np.inf)), np.nextafter(e, np.float32(0)), -e):
            row = np.zeros(2 * block, np.float32)
            row[0] = top if block == 16 else 8.0 * 4 * (1 + m / 8)
            row[1:8] = v
            row[block:block + 7] = v[::-1]
            row[block + 8] = -row[0]
            row[-1] = 2688.0 * 2 if block == 16 else 1.0
            rows.append(row)
    x = torch.from_numpy(np.stack(rows)).cuda()
    check_quantized(x, block, ms.quantize_rows_fp4(x, block=block))


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_random_bits(block):
    """float32 rows of arbitrary mantissas within one scale's reach: quotients close to borders decide exactly."""
    rng = np.random.default_rng(3)
    x = np.exp2(rng.uniform(-3, 3, (4000, 64))).astype(np.float32) * rng.choice([-1, 1], (4000, 64)).astype(np.float32)
    # three quarters of the values sit next to a border of their block's scale
    q, byte, row = fp4_ref.quantize(x, block)
    unit = (fp4_ref.E4M3[byte] * row[:, None] if block == 16 else np.exp2(byte - 127.0))
    edge = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], x.shape) * np.repeat(unit, block, axis=1)
    edge = edge.astype(np.float32)
    edge = np.where(rng.random(x.shape) < 0.5, np.nextafter(edge, np.float32(9e9)), np.nextafter(edge, np.float32(0)))
    near = (rng.random(x.shape) < 0.75) & (np.abs(edge) <= np.abs(x))
    t = torch.from_numpy(np.where(near, edge * np.sign(x), x).astype(np.float32)).cuda()
    check_quantized(t, block, ms.quantize_rows_fp4(t, block=block))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_quantize_extremes(block, dtype):
    big = torch.finfo(DT[dtype]).max
    tiny = torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
    x = torch.zeros(12, 96, dtype=DT[dtype])
    x[0] = big
    x[1] = tiny
    x[2, 3] = float("nan")
    x[2, 40] = 1
    x[3, 90] = float("-inf")
    x[3, :40] = 3
    x[4, 0], x[4, 1] = big, tiny
    x[5, :32], x[5, 32:] = 1e-4, 1
    x[6] = -0.0
    x[7, ::2], x[7, 1::2] = -big, big
    x[8] = torch.finfo(DT[dtype]).smallest_normal
    x[9, 95] = -tiny
    x[10] = torch.linspace(-1, 1, 96)
    x = x.cuda()
    got = ms.quantize_rows_fp4(x, block=block)
    q, byte, row = check_quantized(x, block, got)
    y = ms.dequantize_rows_fp4(*got, block=block, out_dtype=torch.float32).cpu()
    if block == 16:
        assert y[2].isnan().all() and y[3].isnan().all()
    else:
        assert y[2, :32].isnan().all() and y[2, 40] == 1 and y[3, 64:].isnan().all() and (y[3, :32] == 3).all()
    assert not y[[0, 1, 4, 5, 6, 7, 8, 9, 10, 11]].isnan().any()


def test_quantize_empty_and_shapes():
    q, b, s = ms.quantize_rows_fp4(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 32) and b.shape == (0, 1, 32, 4, 4) and s.shape == (0,)
    q, b, s = ms.quantize_rows_fp4(torch.empty(3, 0, device="cuda"))
    assert q.shape == (3, 0) and b.numel() == 0 and (s == 2.0 ** -126).all()
    x = rows_of(5, 24, 64, "bf16").view(2, 3, 4, 64)
    q, b, s = ms.quantize_rows_fp4(x)
    flat = ms.quantize_rows_fp4(x.reshape(24, 64))
    assert q.shape == (2, 3, 4, 32) and s.shape == (2, 3, 4) and torch.equal(q.view(24, 32), flat[0]) and torch.equal(b, flat[1])
    # given outputs, and neighbours left alone
    buf = torch.full((26, 32), 7, dtype=torch.uint8, device="cuda")
    ms.quantize_rows_fp4(x.reshape(24, 64), q=buf[1:25], block_scale=b, scale=s.view(24))
    assert torch.equal(buf[1:25], flat[0]) and (buf[0] == 7).all() and (buf[25] == 7).all()
    # rows of a wider buffer of codes
    wide = torch.zeros(24, 64, dtype=torch.uint8, device="cuda")
    wide[:, 16:48] = flat[0]
    a, c = ms.dequantize_rows_fp4(wide[:, 16:48], flat[1], flat[2]), ms.dequantize_rows_fp4(*flat)
    assert torch.equal(a, c)


def quantized(seed, rows, cols, block, ints=False):
    """(device triple, float64 values without row scales, row scales) of random rows; ints: codes of unit scale."""
    g = torch.Generator().manual_seed(seed)
    if ints:
        x = torch.tensor([0.0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6])[torch.randint(0, 11, (rows, cols), generator=g)]
        x[:, ::16] = 6 if block == 16 else 4  # every block of 16 has the same scale, every block of 32 the scale 1
        if block == 32:
            x = x.clamp(-6, 6)
        x = x.cuda()
    else:
        x = rows_of(seed, rows, cols, "f32")
    q, b, s = ms.quantize_rows_fp4(x, block=block)
    v = ms.dequantize_rows_fp4(q, b, None, block=block, out_dtype=torch.float32).double().cpu().numpy()
    return (q, b, s), v, None if s is None else s.cpu().numpy()


SHAPES = [(1, 1, 1), (1, 128, 64), (1, 300, 4096), (2, 7, 33), (3, 129, 256), (8, 64, 500), (17, 257, 129), (32, 128, 1024), (33, 1000, 96),
          (64, 512, 2048), (100, 100, 100), (128, 256, 512), (129, 255, 255), (200, 40, 4000), (256, 256, 256), (300, 520, 700),
          (257, 9, 1025), (1000, 3, 64), (1025, 128, 320), (2000, 1030, 200), (5, 2000, 8200), (513, 511, 1)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(block, out, M, N, K):
    x, xv, xs = quantized(M * 31 + K, M, K, block)
    w, wv, ws = quantized(N * 37 + K + 1, N, K, block)
    bias = None if (M + N) % 3 == 0 else torch.randn(N, generator=torch.Generator().manual_seed(K)).mul(10).cuda()
    if block == 32 or out == "f16":  # values within f16's range: row scales of the caller's own
        sx, sw = torch.rand(M) * 1e-3 + 1e-4, torch.rand(N) * 1e-2 + 1e-3
        if block == 32:
            big = max(np.abs(xv).max() * np.abs(wv).max() * K, 1.0)
            sx = sx / big * 1e4
        else:
            sx, sw = sx * 1e-6, sw * 1e-3
        x, w = (x[0], x[1], sx.float().cuda()), (w[0], w[1], sw.float().cuda())
        xs, ws = sx.float().numpy(), sw.float().numpy()
    y = ms.linear_fp4(*x, *w, bias, block=block, out_dtype=DT[out])
    ref, err = fp4_ref.linear(xv, wv, xs, ws, None if bias is None else bias.cpu().numpy())
    assert y.shape == (M, N) and np.abs(ref).max() < 6e4 or out != "f16"
    head_ref.within(y.float().cpu().numpy(), ref, err, out)
    again = ms.linear_fp4(*x, *w, bias, block=block, out_dtype=DT[out])
    assert torch.equal(y, again)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", SHAPES + [(1, 4096, 4096), (300, 300, 16384), (4096, 130, 64)])
def test_linear_exact(block, M, N, K):
    """Codes of one scale: every partial sum is a multiple of 2^-2 below 2^22 of it, so no sum rounds."""
    x, xv, xs = quantized(M + K, M, K, block, ints=True)
    w, wv, ws = quantized(N + K + 1, N, K, block, ints=True)
    y = ms.linear_fp4(*x, *w, block=block, out_dtype=torch.float32)
    ref = xv @ wv.T
    if block == 16:
        ref = ref * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    off = np.argwhere(y.double().cpu().numpy() != ref)
    assert not len(off), f"{len(off)} of {ref.size} outputs differ, first at {off[0]}"


def test_linear_layouts():
    """Leading dimensions, rows of wider buffers, outputs given, no columns, no rows, NaN rows."""
    x, xv, xs = quantized(1, 60, 96, 16)
    w, wv, ws = quantized(2, 50, 96, 16)
    y = ms.linear_fp4(*x, *w)
    lead = ms.linear_fp4(x[0].view(3, 20, 48), x[1], x[2].view(3, 20), *w)
    assert lead.shape == (3, 20, 50) and torch.equal(lead.view(60, 50), y)
    wide = torch.zeros(60, 80, dtype=torch.uint8, device="cuda")
    wide[:, 16:64] = x[0]
    assert torch.equal(ms.linear_fp4(wide[:, 16:64], x[1], x[2], *w), y)
    odd = torch.zeros(60, 57, dtype=torch.uint8, device="cuda")
    odd[:, 5:53] = x[0]
    assert torch.equal(ms.linear_fp4(odd[:, 5:53], x[1], x[2], *w), y)
    buf = torch.full((62, 50), 3.0, dtype=torch.bfloat16, device="cuda")
    ms.linear_fp4(*x, *w, out=buf[1:61])
    assert torch.equal(buf[1:61], y) and (buf[0] == 3).all() and (buf[61] == 3).all()
    empty = ms.quantize_rows_fp4(torch.empty(4, 0, device="cuda")), ms.quantize_rows_fp4(torch.empty(5, 0, device="cuda"))
    bias = torch.arange(5.0, device="cuda")
    assert torch.equal(ms.linear_fp4(*empty[0], *empty[1], bias), bias.bfloat16().expand(4, 5))
    none = ms.quantize_rows_fp4(torch.empty(0, 96, device="cuda"))
    assert ms.linear_fp4(*none, *w).shape == (0, 50) and ms.linear_fp4(*x, *none).shape == (60, 0)
    for block in (16, 32):
        t = torch.full((40, 96), 1.5, device="cuda")  # of few enough bits to be held exactly
        t[7, 50] = float("nan")
        a, b = ms.quantize_rows_fp4(t, block=block), ms.quantize_rows_fp4(torch.full((9, 96), 1.5, device="cuda"), block=block)
        y = ms.linear_fp4(*a, *b, block=block, out_dtype=torch.float32).cpu()
        assert y[7].isnan().all() and (y[[i for i in range(40) if i != 7]] == 216).all()
        y = ms.linear_fp4(*b, *a, block=block, out_dtype=torch.float32).cpu()
        assert y[:, 7].isnan().all() and (y[:, [i for i in range(40) if i != 7]] == 216).all()


def test_graph_and_stream():
    """Quantisation, product and reading back on a stream of their own, captured once and replayed on new data."""
    xs = [rows_of(s, 200, 512, "bf16") for s in (1, 2)]
    w = ms.quantize_rows_fp4(rows_of(9, 300, 512, "bf16"))
    want = [ms.linear_fp4(*ms.quantize_rows_fp4(x), *w) for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ms.linear_fp4(*ms.quantize_rows_fp4(x), *w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = ms.linear_fp4(*ms.quantize_rows_fp4(x), *w)
        for i in (1, 0, 1):
            x.copy_(xs[i])
            graph.replay()
            side.synchronize()
            assert torch.equal(y, want[i])
