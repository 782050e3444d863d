"""Parity of the token head's operators with their plain references: row
quantisation, the INT8 linear product, dropout and its gradient."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from maxsim_scoring_gb300 import _native
from tests import head_ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def rows_of(rng, rows, cols, dtype, pad=0, shift=0):
    """A [rows, cols] device tensor whose rows are cols + pad apart and start `shift` elements into their buffer."""
    t = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    buf = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.from_numpy(t))
    return view


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- row quantisation

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [
    (1, 1, 0, 0), (3, 7, 0, 0), (32, 128, 0, 0), (33, 128, 8, 0), (5, 100, 3, 1), (2, 1024, 0, 1), (7, 1000, 24, 8),
    (4, 2048, 0, 0), (3, 4104, 0, 0), (2, 8193, 0, 0), (2, 20000, 8, 0), (1, 70001, 0, 3), (1000, 16, 0, 0), (777, 24, 0, 0),
    (300, 5, 0, 0), (301, 17, 2, 1), (50, 85, 0, 0), (40, 250, 1, 0), (9, 511, 0, 0), (9, 1500, 1, 1), (3, 5001, 0, 0),
    (500, 40, 0, 0), (200, 4, 0, 0), (70, 33, 0, 0), (41, 131, 0, 0), (40, 200, 8, 3), (33, 203, 16, 8), (17, 1039, 0, 0),
    (13, 1100, 0, 4), (9, 1801, 8, 0), (5, 3003, 0, 0), (3, 33001, 0, 0), (2, 40003, 8, 0), (1, 129, 0, 8)])
@pytest.mark.parametrize("normalize", [False, True])
def test_quantize_rows(dtype, rows, cols, pad, shift, normalize):
    x = rows_of(np.random.default_rng(rows + cols), rows, cols, dtype, pad, shift)
    q, scale = ms.quantize_rows(x, normalize=normalize)
    assert ms.device_status() == 0
    ref_q, ref_s, rel = head_ref.quantize(f64(x), normalize)
    assert np.array_equal(q.cpu().numpy(), ref_q)
    assert np.all(np.abs(f64(scale) - ref_s) <= rel * ref_s)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [7, 8, 13, 40, 100, 129, 1024, 3001, 9000])
@pytest.mark.parametrize("normalize", [False, True])
def test_quantize_special_rows(dtype, cols, normalize):
    rng = np.random.default_rng(cols)
    x = rows_of(rng, 10, cols, dtype)
    x[0] = 0.0
    x[1] = -0.0
    x[2, cols // 2] = float("nan")
    x[3, cols - 1] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = torch.finfo(DT[dtype]).max
    x[6] = -torch.finfo(DT[dtype]).max
    x[7] = 0.0
    x[7, cols - 1] = torch.finfo(DT[dtype]).smallest_normal / 4      # a subnormal alone in its row
    x[8] = 0.0
    x[8, 1] = -3.0
    q, scale = ms.quantize_rows(x, normalize=normalize)
    ref_q, ref_s, rel = head_ref.quantize(f64(x), normalize)
    assert np.array_equal(q.cpu().numpy(), ref_q)
    got = f64(scale)
    assert np.array_equal(np.isnan(got), np.isnan(ref_s)) and np.isnan(ref_s).sum() == 3
    fine = ~np.isnan(ref_s)
    assert np.all(np.abs(got - ref_s)[fine] <= (rel * ref_s)[fine])
    assert np.all(got[fine] > 0)


def test_quantize_halfway_codes():
    # quotients on and one unit around every half-integer: fp32 division and ties to even decide
    base = np.arange(-126.5, 127.0, 1.0, dtype=np.float32)
    for a in (127.0, 1.0, 3.0e-5, 0.7):
        for s in (np.float32(a) / np.float32(127), np.float32(a) * (np.float32(1) / np.float32(127))):
            y = (base * s).astype(np.float32)
            x = np.concatenate([[np.float32(a)], y, np.nextafter(y, np.float32(9e9)), np.nextafter(y, np.float32(-9e9))])
            x = torch.from_numpy(x.astype(np.float32)[None]).cuda()
            q, _ = ms.quantize_rows(x)
            assert np.array_equal(q.cpu().numpy(), head_ref.quantize(f64(x), False)[0])


@pytest.mark.parametrize("cols,ld_x,ld_q,shift", [(131, 131, 131, 0), (131, 139, 147, 3), (200, 205, 205, 5), (1039, 1040, 1048, 7),
                                                  (300, 301, 302, 1), (40, 48, 48, 8), (33001, 33009, 33001, 2)])
def test_quantize_rows_leaves_what_is_not_theirs(cols, ld_x, ld_q, shift):
    # codes between other bytes, values between NaN: neither the one nor the other may leak
    lib = _native.lib()
    rng = np.random.default_rng(cols)
    rows = 7
    for name, dt in DT.items():
        x = torch.full((shift + rows * ld_x,), float("nan"), dtype=dt, device="cuda")
        view = x[shift:].view(rows, ld_x)
        view[:, :cols] = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to("cuda", dt)
        q = torch.full((shift + rows * ld_q,), 77, dtype=torch.int8, device="cuda")
        codes_view = q[shift:].view(rows, ld_q)
        scale = torch.empty(rows, device="cuda")
        rc = lib.maxsim_quantize_rows(view.data_ptr(), ms.ops._DT_ANY[dt], rows, cols, ld_x, 0, codes_view.data_ptr(), ld_q,
                                      scale.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        ref_q, ref_s, rel = head_ref.quantize(f64(view[:, :cols]), False)
        assert np.array_equal(codes_view[:, :cols].cpu().numpy(), ref_q)
        assert np.all(np.abs(f64(scale) - ref_s) <= rel * ref_s)
        assert (codes_view[:, cols:] == 77).all() and (q[:shift] == 77).all()


def test_quantize_empty_and_shapes():
    q, s = ms.quantize_rows(torch.empty((0, 16), device="cuda"))
    assert q.shape == (0, 16) and s.shape == (0,)
    q, s = ms.quantize_rows(torch.empty((3, 0), device="cuda"), normalize=True)
    assert q.shape == (3, 0) and (s == 2.0 ** -126).all()
    x = torch.randn(2, 3, 5, 32, device="cuda")
    q, s = ms.quantize_rows(x)
    assert q.shape == x.shape and s.shape == (2, 3, 5)
    x = torch.randn(4, 6, 40, device="cuda")[..., :32]            # rows of a wider buffer, three dimensions
    q2, s2 = ms.quantize_rows(x)
    q3, s3 = ms.quantize_rows(x.contiguous())
    assert torch.equal(q2, q3) and torch.equal(s2, s3)
    t = torch.randn(32, 6, device="cuda").t()                     # columns apart: copied
    assert torch.equal(ms.quantize_rows(t)[0], ms.quantize_rows(t.contiguous())[0])
    q = torch.empty((6, 32), dtype=torch.int8, device="cuda")
    assert ms.quantize_rows(t, q=q)[0] is q
    with pytest.raises(ValueError):
        ms.quantize_rows(t, q=q.t())


def test_quantize_rows_of_a_wider_output():
    # the C entry takes a stride for q; what lies between its rows stays
    x = torch.randn(9, 48, device="cuda")
    q = torch.full((9, 64), 55, dtype=torch.int8, device="cuda")
    s = torch.empty(9, device="cuda")
    rc = _native.lib().maxsim_quantize_rows(x.data_ptr(), _native.F32, 9, 48, 48, 0, q.data_ptr(), 64, s.data_ptr(),
                                            torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(q[:, :48], ms.quantize_rows(x)[0]) and (q[:, 48:] == 55).all()


# ---------------------------------------------------------------- INT8 linear

def codes(rng, rows, cols, pad=0, shift=0, low=-127):
    buf = torch.full((rows * (cols + pad) + shift,), 111, dtype=torch.int8, device="cuda")
    view = buf[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.from_numpy(rng.integers(low, 128, size=(rows, cols)).astype(np.int8)))
    return view


def check_linear(x, w, dtype, bias, rng, scales=None):
    M, N = x.shape[0], w.shape[0]
    xs = rng.uniform(0.01, 0.05, M).astype(np.float32) if scales is None else scales
    ws = rng.uniform(0.001, 0.002, N).astype(np.float32)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    dev = [torch.from_numpy(v).cuda() if v is not None else None for v in (xs, ws, b)]
    got = ms.linear_int8(x, dev[0], w, dev[1], dev[2], out_dtype=DT[dtype])
    assert ms.device_status() == 0
    assert got.dtype == DT[dtype] and got.shape == (M, N)
    ref, bound = head_ref.linear(x.cpu().numpy(), xs, w.cpu().numpy(), ws, b)
    head_ref.within(f64(got), ref, bound, dtype)
    return got


SHAPES = [(1, 1, 1), (1, 16, 16), (1, 4096, 4096), (2, 33, 64), (3, 128, 1024), (8, 100, 48), (9, 17, 80),
          (16, 256, 512), (17, 130, 144), (32, 128, 1024), (33, 257, 272), (64, 64, 4096), (64, 1000, 320),
          (65, 128, 128), (65, 300, 64), (100, 16, 2048), (127, 129, 1040), (128, 128, 16), (129, 255, 112),
          (200, 256, 256), (255, 257, 384), (256, 256, 128), (257, 512, 1024), (500, 100, 4096), (700, 1100, 640),
          (1000, 128, 768), (2049, 384, 96), (300, 2000, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,bias", [("bf16", True), ("f32", False)])
def test_linear_int8(M, N, K, dtype, bias):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    check_linear(codes(rng, M, K), codes(rng, N, K, low=-128), dtype, bias, rng)


# several tiles for every pair of SMs: each width and orientation, weights kept in shared memory, K cut into slices
@pytest.mark.parametrize("M,N,K,dtype", [
    (20001, 128, 1024, "f16"), (19500, 100, 1008, "f32"), (30011, 64, 2048, "bf16"), (40000, 33, 176, "f32"),
    (20000, 128, 1040, "bf16"), (6100, 2050, 272, "bf16"), (6000, 2001, 144, "f32"), (1500, 8100, 128, "f16"),
    (700, 16000, 80, "f32"), (5000, 700, 512, "f16"), (90, 20000, 96, "bf16"), (150, 300, 9000, "bf16"),
    (300, 120, 8000, "f32"), (40, 1000, 16000, "f16"), (20003, 120, 333, "bf16"),
    (20000, 48, 640, "f16"), (400, 9000, 640, "f32"), (9000, 400, 640, "f16"), (130, 9000, 640, "f16"), (9000, 130, 640, "f32"),
    (60, 16000, 640, "f32"), (16000, 60, 2112, "bf16"), (16000, 60, 2112, "f32")])
def test_linear_int8_many_tiles(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    check_linear(codes(rng, M, K), codes(rng, N, K), dtype, True, rng)


@pytest.mark.parametrize("M,N,K", [(1, 5, 3), (7, 40, 33), (40, 130, 1111), (64, 31, 97), (70, 50, 1), (129, 300, 515),
                                   (600, 200, 77)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 0), (16, 3), (0, 16)])
def test_linear_int8_odd_rows(M, N, K, pad, shift):
    rng = np.random.default_rng(M + N + K + pad + shift)
    check_linear(codes(rng, M, K, pad, shift), codes(rng, N, K, 0, shift), "f16", True, rng)


@pytest.mark.parametrize("M,N,K", [(3000, 200, 301), (200, 3000, 301), (5000, 600, 257), (600, 5000, 250), (20000, 70, 99)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 1), (16, 3), (0, 16)])
def test_linear_int8_odd_rows_of_large_products(M, N, K, pad, shift):
    rng = np.random.default_rng(M + N + K + pad + shift)
    check_linear(codes(rng, M, K, pad, shift), codes(rng, N, K, 0, shift), "bf16", True, rng)


def test_linear_int8_extreme_sums():
    # every product +-16384 or 16129: sums up to K * 2^14, beyond 2^24 in both directions
    rng = np.random.default_rng(3)
    for M in (5, 200):
        for K in (1024, 4096, 20000):
            x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
            w = torch.full((40, K), -128, dtype=torch.int8, device="cuda")
            w[::2] = 127
            x[1::2] = 127
            check_linear(x, w, "f32", False, rng)


@pytest.mark.parametrize("M,N,K", [(20, 100, 16384), (700, 300, 16384), (300, 1500, 6000), (2500, 600, 3000)])
def test_linear_int8_one_signed_sums(M, N, K):
    # sums that grow past 2^24 and stay there: the fp32 accumulator rounds, within its bound
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.integers(90, 128, size=(M, K)).astype(np.int8)).cuda()
    w = torch.from_numpy(rng.integers(90, 128, size=(N, K)).astype(np.int8)).cuda()
    check_linear(x, w, "f32", False, rng)


def test_linear_int8_longest_sum():
    K = 131071                                                     # the largest K, for both kernels
    rng = np.random.default_rng(5)
    for M in (2, 130):
        check_linear(codes(rng, M, K), codes(rng, 20, K), "f32", True, rng)
    with pytest.raises(_native.MaxSimError):
        z = torch.zeros((2, K + 1), dtype=torch.int8, device="cuda")
        ms.linear_int8(z, torch.ones(2, device="cuda"), z, torch.ones(2, device="cuda"))


def test_linear_int8_nonfinite_scales_stay_in_their_rows():
    rng = np.random.default_rng(6)
    for M, N in ((6, 96), (200, 96), (8000, 96), (20000, 96), (300, 9000), (4000, 1000)):
        x, w = codes(rng, M, 256), codes(rng, N, 256)
        xs = rng.uniform(0.01, 0.05, M).astype(np.float32)
        xs[2], xs[4], xs[5] = np.nan, np.inf, 0.0
        x[2] = 0
        ws = rng.uniform(0.001, 0.002, N).astype(np.float32)
        got = f64(ms.linear_int8(x, torch.from_numpy(xs).cuda(), w, torch.from_numpy(ws).cuda(), out_dtype=torch.float32))
        assert np.isnan(got[2]).all() and (got[5] == 0).all()
        fine = [r for r in range(M) if r not in (2, 4)]
        ref, bound = head_ref.linear(x.cpu().numpy()[fine], xs[fine], w.cpu().numpy(), ws, None)
        head_ref.within(got[fine], ref, bound, "f32")
        assert not np.isfinite(got[4]).any()                       # infinity, or NaN where the sum is 0


def test_linear_int8_empty():
    one = torch.ones(4, device="cuda")
    b = torch.tensor([1.0, -2.0, 3.0, 0.5], device="cuda")
    z = torch.empty((4, 0), dtype=torch.int8, device="cuda")
    for M in (4, 100):
        zx = torch.empty((M, 0), dtype=torch.int8, device="cuda")
        out = ms.linear_int8(zx, torch.ones(M, device="cuda"), z, one, b, out_dtype=torch.float32)
        assert torch.equal(out, b.expand(M, 4))
        assert (ms.linear_int8(zx, torch.ones(M, device="cuda"), z, one, out_dtype=torch.float32) == 0).all()
    x = torch.zeros((4, 32), dtype=torch.int8, device="cuda")
    assert ms.linear_int8(x[:0], one[:0], x, one).shape == (0, 4)
    assert ms.linear_int8(x, one, x[:0], one[:0]).shape == (4, 0)
    assert ms.linear_int8(x.view(2, 2, 32), one.view(2, 2), x, one, b).shape == (2, 2, 4)


def test_linear_int8_rows_of_a_wider_output():
    rng = np.random.default_rng(8)
    lib = _native.lib()
    for M, shapes in ((3, ((70, 77, 3), (64, 96, 0), (300, 301, 1))), (150, ((70, 77, 3), (64, 96, 0), (300, 301, 1))),
                      (9000, ((300, 301, 1), (304, 312, 0), (300, 302, 2), (606, 618, 4))), (300, ((9000, 9001, 3), (9000, 9008, 0))),
                      (20000, ((70, 77, 3), (128, 136, 0), (50, 56, 8), (33, 34, 1))), (2000, ((4100, 4101, 0),)),
                      (4100, ((2000, 2008, 0), (1999, 2000, 8)))):
        for N, ld, off in shapes:
            x, w = codes(rng, M, 128), codes(rng, N, 128)
            xs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
            for name, dt in DT.items():
                ref = ms.linear_int8(x, xs, w, ws, out_dtype=dt)
                buf = torch.full((M * ld + off,), 7.0, dtype=dt, device="cuda")
                out = buf[off:].view(M, ld)
                need = lib.maxsim_workspace_size(_native.OP_LINEAR_INT8, M, N, 128, 128, 128)
                work = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
                rc = lib.maxsim_linear_int8(x.data_ptr(), 128, xs.data_ptr(), w.data_ptr(), 128, ws.data_ptr(), None, M, N,
                                            128, ms.ops._DT_ANY[dt], out.data_ptr(), ld, work.data_ptr(), need,
                                            torch.cuda.current_stream().cuda_stream)
                assert rc == 0
                assert torch.equal(out[:, :N], ref) and (out[:, N:] == 7).all() and (buf[:off] == 7).all()


def test_linear_int8_repeats_and_other_streams():
    rng = np.random.default_rng(9)
    for M, N, K in ((5, 300, 2048), (48, 1000, 1000), (300, 500, 4096), (129, 140, 1111), (20000, 128, 512),
                    (500, 9000, 256), (5000, 2000, 272)):
        x, w = codes(rng, M, K), codes(rng, N, K)
        xs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        first = ms.linear_int8(x, xs, w, ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = [ms.linear_int8(x, xs, w, ws) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(first, a) for a in again)


@pytest.mark.parametrize("M,N,K", [(4, 300, 512), (700, 1100, 640), (150, 300, 9000), (20000, 64, 256)])
def test_linear_int8_in_a_cuda_graph(M, N, K):
    # the call only enqueues: captured with its dependent launches and replayed on new values
    rng = np.random.default_rng(K)
    x, w = codes(rng, M, K), codes(rng, N, K)
    xs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    ms.linear_int8(x, xs, w, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ms.linear_int8(x, xs, w, ws)
    for _ in range(3):
        x.copy_(codes(rng, M, K))
        graph.replay()
        assert torch.equal(out, ms.linear_int8(x, xs, w, ws))
    assert ms.device_status() == 0


# ---------------------------------------------------------------- dropout

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [
    (1, 1, 0, 0), (1, 7, 0, 0), (3, 8, 0, 0), (5, 13, 0, 0), (5, 13, 3, 1), (32, 1024, 0, 0), (17, 1023, 1, 0), (9, 256, 8, 0),
    (9, 256, 8, 3), (4, 4100, 4, 0), (1000, 3, 0, 0), (2, 70001, 0, 0), (130, 1000, 0, 1)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_fwd(dtype, rows, cols, pad, shift, residual):
    rng = np.random.default_rng(rows * 3 + cols)
    x = rows_of(rng, rows, cols, dtype, pad, shift)
    r = rows_of(rng, rows, cols, dtype, 0 if pad else 5, shift) if residual else None
    seed, offset = 0xDEADBEEF12345678, (7 << 32) + 5
    y = ms.dropout_fwd(x, 0.3, seed, offset, r)
    ref, bound = head_ref.dropout(f64(x), 0.3, seed, offset, None if r is None else f64(r))
    head_ref.within(f64(y), ref, bound, dtype)
    if not residual:
        assert np.array_equal(f64(y) != 0, head_ref.keep_mask(rows, cols, 0.3, seed, offset) & (f64(x) != 0))
        assert torch.equal(y, ms.dropout_bwd(x, 0.3, seed, offset))   # the gradient is the same map


@pytest.mark.parametrize("p", [0.0, 1e-6, 1.0 / 65536, 0.5, 0.99999, 1.0])
def test_dropout_rates(p):
    x = rows_of(np.random.default_rng(1), 50, 77, "f32")
    r = rows_of(np.random.default_rng(2), 50, 77, "f32")
    y = ms.dropout_fwd(x, p, 3, 4, r)
    ref, bound = head_ref.dropout(f64(x), p, 3, 4, f64(r))
    head_ref.within(f64(y), ref, bound, "f32")
    if round(p * 65536) == 65536:
        assert torch.equal(y, r)
    with pytest.raises(_native.MaxSimError):
        ms.dropout_fwd(x, p + 1.5, 3)


@pytest.mark.parametrize("cols", [64, 77])
def test_dropout_nonfinite_values(cols):
    x = rows_of(np.random.default_rng(1), 20, cols, "bf16")
    x[3] = float("nan")
    x[4] = float("inf")
    x[5] = -float("inf")
    y = ms.dropout_fwd(x, 0.5, 3, 4)
    keep = head_ref.keep_mask(20, cols, 0.5, 3, 4)
    got = f64(y)
    assert (got[3:6][~keep[3:6]] == 0).all()                        # a dropped NaN or infinity is 0
    assert np.isnan(got[3][keep[3]]).all() and np.isposinf(got[4][keep[4]]).all() and np.isneginf(got[5][keep[5]]).all()
    assert (ms.dropout_fwd(x, 1.0, 3, 4) == 0).all()


@pytest.mark.parametrize("cols", [96, 101])
def test_dropout_in_place(cols):
    x = rows_of(np.random.default_rng(1), 40, cols, "f16")
    r = rows_of(np.random.default_rng(2), 40, cols, "f16")
    want = ms.dropout_fwd(x, 0.2, 9, 1, r)
    into_r = r.clone()
    assert ms.dropout_fwd(x, 0.2, 9, 1, into_r, out=into_r) is into_r and torch.equal(into_r, want)
    into_x = x.clone()
    assert torch.equal(ms.dropout_fwd(into_x, 0.2, 9, 1, r, out=into_x), want)


def test_dropout_mask_does_not_depend_on_layout():
    x = torch.ones(64, 96, device="cuda")
    y = ms.dropout_fwd(x, 0.4, 11, 2)
    wide = torch.ones(64, 200, device="cuda")[:, 3:99]
    assert torch.equal(y, ms.dropout_fwd(wide, 0.4, 11, 2))
    assert torch.equal(y, ms.dropout_fwd(x.half(), 0.4, 11, 2).bool() * y)
    assert torch.equal(y.view(8, 8, 96), ms.dropout_fwd(x.view(8, 8, 96), 0.4, 11, 2))
    assert not torch.equal(y, ms.dropout_fwd(x, 0.4, 11, 3)) and not torch.equal(y, ms.dropout_fwd(x, 0.4, 12, 2))


def test_dropout_counters_beyond_32_bits():
    # the last elements of a matrix of more than 2^35 would not fit here; more than 2^32 elements do
    rows, cols = 4_300_001, 1000
    x = torch.ones((rows, cols), dtype=torch.float16, device="cuda")
    y = ms.dropout_fwd(x, 0.5, 21, 22, out=x)
    for row in (0, 4_294_967, 4_294_968, rows - 1):
        first = row * cols // 8
        words = head_ref.philox4x32_10(np.arange(first, (row * cols + cols) // 8 + 1), 21, 22)
        halves = np.stack([words & 0xFFFF, words >> 16], axis=-1).reshape(-1)[row * cols - 8 * first:][:cols]
        assert np.array_equal(y[row].bool().cpu().numpy(), halves >= 32768)


def test_dropout_empty():
    assert ms.dropout_fwd(torch.empty((0, 5), device="cuda"), 0.1, 0).shape == (0, 5)
    assert ms.dropout_fwd(torch.empty((5, 0), device="cuda"), 0.1, 0).shape == (5, 0)
    assert ms.dropout_bwd(torch.empty((2, 0, 5), device="cuda"), 0.1, 0).shape == (2, 0, 5)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_dropout_autograd(dtype):
    rng = np.random.default_rng(4)
    x = rows_of(rng, 12, 50, dtype).clone().requires_grad_()
    r = rows_of(rng, 12, 50, dtype).clone().requires_grad_()
    g = rows_of(rng, 12, 50, dtype)
    y = ms.dropout(x, 0.25, 5, 6, r)
    y.backward(g)
    ref, bound = head_ref.dropout(f64(g), 0.25, 5, 6)
    head_ref.within(f64(x.grad), ref, bound, dtype)
    assert torch.equal(r.grad, g)
    # a broadcast gradient (the sum's), and no gradient where none is wanted
    x2 = x.detach().requires_grad_()
    ms.dropout(x2, 0.25, 5, 6, r.detach()).sum().backward()
    one, bound = head_ref.dropout(np.ones((12, 50)), 0.25, 5, 6)
    head_ref.within(f64(x2.grad), one, bound, dtype)


def test_dropout_gradient_by_differences():
    # the map is linear for a given mask: central differences with h = 2 are the gradient but for rounding
    rng = np.random.default_rng(6)
    x = rows_of(rng, 6, 20, "f32")
    g = rows_of(rng, 6, 20, "f32")
    dx = f64(ms.dropout_bwd(g, 0.3, 8, 9))
    for r, c in [(0, 0), (2, 7), (5, 19), (3, 11), (1, 3), (4, 8)]:
        up, down = x.clone(), x.clone()
        up[r, c] += 2.0
        down[r, c] -= 2.0
        fu, fd = (f64(ms.dropout_fwd(v, 0.3, 8, 9)) for v in (up, down))
        diff = ((fu - fd) * f64(g)).sum() / (f64(up)[r, c] - f64(down)[r, c])
        # the two outputs carry two roundings each
        tol = 8 * head_ref.U * (abs(fu[r, c]) + abs(fd[r, c])) * abs(f64(g)[r, c]) + 4 * head_ref.U * abs(diff)
        assert abs(diff - dx[r, c]) <= tol
