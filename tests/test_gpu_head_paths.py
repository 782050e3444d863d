"""Paths of the token head that its binding or its smallest sizes do not reach:
dropout into rows apart, in place with strides, and over more elements than a
grid takes at once; the quantiser over more rows than a grid takes at once;
sliced products of padded rows; weights kept in shared memory in a CUDA graph."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from maxsim_scoring_gb300 import _native
from tests import head_ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SENTINEL = 77.0


def stream():
    return torch.cuda.current_stream().cuda_stream


def f64(t):
    return t.double().cpu().numpy()


def rows_apart(values, ld, shift, dtype):
    """values [rows, cols] in rows ld apart, `shift` elements into a buffer of sentinels: (buffer, view [rows, ld])."""
    rows, cols = values.shape
    buf = torch.full((shift + rows * ld + 8,), SENTINEL, dtype=DT[dtype], device="cuda")
    view = buf[shift:shift + rows * ld].view(rows, ld)
    view[:, :cols] = torch.as_tensor(values).to("cuda", DT[dtype])
    return buf, view


def untouched(buf, view, cols, shift):
    end = shift + view.numel()
    return bool((view[:, cols:] == SENTINEL).all() and (buf[:shift] == SENTINEL).all() and (buf[end:] == SENTINEL).all())


# ---------------------------------------------------------------- dropout

# rows of 16-byte pieces apart; rows off their boundaries, at least as long as a warp's run and shorter; one row;
# each with few elements, and with more than a grid takes at once
LAYOUTS = [(5, 64, 80, 72, 96, 0), (7, 1024, 1032, 1040, 1024, 8), (6, 300, 301, 307, 303, 0), (6, 257, 260, 258, 259, 3),
           (40, 33, 40, 37, 35, 1), (9, 5, 7, 6, 8, 0), (1, 1000, 1001, 1002, 1003, 1), (12, 256, 256, 257, 256, 0),
           (5200, 1024, 1032, 1040, 1032, 8), (3000, 1003, 1004, 1005, 1006, 1), (40000, 101, 102, 103, 104, 0)]


@pytest.mark.parametrize("rows,cols,ld_x,ld_y,ld_r,shift", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_into_rows_apart(rows, cols, ld_x, ld_y, ld_r, shift, dtype, residual):
    rng = np.random.default_rng(rows + cols)
    x_buf, x = rows_apart(rng.standard_normal((rows, cols)), ld_x, shift, dtype)
    r_buf, r = rows_apart(rng.standard_normal((rows, cols)), ld_r, shift, dtype)
    y_buf, y = rows_apart(np.zeros((rows, cols)), ld_y, shift, dtype)
    seed, offset = 0x123456789ABCDEF, 3
    lib, dt = _native.lib(), ms.ops._DT_ANY[DT[dtype]]
    rc = lib.maxsim_dropout_fwd(x.data_ptr(), dt, rows, cols, ld_x, r.data_ptr() if residual else None, ld_r if residual else 0,
                                0.3, seed, offset, y.data_ptr(), ld_y, stream())
    assert rc == 0
    ref, bound = head_ref.dropout(f64(x[:, :cols]), 0.3, seed, offset, f64(r[:, :cols]) if residual else None)
    head_ref.within(f64(y[:, :cols]), ref, bound, dtype)
    assert untouched(y_buf, y, cols, shift) and untouched(x_buf, x, cols, shift)
    if not residual:
        d_buf, d = rows_apart(np.zeros((rows, cols)), ld_y, shift, dtype)
        assert lib.maxsim_dropout_bwd(x.data_ptr(), dt, rows, cols, ld_x, 0.3, seed, offset, d.data_ptr(), ld_y, stream()) == 0
        assert torch.equal(d_buf, y_buf)


@pytest.mark.parametrize("rows,cols,ld,shift", [(50, 64, 80, 0), (50, 1024, 1032, 8), (50, 300, 301, 0), (50, 33, 40, 1), (900, 3001, 3003, 3)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_dropout_in_place_with_strides(rows, cols, ld, shift, dtype, into):
    rng = np.random.default_rng(cols)
    x_buf, x = rows_apart(rng.standard_normal((rows, cols)), ld, shift, dtype)
    r_buf, r = rows_apart(rng.standard_normal((rows, cols)), ld, shift, dtype)
    ref, bound = head_ref.dropout(f64(x[:, :cols]), 0.3, 1, 2, f64(r[:, :cols]))
    y_buf, y = (x_buf, x) if into == "x" else (r_buf, r)
    rc = _native.lib().maxsim_dropout_fwd(x.data_ptr(), ms.ops._DT_ANY[DT[dtype]], rows, cols, ld, r.data_ptr(), ld, 0.3, 1, 2,
                                          y.data_ptr(), ld, stream())
    assert rc == 0
    head_ref.within(f64(y[:, :cols]), ref, bound, dtype)
    assert untouched(y_buf, y, cols, shift)


@pytest.mark.parametrize("rows,cols,pad", [(3000, 1003, 1), (3001, 1003, 0), (12000, 1000, 8), (700000, 8, 0), (300000, 13, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_of_more_than_a_grid(rows, cols, pad, dtype):
    # runs, rows of pieces, and rows gathered into runs
    rng = np.random.default_rng(cols)
    x = rows_apart(rng.standard_normal((rows, cols), dtype=np.float32), cols + pad, 0, dtype)[1][:, :cols]
    r = torch.from_numpy(rng.standard_normal((rows, cols), dtype=np.float32)).to("cuda", DT[dtype])
    y = ms.dropout_fwd(x, 0.1, 7, 8, r)
    ref, bound = head_ref.dropout(f64(x), 0.1, 7, 8, f64(r))
    head_ref.within(f64(y), ref, bound, dtype)


# ---------------------------------------------------------------- row quantisation

# more rows than the grid holds for groups of a thread, 8, 32, 128 and 512 threads, and for the longest rows
@pytest.mark.parametrize("rows,cols", [(400000, 16), (100000, 40), (50000, 200), (100000, 203), (20000, 1024), (15000, 1025), (5000, 4104),
                                       (4000, 4099), (1300, 20000), (1300, 20001), (700, 33001), (700, 40000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("normalize", [False, True])
def test_quantize_more_rows_than_a_grid(rows, cols, dtype, normalize):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    x = x.to(DT[dtype])
    x[::7, cols // 2] = float("inf")           # neighbours of rows that are marked
    q, scale = ms.quantize_rows(x, normalize=normalize)
    assert ms.device_status() == 0
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[::7] = True
    xf = torch.where(bad[:, None], torch.zeros((), device="cuda"), x.float())
    s = (xf.abs().amax(1) * float(np.float32(1) / np.float32(127))).clamp(min=2.0 ** -126)
    # tie and division as in the definition: float32 quotients, rounded to even
    assert torch.equal(q, torch.round(xf / s[:, None]).clamp(-127, 127).to(torch.int8))
    assert bool(torch.isnan(scale[bad]).all())
    got, fine = scale[~bad].double(), xf[~bad].double()
    if normalize:
        want, rel = (s[~bad].double() / fine.norm(dim=1)), (cols / 2 + 12) * head_ref.U
    else:
        want, rel = s[~bad].double(), 0.0
    assert bool(((got - want).abs() <= rel * want).all())


# ---------------------------------------------------------------- INT8 linear

def padded_codes(rng, rows, cols, pad):
    buf = torch.full((rows, cols + pad), 111, dtype=torch.int8, device="cuda")
    buf[:, :cols] = torch.from_numpy(rng.integers(-128, 128, size=(rows, cols)).astype(np.int8))
    return buf[:, :cols]


@pytest.mark.parametrize("M,N,K", [(300, 121, 9000), (300, 124, 9001), (700, 301, 16384), (2500, 302, 9000), (301, 300, 9007), (130, 300, 20001)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 5])
def test_linear_of_few_tiles_cut_along_k(M, N, K, dtype, pad):
    rng = np.random.default_rng(M + N + K + pad)
    x, w = padded_codes(rng, M, K, pad), padded_codes(rng, N, K, pad)
    xs, ws = rng.uniform(0.01, 0.05, M).astype(np.float32), rng.uniform(0.001, 0.002, N).astype(np.float32)
    b = rng.standard_normal(N).astype(np.float32)
    y = ms.linear_int8(x, *(torch.from_numpy(v).cuda() for v in (xs,)), w, *(torch.from_numpy(v).cuda() for v in (ws, b)),
                       out_dtype=DT[dtype])
    assert ms.device_status() == 0
    dot = (x.double() @ w.double().t()).cpu().numpy()                      # exact
    ref = dot * xs.astype(np.float64)[:, None] * ws.astype(np.float64) + b.astype(np.float64)
    # the sum's rounding, two scale products, the bias
    bound = 4 * head_ref.U * np.abs(ref - b) + head_ref.U * np.abs(ref)
    head_ref.within(f64(y), ref, bound, dtype)


@pytest.mark.parametrize("M,N,K,dtype", [(20000, 128, 1024, "f16"), (20000, 64, 2048, "bf16"), (20000, 50, 2048, "f32"), (2500, 302, 9000, "bf16")])
def test_linear_in_a_cuda_graph(M, N, K, dtype):
    # weights kept in shared memory, and slices with their join
    rng = np.random.default_rng(K)
    x, w = padded_codes(rng, M, K, 0), padded_codes(rng, N, K, 0)
    xs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    ms.linear_int8(x, xs, w, ws, out_dtype=DT[dtype])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ms.linear_int8(x, xs, w, ws, out_dtype=DT[dtype])
    for _ in range(3):
        x.copy_(padded_codes(rng, M, K, 0))
        graph.replay()
        assert torch.equal(out, ms.linear_int8(x, xs, w, ws, out_dtype=DT[dtype]))
    assert ms.device_status() == 0


@pytest.mark.parametrize("N", [1, 3, 8, 16, 24])
@pytest.mark.parametrize("swap", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_narrower_than_a_tile(N, swap, dtype):
    # boxes and tiles that reach past the smaller operand's last row; swapped: few tokens, too many for the other kernel
    rng = np.random.default_rng(N)
    M, N, K = (17 + N, 120000, 200) if swap else (120000, N, 200)
    x, w = padded_codes(rng, M, K, 0), padded_codes(rng, N, K, 0)
    y = ms.linear_int8(x, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), out_dtype=DT[dtype])
    assert ms.device_status() == 0
    assert torch.equal(y, (x.double() @ w.double().t()).float().to(DT[dtype]))
