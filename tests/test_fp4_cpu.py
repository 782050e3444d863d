"""The 4-bit rows and the log probabilities without a GPU: their references
pinned, their entry points' argument checks, their binding's refusals."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from maxsim_scoring_gb300 import _native
from maxsim_scoring_gb300 import build as nvbuild
from tests import fp4_ref, logprobs_ref
from tests.test_devices_cpu import fake  # noqa: F401

FAKE = 0x10000  # aligned fake device address: never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return _native.lib()


def test_tables():
    assert fp4_ref.E4M3[0] == 0 and fp4_ref.E4M3[1] == 2.0 ** -9 and fp4_ref.E4M3[56] == 1 and fp4_ref.E4M3[126] == 448
    own = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(fp4_ref.E4M3, own)
    v = np.array([0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.01, 9])
    assert fp4_ref.CODES[fp4_ref.round_quotient(v, np.ones(11), fp4_ref.CODES)].tolist() == [0, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6]
    assert np.array_equal(fp4_ref.nearest(v, fp4_ref.CODES), fp4_ref.round_quotient(v, np.ones(11), fp4_ref.CODES))


def test_quantize_reference_by_hand():
    x = np.zeros((2, 33))
    x[0, :4] = [6, -3, 0.25, 0.26]
    x[0, 32] = 0.375                       # 2^-2 * 1.5: unit 2^-4, code 6
    x[1, 5] = np.inf
    q, byte, row = fp4_ref.quantize(x, 32)
    assert row is None and byte.tolist() == [[127, 123], [255, 119 - 119]]
    assert q.shape == (2, 32) and q[0, :2].tolist() == [0xD7, 0x10] and q[0, 16] == 7 and not q[1].any()
    x = np.zeros((1, 16))
    x[0, 0], x[0, 1], x[0, 2] = 2688, 448 * 2.5, -448 * 2.51
    q, byte, row = fp4_ref.quantize(x, 16)
    assert row.tolist() == [1.0] and byte.tolist() == [[126]] and q[0, :2].tolist() == [0x47, 0x0D]
    v = fp4_ref.values(q, byte, 16)
    assert v[0, :3].tolist() == [2688, 896, -1344]
    assert fp4_ref.tiles(np.arange(10, dtype=np.uint8)[None])[0, 2, 0, 0].tolist() == [8, 9, 0, 0]


def test_logprobs_reference_by_hand():
    x = np.log(np.array([[1.0, 2, 5], [1, 1, 2]]))
    out, _ = logprobs_ref.forward(x, np.array([[2, -1], [0, 1]]), np.array([[1, 1, 1], [1, 0, 1]]), 1.0, 3)
    assert np.allclose(out["logprob"][0], [np.log(5 / 8), 0]) and np.isclose(out["logprob"][1, 0], np.log(1 / 3))
    assert out["logprob"][1, 1] == -np.inf
    assert np.isclose(out["entropy"][0], -(1 / 8 * np.log(1 / 8) + 2 / 8 * np.log(2 / 8) + 5 / 8 * np.log(5 / 8)))
    assert out["top_idx"].tolist() == [[2, 1, 0], [2, 0, -1]]


@pytest.mark.parametrize("mask", [False, True])
def test_logprobs_gradient_reference_against_differences(mask):
    rng = np.random.default_rng(0)
    x, t = rng.standard_normal((4, 9)), np.array([[0, 3], [8, 8], [-1, 2], [5, -1]])
    m = np.ones((4, 9), dtype=np.uint8)
    if mask:
        m[:, 1] = 0
        m[1, 7] = 0
    g, ge, gt = rng.standard_normal((4, 2)), rng.standard_normal(4), rng.standard_normal((4, 3))

    def loss(x):
        out, _ = logprobs_ref.forward(x, t, m, 1.3, 3)
        return (np.where(np.isfinite(out["logprob"]), out["logprob"], 0) * g).sum() + (out["entropy"] * ge).sum() + (out["top_logprob"] * gt).sum()
    out, err = logprobs_ref.forward(x, t, m, 1.3, 3)
    dx, _ = logprobs_ref.backward(out, err, t, 1.3, g, ge, gt, m)
    for r in range(4):
        for j in range(9):
            h = np.zeros_like(x)
            h[r, j] = 1e-5
            assert abs((loss(x + h) - loss(x - h)) / 2e-5 - dx[r, j]) < 1e-7


def test_quantize_host_validation(lib):
    def quant(**kw):
        a = dict(x=FAKE, dt=0, rows=4, cols=64, ld=64, block=16, q=FAKE, ld_q=32, b=FAKE, s=FAKE, st=None)
        a.update(kw)
        return lib.maxsim_quantize_rows_fp4(*a.values())
    assert quant(rows=0) == 0
    assert quant(dt=3) == 1 and quant(block=8) == 1 and quant(rows=-1) == 1 and quant(cols=-1) == 1
    assert quant(ld=63) == 1 and quant(ld_q=31) == 1 and quant(ld_q=40) == 1 and quant(cols=65, ld=65) == 1
    assert quant(ld=1 << 60) == 1
    assert quant(rows=(1 << 31) - 1) == 2 and quant(cols=(1 << 31) - 1, ld=1 << 31, ld_q=1 << 31) == 2
    assert quant(x=None) == 1 and quant(q=None) == 1 and quant(b=None) == 1 and quant(s=None) == 1
    assert quant(x=FAKE + 1) == 1 and quant(q=FAKE + 8) == 1 and quant(b=FAKE + 4) == 1 and quant(s=FAKE + 2) == 1


def test_dequantize_host_validation(lib):
    def deq(**kw):
        a = dict(q=FAKE, ld_q=32, b=FAKE, s=None, rows=4, cols=64, block=32, dt=1, y=FAKE, ld_y=64, st=None)
        a.update(kw)
        return lib.maxsim_dequantize_rows_fp4(*a.values())
    assert deq(rows=0) == 0 and deq(cols=0) == 0
    assert deq(dt=3) == 1 and deq(block=64) == 1 and deq(rows=-1) == 1 and deq(cols=-1) == 1
    assert deq(ld_y=63) == 1 and deq(ld_q=31) == 1 and deq(ld_q=33) == 1
    assert deq(rows=(1 << 31) - 1) == 2
    assert deq(q=None) == 1 and deq(b=None) == 1 and deq(y=None) == 1
    assert deq(q=FAKE + 8) == 1 and deq(b=FAKE + 8) == 1 and deq(s=FAKE + 1) == 1 and deq(y=FAKE + 1) == 1


def test_linear_host_validation(lib):
    def linear(**kw):
        a = dict(x=FAKE, ld_x=32, xb=FAKE, xs=None, w=FAKE, ld_w=32, wb=FAKE, ws=None, bias=None, M=4, N=8, K=64, block=16, dt=1,
                 out=FAKE, ld_out=8, st=None)
        a.update(kw)
        return lib.maxsim_linear_fp4(*a.values())
    assert linear(M=0) == 0 and linear(N=0) == 0
    assert linear(dt=7) == 1 and linear(block=0) == 1 and linear(M=-1) == 1 and linear(N=-1) == 1 and linear(K=-32) == 1
    assert linear(K=48) == 1 and linear(ld_x=16) == 1 and linear(ld_w=40) == 1 and linear(ld_out=7) == 1
    assert linear(M=1 << 31) == 2 and linear(K=1 << 31, ld_x=1 << 31, ld_w=1 << 31) == 2
    assert linear(K=(1 << 28) + 32, ld_x=1 << 28, ld_w=1 << 28) == 2 and linear(ld_x=1 << 40) == 2 and linear(ld_w=1 << 40) == 2
    assert linear(x=None) == 1 and linear(w=None) == 1 and linear(xb=None) == 1 and linear(wb=None) == 1 and linear(out=None) == 1
    assert linear(x=FAKE + 8) == 1 and linear(w=FAKE + 1) == 1 and linear(xb=FAKE + 8) == 1 and linear(wb=FAKE + 4) == 1
    assert linear(xs=FAKE + 2) == 1 and linear(ws=FAKE + 2) == 1 and linear(bias=FAKE + 2) == 1 and linear(out=FAKE + 1) == 1


def logprobs(lib, **kw):
    a = dict(x=FAKE, dt=2, rows=4, n=100, ld=100, t=FAKE, T=1, mask=None, ld_mask=0, scale=1.0, k=5, lp=FAKE, h=FAKE, ti=FAKE,
             tl=FAKE, stats=FAKE, st=None)
    a.update(kw)
    return lib.maxsim_logprobs_fwd(*a.values())


def logprobs_bwd(lib, **kw):
    a = dict(x=FAKE, dt=2, rows=4, n=100, ld=100, t=FAKE, T=1, mask=None, ld_mask=0, scale=1.0, stats=FAKE, h=FAKE, g=FAKE, gh=FAKE,
             ti=FAKE, gt=FAKE, k=5, dx=FAKE, ld_dx=100, st=None)
    a.update(kw)
    return lib.maxsim_logprobs_bwd(*a.values())


@pytest.mark.parametrize("f", [logprobs, logprobs_bwd])
def test_logprobs_host_validation(lib, f):
    assert f(lib, rows=0) == 0
    assert f(lib, dt=4) == 1 and f(lib, rows=-1) == 1 and f(lib, n=0, ld=0) == 1 and f(lib, T=-1) == 1 and f(lib, k=-1) == 1
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e300, 1e-300):
        assert f(lib, scale=scale) == 1
    assert f(lib, ld=99) == 1 and f(lib, mask=FAKE, ld_mask=99) == 1 and f(lib, k=101) == 1
    assert f(lib, k=65) == 2 and f(lib, T=257) == 2 and f(lib, rows=1 << 31) == 2
    assert f(lib, n=(1 << 31) - 1, ld=1 << 31, **({"ld_dx": 1 << 31} if f is logprobs_bwd else {})) == 2
    assert f(lib, x=None) == 1 and f(lib, x=FAKE + 2) == 1 and f(lib, t=None) == 1 and f(lib, t=FAKE + 4) == 1
    assert f(lib, h=None) == 1 and f(lib, stats=None) == 1 and f(lib, stats=FAKE + 2) == 1 and f(lib, ti=None) == 1
    if f is logprobs:
        assert f(lib, lp=None) == 1 and f(lib, tl=None) == 1 and f(lib, tl=FAKE + 1) == 1
    else:
        assert f(lib, dx=None) == 1 and f(lib, dx=FAKE + 2) == 1 and f(lib, ld_dx=99) == 1 and f(lib, gt=FAKE + 2) == 1


def test_logprobs_gradient_over_the_logits(lib):
    """Every warp reads the given columns' logits, so the gradient may not share elements with them."""
    f = lambda **kw: logprobs_bwd(lib, **kw)  # noqa: E731
    assert f(dx=FAKE) == 1 and f(dx=FAKE + 4) == 1 and f(dx=FAKE + 4 * 399) == 1 and f(dx=FAKE + 4 * 200, rows=1, n=201, ld=201, ld_dx=201) == 1
    assert f(x=FAKE + 4 * 50, dx=FAKE, ld=250, ld_dx=250) == 1          # columns that overlap, of one buffer
    assert f(dx=FAKE + 4 * 100, ld=200, ld_dx=250) == 1                 # rows that meet somewhere


def test_binding_refusals():
    cpu = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        ms.quantize_rows_fp4(cpu)                                       # not on a GPU
    with pytest.raises(TypeError):
        ms.quantize_rows_fp4(cpu.double())
    with pytest.raises(ValueError):
        ms.quantize_rows_fp4(cpu, block=64)
    with pytest.raises(ValueError):
        ms.quantize_rows_fp4(cpu, block=32, scale=torch.ones(4))
    q, b = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ms.dequantize_rows_fp4(q, b)
    with pytest.raises(TypeError):
        ms.dequantize_rows_fp4(q, b, out_dtype=torch.int8)
    with pytest.raises(ValueError):
        ms.linear_fp4(q, b, None, q, b, None)
    with pytest.raises(TypeError):
        ms.linear_fp4(q, b, None, q, b, None, out_dtype=torch.int8)
    with pytest.raises(ValueError):
        ms.logprobs_fwd(cpu, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        ms.logprobs_fwd(cpu.double(), None)
    with pytest.raises(TypeError):
        ms.logprobs_bwd(cpu.double(), None, None, cpu, cpu)


def test_binding_refusals_on_a_device(fake):  # noqa: F811
    """What the binding asks of its operands once they are on a GPU."""
    x = torch.zeros(4, 64)
    q, b, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), torch.ones(4)
    t = torch.zeros(4, dtype=torch.int64)
    for wrong, kind in [
            (lambda: ms.quantize_rows_fp4(x, q=q[:3]), ValueError), (lambda: ms.quantize_rows_fp4(x, block_scale=b.float()), ValueError),
            (lambda: ms.dequantize_rows_fp4(q, b[:, :, :16], s), ValueError), (lambda: ms.dequantize_rows_fp4(q.int(), b, s), TypeError),
            (lambda: ms.dequantize_rows_fp4(q, b, s.double()), TypeError), (lambda: ms.dequantize_rows_fp4(q, b, s[:3]), ValueError),
            (lambda: ms.dequantize_rows_fp4(q, b, s, cols=32), ValueError), (lambda: ms.dequantize_rows_fp4(q, b, s, cols=65), ValueError),
            (lambda: ms.dequantize_rows_fp4(q[:, :20], b, s), ValueError), (lambda: ms.dequantize_rows_fp4(q, b, s, block=8), ValueError),
            (lambda: ms.linear_fp4(q, b, s, q[:, :16], b, s), ValueError), (lambda: ms.linear_fp4(q, b, s, q[0], b, s), ValueError),
            (lambda: ms.linear_fp4(q, b, s, q, b, s, torch.zeros(5)), ValueError), (lambda: ms.linear_fp4(q, b, s, q, b, s, s.half()), TypeError),
            (lambda: ms.linear_fp4(q, b, s, q, b, s, out=torch.zeros(4, 4)), ValueError),
            (lambda: ms.logprobs_fwd(x[:, :0], None), ValueError), (lambda: ms.logprobs_fwd(x, t.float()), TypeError),
            (lambda: ms.logprobs_fwd(x, t[:3]), ValueError), (lambda: ms.logprobs_fwd(x, t, x), TypeError),
            (lambda: ms.logprobs_fwd(x, t, torch.ones(63, dtype=torch.bool)), ValueError),
            (lambda: ms.logprobs_bwd(x, t, None, torch.zeros(4, 3), s), ValueError),
            (lambda: ms.logprobs_bwd(x, None, None, torch.zeros(4, 2), s, grad_logprob=s), ValueError),
            (lambda: ms.logprobs_bwd(x, t, None, torch.zeros(4, 2), s, grad_logprob=s.double()), TypeError),
            (lambda: ms.logprobs_bwd(x, t, None, torch.zeros(4, 2), s, grad_top=torch.zeros(4, 2)), ValueError),
            (lambda: ms.logprobs_bwd(x, t, None, torch.zeros(4, 2), s, out=torch.zeros(4, 63)), ValueError)]:
        with pytest.raises(kind):
            wrong()


def test_tensors_on_another_device(fake):  # noqa: F811
    devices, library = fake
    x, t, s = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64), torch.ones(4)
    q, b = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8)
    ms.quantize_rows_fp4(x)
    ms.dequantize_rows_fp4(q, b, s)
    ms.linear_fp4(q, b, s, q, b, s, s)
    ms.logprobs_fwd(x, t, k=2)
    ms.logprobs_bwd(x, t, None, torch.zeros(4, 2), s, grad_logprob=s)
    assert library.calls == [(name, 1, 101) for name in ("maxsim_quantize_rows_fp4", "maxsim_dequantize_rows_fp4", "maxsim_linear_fp4",
                                                         "maxsim_logprobs_fwd", "maxsim_logprobs_bwd")]
    assert devices.current == 0
