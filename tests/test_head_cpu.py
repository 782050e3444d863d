"""The token head without a GPU: its references pinned, its entry points'
argument checks, and its binding's refusals."""
import ctypes

import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from maxsim_scoring_gb300 import _native
from maxsim_scoring_gb300 import build as nvbuild
from tests import head_ref

FAKE = 0x10000  # aligned fake device address: never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return _native.lib()


def test_philox_known_answers():
    # the published known-answer vectors of Philox4x32-10
    def one(ctr, key):
        return head_ref.philox4x32_10(np.array([ctr[0] | ctr[1] << 32], dtype=np.uint64), key[0] | key[1] << 32,
                                      ctr[2] | ctr[3] << 32)[0].tolist()
    assert one([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert one([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert one([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_mask_rate_and_independence():
    k = head_ref.keep_mask(400, 500, 0.25, 7, 0)
    n = k.size
    assert abs(k.mean() - 0.75) < 5 * np.sqrt(0.25 * 0.75 / n)
    other = head_ref.keep_mask(400, 500, 0.25, 7, 1)
    agree = (k == other).mean()                    # independent: 0.75^2 + 0.25^2
    assert abs(agree - 0.625) < 5 * np.sqrt(0.625 * 0.375 / n)
    assert head_ref.keep_mask(3, 5, 0.0, 1, 1).all() and not head_ref.keep_mask(3, 5, 1.0, 1, 1).any()


def test_quantize_reference_by_hand():
    q, s, _ = head_ref.quantize(np.array([[127, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1, np.inf, 2, 3]], np.float32), False)
    assert q.tolist() == [[127, -64, 0, 2], [0, 0, 0, 0], [0, 0, 0, 0]]    # ties to even
    assert s[0] == 1.0 and s[1] == 2.0 ** -126 and np.isnan(s[2])
    q, s, _ = head_ref.quantize(np.array([[3.0, 4.0]], np.float32), True)
    assert q.tolist() == [[95, 127]] and np.allclose(q[0] * s[0], [0.6, 0.8], atol=0.5 / 127)


def test_quantize_host_validation(lib):
    f = lib.maxsim_quantize_rows
    # x, dtype, rows, cols, ld_x, normalize, q, ld_q, scale, stream
    assert f(FAKE, 0, 0, 8, 8, 0, FAKE, 8, FAKE, None) == 0             # nothing to do
    assert f(FAKE, 3, 4, 8, 8, 0, FAKE, 8, FAKE, None) == 1             # dtype
    assert f(FAKE, 0, -1, 8, 8, 0, FAKE, 8, FAKE, None) == 1
    assert f(FAKE, 0, 4, -8, 8, 0, FAKE, 8, FAKE, None) == 1
    assert f(FAKE, 0, 4, 8, 7, 0, FAKE, 8, FAKE, None) == 1             # rows overlap
    assert f(FAKE, 0, 4, 8, 8, 0, FAKE, 7, FAKE, None) == 1
    assert f(FAKE, 0, 4, 8, 1 << 60, 0, FAKE, 8, FAKE, None) == 1       # beyond 64-bit addresses
    assert f(FAKE, 0, 1 << 31, 8, 8, 0, FAKE, 8, FAKE, None) == 2
    assert f(None, 0, 4, 8, 8, 0, FAKE, 8, FAKE, None) == 1
    assert f(FAKE, 0, 4, 8, 8, 0, None, 8, FAKE, None) == 1
    assert f(FAKE, 0, 4, 8, 8, 0, FAKE, 8, None, None) == 1
    assert f(FAKE + 1, 0, 4, 8, 8, 0, FAKE, 8, FAKE, None) == 1         # f16 at an odd address
    assert f(FAKE + 2, 2, 4, 8, 8, 0, FAKE, 8, FAKE, None) == 1         # f32 off its alignment
    assert f(FAKE, 0, 4, 8, 8, 0, FAKE, 8, FAKE + 2, None) == 1


def linear(lib, **kw):
    a = dict(x=FAKE, ld_x=64, xs=FAKE, w=FAKE, ld_w=64, ws=FAKE, bias=None, M=4, N=32, K=64, dt=1, out=FAKE, ld_out=32,
             work=FAKE, work_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.maxsim_linear_int8(*a.values())


def test_linear_host_validation(lib):
    assert linear(lib, M=0) == 0 and linear(lib, N=0) == 0              # nothing to do
    assert linear(lib, dt=5) == 1
    assert linear(lib, M=-1) == 1 and linear(lib, N=-1) == 1 and linear(lib, K=-1) == 1
    assert linear(lib, ld_x=63) == 1 and linear(lib, ld_w=63) == 1 and linear(lib, ld_out=31) == 1
    assert linear(lib, K=131072, ld_x=131072, ld_w=131072) == 2         # the sum would pass 32 bits
    assert linear(lib, M=1 << 31) == 2
    assert linear(lib, out=None) == 1 and linear(lib, out=FAKE + 1) == 1
    assert linear(lib, dt=2, out=FAKE + 2) == 1
    assert linear(lib, xs=None) == 1 and linear(lib, ws=None) == 1 and linear(lib, xs=FAKE + 2) == 1
    assert linear(lib, bias=FAKE + 2) == 1
    assert linear(lib, x=None) == 1 and linear(lib, w=None) == 1


def test_linear_workspace_sizes(lib):
    size = lib.maxsim_workspace_size
    assert size(11, -1, 8, 8, 8, 8) == ctypes.c_size_t(-1).value
    assert size(11, 4, 8, 131072, 131072, 131072) == ctypes.c_size_t(-1).value
    assert size(11, 4, 64, 64, 64, 64) != ctypes.c_size_t(-1).value


def test_dropout_host_validation(lib):
    f, b = lib.maxsim_dropout_fwd, lib.maxsim_dropout_bwd
    def fwd(**kw):
        a = dict(x=FAKE, dt=0, rows=4, cols=8, ld=8, res=None, ld_r=0, p=0.1, seed=1, offset=0, y=FAKE, ld_y=8, st=None)
        a.update(kw)
        return f(*a.values())
    assert fwd(rows=0) == 0 and fwd(cols=0) == 0                        # nothing to do
    assert fwd(dt=9) == 1 and fwd(rows=-1) == 1 and fwd(cols=-1) == 1
    for p in (-0.01, 1.01, float("nan"), float("inf")):
        assert fwd(p=p) == 1
    assert fwd(ld=7) == 1 and fwd(ld_y=7) == 1 and fwd(res=FAKE, ld_r=7) == 1
    assert fwd(x=None) == 1 and fwd(y=None) == 1
    assert fwd(x=FAKE + 1) == 1 and fwd(y=FAKE + 1) == 1 and fwd(res=FAKE + 1, ld_r=8) == 1
    assert fwd(rows=1 << 31) == 2
    assert b(FAKE, 0, 4, 8, 8, 2.0, 1, 0, FAKE, 8, None) == 1
    assert b(FAKE, 0, 0, 8, 8, 0.5, 1, 0, FAKE, 8, None) == 0


def test_binding_refusals():
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        ms.quantize_rows(cpu)                                           # not on a GPU
    with pytest.raises(TypeError):
        ms.quantize_rows(cpu.double())
    with pytest.raises(TypeError):
        ms.dropout_fwd(cpu.int(), 0.1, 0)
    with pytest.raises(ValueError):
        ms.dropout_fwd(cpu, 0.1, 0)
    with pytest.raises(ValueError):
        ms.dropout_fwd(cpu, 0.1, 0, residual=torch.zeros(8))            # no broadcasting
    with pytest.raises(TypeError):
        ms.dropout_bwd(cpu.int(), 0.1, 0)
    i8, s = torch.zeros(4, 8, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError):
        ms.linear_int8(i8, s, i8, s)
    with pytest.raises(TypeError):
        ms.linear_int8(cpu, s, i8, s)
    with pytest.raises(TypeError):
        ms.linear_int8(i8, s.double(), i8, s)
    with pytest.raises(TypeError):
        ms.linear_int8(i8, s, i8, s, out_dtype=torch.int8)
