"""The token head's operators at the ends of their ranges: rows of almost 2^31
elements, matrices of more than 2^31 and 2^32 elements in every layout."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from maxsim_scoring_gb300 import _native
from tests import head_ref

pytestmark = pytest.mark.gpu


def room(n_bytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < n_bytes + (4 << 30):
        pytest.skip("not enough free device memory")


def stream():
    return torch.cuda.current_stream().cuda_stream


def keep_window(first, count, p, seed, offset):
    """The kept elements among first .. first + count - 1 of the row-major matrix."""
    words = head_ref.philox4x32_10(np.arange(first // 8, (first + count + 7) // 8), seed, offset)
    halves = np.stack([words & 0xFFFF, words >> 16], axis=-1).reshape(-1)
    return halves[first % 8:][:count] >= round(p * 65536)


def quantize_chunked(x, step=1 << 27):
    """The definition in float32 on the device, a piece at a time: (codes by piece, scale) of one row."""
    a = max(x[i:i + step].abs().max().float() for i in range(0, len(x), step))
    s = torch.clamp(a * (np.float32(1) / np.float32(127)).item(), min=2.0 ** -126)
    for i in range(0, len(x), step):
        yield i, torch.round(x[i:i + step].float() / s).clamp(-127, 127).to(torch.int8), s


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 15])
def test_quantize_longest_rows(cols):
    # 16-bit rows off their 16-byte boundaries, read in the chunks that they touch: cols plus a chunk's
    # elements passes 32 bits; 2^31 - 8 is read in whole chunks
    room(2 * cols * 3)
    x = torch.zeros((2, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for r in range(2):
        for first in (0, 1 << 20, cols // 2, cols - 5000):
            x[r, first:first + 5000] = torch.randn(5000, generator=g, device="cuda").to(torch.bfloat16)
    x[0, cols - 1], x[1, cols - 2] = 31.0, -17.0               # each row's largest value among its last ones
    q, scale = ms.quantize_rows(x)
    assert ms.device_status() == 0
    for r in range(2):
        for i, want, s in quantize_chunked(x[r]):
            assert torch.equal(q[r, i:i + len(want)], want)
        assert scale[r] == s


def test_dropout_rows_of_almost_32_bits():
    # odd rows apart: a run of 256 elements that starts 31 elements before 2^31 in its row, whose last
    # lane's column passes 32 bits
    rows, cols = 11, 2 ** 31 - 25
    ld = cols + 1
    start = (10 * cols - 1) // 256 * 256 - 9 * cols
    assert start + 31 >= 2 ** 31 > start and start < cols
    room(rows * ld * 2)
    x = torch.ones((rows, ld), dtype=torch.float16, device="cuda")
    x[:, cols] = 5.0
    rc = _native.lib().maxsim_dropout_fwd(x.data_ptr(), _native.F16, rows, cols, ld, None, 0, 0.25, 21, 22, x.data_ptr(), ld,
                                          stream())
    assert rc == 0
    assert (x[:, cols] == 5).all()                              # what lies between the rows
    kept = np.float16(np.float32(65536 / 49152))
    for r in range(rows):
        for first in (0, cols // 3, cols - 2000):
            got = x[r, first:first + 2000].cpu().numpy()
            assert np.array_equal(got, np.where(keep_window(r * cols + first, 2000, 0.25, 21, 22), kept, np.float16(0)))


LARGE = 4_300_001                                               # rows of about 1,000: more than 2^32 elements


@pytest.mark.parametrize("cols,pad_x,pad_y", [(1000, 1, 0), (1000, 8, 8), (1000, 0, 1), (1001, 0, 0)])
def test_dropout_beyond_32_bits_in_every_layout(cols, pad_x, pad_y):
    # rows gathered into a run, rows of pieces, rows of single elements, a run
    ld_x, ld_y = cols + pad_x, cols + pad_y
    room(2 * LARGE * (ld_x + ld_y))
    x = torch.ones((LARGE, ld_x), dtype=torch.float16, device="cuda")
    y = torch.full((LARGE, ld_y), 5.0, dtype=torch.float16, device="cuda")
    x[:, cols:] = float("nan")
    rc = _native.lib().maxsim_dropout_fwd(x.data_ptr(), _native.F16, LARGE, cols, ld_x, None, 0, 0.25, 21, 22, y.data_ptr(), ld_y,
                                          stream())
    assert rc == 0
    assert (y[:, cols:] == 5).all()
    kept = np.float16(np.float32(65536 / 49152))
    for row in (0, 2 ** 31 // cols - 1, 2 ** 31 // cols, 2 ** 31 // cols + 1, 2 ** 32 // cols - 1, 2 ** 32 // cols, LARGE - 1):
        assert np.array_equal(y[row, :cols].cpu().numpy(),
                              np.where(keep_window(row * cols, cols, 0.25, 21, 22), kept, np.float16(0)))
    rate = torch.stack([(y[i:i + (1 << 16), :cols] != 0).sum() for i in range(0, LARGE, 1 << 16)]).sum().item() / (LARGE * cols)
    assert abs(rate - 0.75) < 6 * (0.25 * 0.75 / (LARGE * cols)) ** 0.5


@pytest.mark.parametrize("cols,dtype", [(1000, torch.bfloat16), (1001, torch.bfloat16), (1001, torch.float32)])
def test_quantize_beyond_32_bits(cols, dtype):
    # rows in whole chunks, in the chunks that they touch, in single elements
    room(LARGE * cols * (dtype.itemsize + 1))
    x = torch.empty((LARGE, cols), dtype=dtype, device="cuda")
    for i in range(0, LARGE, 1 << 18):
        x[i:i + (1 << 18)].normal_()
    q, scale = ms.quantize_rows(x)
    for i in range(0, LARGE, 1 << 18):
        part = x[i:i + (1 << 18)].float()
        s = (part.abs().amax(1) * (np.float32(1) / np.float32(127)).item()).clamp(min=2.0 ** -126)
        assert torch.equal(scale[i:i + (1 << 18)], s)
        assert torch.equal(q[i:i + (1 << 18)], torch.round(part / s[:, None]).clamp(-127, 127).to(torch.int8))
