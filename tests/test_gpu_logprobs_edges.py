"""Log probabilities and their gradient where rows are broken, empty or given
gradients that are not finite."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# a warp a row, a block a row, the blocks of a cluster a row
COLUMNS = [40, 3000, 200000]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", COLUMNS)
@pytest.mark.parametrize("k", [0, 3])
def test_minus_infinity_in_a_broken_row(dtype, n, k):
    """A row that holds a NaN or plus infinity gives NaN for its active columns of minus infinity too."""
    x = torch.randn(6, n, generator=torch.Generator().manual_seed(n)).to(dtype)
    t = torch.tensor([[2, 5, -1, n - 1]]).repeat(6, 1)
    mask = torch.ones(6, n, dtype=torch.bool)
    x[:, 2] = -INF            # given, and active but in rows 1 and 3
    mask[1, 2] = mask[3, 2] = False
    x[0, 7] = x[1, 7] = NAN
    x[2, n - 3] = x[3, n - 3] = INF
    x[4] = -INF               # empty
    x[4, 9], mask[4, 9] = NAN, False
    want = torch.full((6, 4), NAN)
    want[:, 2] = 0
    want[1, 0] = want[3, 0] = -INF
    want[4, [0, 1, 3]] = -INF
    y = x[5].double()
    lp = (y - torch.logsumexp(y, 0))[t[5].clamp(min=0)]
    x, t, mask = x.cuda(), t.cuda(), mask.cuda()
    logprob, entropy, _, _, stats = ms.logprobs_fwd(x, t, mask, k=k)
    got = logprob.cpu()
    assert np.array_equal(got[:5].numpy(), want[:5].numpy(), equal_nan=True)
    assert got[5, 0] == -INF and got[5, 2] == 0
    # units of 2^-24: a thread's sum and the merges 64, exponentials 4 and their arguments 60, the logarithm 34, the difference 50
    assert (got[5, [1, 3]].double() - lp[[1, 3]]).abs().max() < 2.0 ** -16
    assert entropy[:4].isnan().all() and entropy[4] == 0
    # without a mask: rows 0 and 2 again
    assert torch.equal(ms.logprobs_fwd(x[::2], t[::2], k=k)[0][:2].isnan(), want[[0, 2]].isnan().cuda())
    dx = ms.logprobs_bwd(x, t, mask, stats, entropy, grad_logprob=torch.ones(6, 4, device="cuda"))
    assert dx[:4][mask[:4]].isnan().all() and not dx[:4][~mask[:4]].any() and not dx[4].any() and dx[5].isfinite().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,pad", [(40, 0), (41, 3), (3000, 0), (3001, 3)])
def test_gradients_that_are_not_finite(dtype, n, pad):
    """They reach their own row's active columns; inactive ones and rows without any are 0, other rows as without them."""
    g = torch.Generator().manual_seed(n)
    x = torch.randn(8, n + pad, generator=g).to(dtype).cuda()[:, :n]
    mask = (torch.rand(8, n, generator=g) < 0.6).cuda()
    mask[:, 5] = True
    mask[6] = False
    x[7] = -INF
    t = torch.full((8, 2), 5).cuda()
    t[:, 1] = n - 1
    _, h, top, _, st = ms.logprobs_fwd(x, t, mask, k=2)
    gl, ge, gt = torch.randn(8, 2, generator=g).cuda(), torch.randn(8, generator=g).cuda(), torch.randn(8, 2, generator=g).cuda()
    fine = ms.logprobs_bwd(x, t, mask, st, h, grad_logprob=gl, grad_entropy=ge, top_idx=top, grad_top=gt)
    gl[0, 0], ge[1], gt[2, 1], gl[6], ge[7] = INF, NAN, -INF, NAN, INF
    ge[3], gl[7, 0] = INF, NAN
    dx = ms.logprobs_bwd(x, t, mask, st, h, grad_logprob=gl, grad_entropy=ge, top_idx=top, grad_top=gt)
    assert not dx[~mask].any() and not dx[6:].any()
    assert torch.equal(dx[4:6], fine[4:6])
    for r in range(4):
        assert not dx[r][mask[r]].isfinite().any()
    plain = ms.logprobs_fwd(x, t)
    dx = ms.logprobs_bwd(x, t, None, plain[4], plain[1], grad_logprob=gl, grad_entropy=ge)
    assert not dx[7].any() and dx[4:6].isfinite().all()


@pytest.mark.parametrize("low", [-1e29, -1e20, -7e4])
def test_large_entropy_gradient_beside_masked_values(low):
    """Logits masked by a large negative value have p = 0 and pass nothing, however large the entropy's gradient."""
    x = torch.randn(3, 3000, generator=torch.Generator().manual_seed(2)).cuda()
    x[:, 1000:] = low
    _, h, _, _, st = ms.logprobs_fwd(x, None)
    ge = torch.tensor([1.0, 1e12, -1e20], device="cuda")
    dx = ms.logprobs_bwd(x, None, None, st, h, grad_entropy=ge)
    assert not dx[:, 1000:].any() and dx.isfinite().all()
    lp = torch.log_softmax(x.double(), 1)
    p, inner = lp.exp(), lp - (lp.exp() * lp.clamp(min=-1e6)).sum(1, keepdim=True)
    # log p is known to 2^-16 (as above), the entropy to 2^-15 and p to 2^-15 of itself
    near = (dx.double() + ge.double()[:, None] * p * inner).abs() <= ge.double().abs()[:, None] * p * (1 + inner.abs()) * 2.0 ** -14
    assert near[:, :1000].all()
