"""Log probabilities of long rows held to single columns: sums of equal values,
one large column in every place, and bounds from the longest chain of additions."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import head_ref, logprobs_ref
from tests.test_gpu_logprobs import full_mask, make

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,pad", [(1, 0), (7, 0), (33, 1), (1000, 0), (2047, 3), (4099, 0), (20000, 0), (32003, 5), (131072, 0), (200001, 1), (300000, 0)])
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_equal_values_are_counted(n, pad, rows, dtype):
    """Every exponential is 1, so the sum is the number of active columns, exactly; its logarithm is off by 2 units of the last place."""
    if rows == 700 and n > 40000:
        rows = 200
    x = torch.full((rows, n + pad), 3.5, dtype=DT[dtype], device="cuda")[:, :n]
    t = torch.full((rows, 2), n - 1, device="cuda")
    t[:, 0] = 0
    g = torch.Generator(device="cuda").manual_seed(n)
    for mask in (None, torch.rand(n, generator=g, device="cuda") < 0.7, torch.rand(rows, n, generator=g, device="cuda") < 0.4):
        for k in (0, 5):
            logprob, entropy, top, _, stats = ms.logprobs_fwd(x, t, mask, k=min(k, n))
            active = torch.ones(rows, n, dtype=torch.bool, device="cuda") if mask is None else mask.expand(rows, n)
            count = active.sum(1).double()
            some = count > 0
            L = torch.log2(count[some])
            # one column more or less is 1.44 / n >= 4.8e-6
            assert ((stats[some, 1].double() - L).abs() <= 2 * 2.0 ** -23 * torch.exp2(torch.floor(torch.log2(L.clamp(min=1))))).all()
            # 2 units of L's last place (2^-18 at most) times ln 2, and three roundings of 12.7
            assert ((entropy[some].double() - L * np.log(2)).abs() <= 2.0 ** -17).all()
            want = torch.where(active[:, [0, n - 1]], -torch.log(count)[:, None], -float("inf"))
            same = torch.isinf(want) == torch.isinf(logprob)
            assert same.all() and (torch.where(torch.isinf(want), 0.0, want - logprob).abs() <= 2.0 ** -17).all()


@pytest.mark.parametrize("n,rows,dtype,step", [(40, 40, "f32", 1), (1000, 1000, "bf16", 1), (1021, 3000, "f16", 1), (4099, 64, "f32", 1), (8195, 700, "bf16", 1),
                                               (16384, 8, "f32", 1), (32003, 8, "bf16", 1), (131072, 8, "bf16", 3), (200001, 4, "f32", 7)])
@pytest.mark.parametrize("masked", [False, True])
def test_one_large_column_in_every_place(n, rows, dtype, step, masked):
    """A column that holds almost all of the row's sum, once in every place (in every step-th, and at every border of 1,024
    columns): its log probability would be far off if it were left out, or counted twice."""
    g = torch.Generator(device="cuda").manual_seed(n)
    places = torch.arange(0, n, step, device="cuda")
    if step > 1:
        edges = torch.arange(0, n, 1024, device="cuda")
        places = torch.cat([places, *((edges + d).clamp(0, n - 1) for d in (-8, -4, -1, 0, 1, 4, 7))])
    places = places[torch.arange(-(-len(places) // rows) * rows, device="cuda") % len(places)]
    mask = (torch.rand(n, generator=g, device="cuda") < 0.5) if masked else None
    x = torch.zeros(rows, n, dtype=DT[dtype], device="cuda")
    row = torch.arange(rows, device="cuda")
    others = n if mask is None else int(mask.sum())
    for at in places.view(-1, rows):
        x[row, at] = 20.0
        logprob, entropy, top, _, _ = ms.logprobs_fwd(x, at, mask, k=2)
        on = torch.ones(rows, dtype=torch.bool, device="cuda") if mask is None else mask[at]
        want = -np.log1p((others - 1) * np.exp(-20.0))  # above -4.2e-4
        # the sum is just above 1: 12 merges lose 2^-24 each, and its own thread's other columns (128 of e^-20 at most) are lost
        assert (torch.where(on, logprob - want, 0.0).abs() < 2e-6).all() and (logprob[~on] == -float("inf")).all()
        assert (torch.where(on, entropy, 0.0) < 0.01).all() and (entropy[~on] > 0.9 * np.log(others)).all()
        assert torch.equal(top[on, 0].long(), at[on])
        x[row, at] = 0.0
    assert ms.device_status() == 0


def chain_bounds(ref, err, x, scale, mask, n):
    """logprobs_ref's bounds with the roundings of the longest chain of additions in place of n: at most n / 256 additions of a
    thread of 128 (two sums each) in a row of its own block, 64 of a warp's thread and of the merges, and an exponential's
    2^-21 for every batch in which the maximum rises (16 columns of a thread or more)."""
    y = np.where(mask != 0, x, -np.inf) if mask is not None else x
    m = y.max(axis=1, keepdims=True)
    d = np.where(np.isfinite(y), scale * (y - m), 0.0)
    p = np.where(np.isfinite(y), ref["p"], 0.0)
    D, L = (p * np.abs(d)).sum(1), np.abs(np.log(np.where(np.isfinite(y), np.exp(d), 0.0).sum(1)))
    rel = 2.0 ** -21 * (9 + n / 2048) + 2 * (n / 256 + 64) * U + 8 * U * D
    lp = 5 * U * np.abs(d) + (rel + 4 * U * L)[:, None]
    return rel, lp, 2 * rel * (1 + D) + 4 * U * (L + D) + 4 * U * D * L


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("mask", [None, "columns", "rows"])
@pytest.mark.parametrize("rows,n,pad,k,scale", [(3, 1024, 0, 0, 1.0), (40, 3000, 1, 2, 0.7), (700, 9001, 3, 0, 1.0), (2, 20000, 0, 64, 2.0), (1, 70001, 0, 20, 1.0),
                                                (2, 131072, 0, 5, 1.0), (3, 300000, 0, 0, 0.3)])
def test_long_rows_within_their_chains(dtype, mask, rows, n, pad, k, scale):
    x, t, m = make(rows + n, rows, n, dtype, 2, mask, pad)
    t[:, 1] = torch.arange(rows, device="cuda") % n
    xd, md = x.double().cpu().numpy(), full_mask(m, x)
    if rows == 3 and mask == "rows":
        m[1], md[1] = True, 1  # make leaves the middle row empty
    if rows == 1 and mask == "rows":
        m[0, : n // 2], md[0, : n // 2] = True, 1
    ref, err = logprobs_ref.forward(xd, t.cpu().numpy(), md, scale, k)
    fine = np.isfinite(ref["lp"]).any(axis=1)
    rel, lp, H = (v[fine] for v in chain_bounds(ref, err, np.where(fine[:, None], xd, 0.0), scale, None if md is None else np.where(fine[:, None], md, 1), n))
    logprob, entropy, top, top_lp, stats = (None if v is None else v.cpu().numpy()[fine] for v in ms.logprobs_fwd(x, t, m, scale=scale, k=k))
    tn = t.cpu().numpy()[fine]
    at = np.take_along_axis(lp, np.maximum(tn, 0), 1)
    head_ref.within(logprob, ref["logprob"][fine], np.where(tn >= 0, at, 0), "f32")
    head_ref.within(entropy, ref["entropy"][fine], H, "f32")
    if k:
        assert np.array_equal(top, ref["top_idx"][fine])
        head_ref.within(top_lp, ref["top_logprob"][fine], np.take_along_axis(lp, np.maximum(top, 0), 1), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [0, 1, 7, 64])
def test_clusters_with_parts_that_are_not_active(dtype, k):
    """Long rows whose active columns all lie in some of the blocks' shares: in front, behind, in the middle, a single one, fewer than k."""
    n = 200000
    g = torch.Generator().manual_seed(k)
    x = torch.randn(6, n, generator=g).to(DT[dtype])
    mask = torch.zeros(6, n, dtype=torch.bool)
    for r, (a, b) in enumerate([(0, 9000), (n - 3000, n), (90000, 100000), (123456, 123457), (50000, 50040), (0, n)]):
        mask[r, a:b] = True
    x[5, 12500:] = -float("inf")
    t = torch.tensor([[5, 8999], [n - 1, n - 3000], [95000, 0], [123456, 7], [50000, 50039], [100, 20000]])
    ref, err = logprobs_ref.forward(x.double().numpy(), t.numpy(), mask.numpy().astype(np.uint8), 1.0, k)
    _, lp, H = chain_bounds(ref, err, x.double().numpy(), 1.0, mask.numpy(), n)
    logprob, entropy, top, top_lp, _ = ms.logprobs_fwd(x.cuda(), t.cuda(), mask.cuda(), k=k)
    head_ref.within(logprob.cpu().numpy(), ref["logprob"], np.take_along_axis(lp, t.numpy(), 1), "f32")
    head_ref.within(entropy.cpu().numpy(), ref["entropy"], H, "f32")
    if k:
        assert np.array_equal(top.cpu().numpy(), ref["top_idx"])
        head_ref.within(top_lp.cpu().numpy(), ref["top_logprob"], np.take_along_axis(lp, np.maximum(ref["top_idx"], 0), 1), "f32")
    assert ms.device_status() == 0
