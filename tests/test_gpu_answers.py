"""The 4-bit head, its index and the answers' probabilities, one after another
as a user calls them."""
import os
import sys

import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import fp4_ref, head_ref, logprobs_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import token_head  # noqa: E402

pytestmark = pytest.mark.gpu


def codes(rng, *shape):
    """Values of 4-bit codes; every block of 32 holds a 6, so that its scale is 1."""
    x = rng.choice(fp4_ref.CODES, size=shape) * rng.choice([-1, 1], size=shape)
    x[..., ::32] = 6
    return x


def test_head_index_scores_and_answers():
    """Hidden states, the 4-bit head, the 4-bit index, MaxSim, probabilities: the head picks columns, so that every
    value up to the scores is exact, and the rest is held to the bounds of 32 bits."""
    rng = np.random.default_rng(4)
    nq, nd, lq, ld, hidden, dim = 9, 40, 7, 33, 256, 128
    q, d = codes(rng, nq, lq, hidden), codes(rng, nd, ld, hidden)
    pick = rng.permutation(hidden)[:dim]
    weight = np.zeros((dim, hidden))
    weight[np.arange(dim), pick] = 1.0
    dev = lambda v: torch.from_numpy(v).to(torch.bfloat16).cuda()  # noqa: E731
    w = ms.quantize_rows_fp4(dev(weight), block=32)
    qe, de = (ms.linear_fp4(*ms.quantize_rows_fp4(dev(v), block=32), *w, block=32) for v in (q, d))
    assert np.array_equal(qe.double().cpu().numpy(), q[..., pick]) and np.array_equal(de.double().cpu().numpy(), d[..., pick])
    index = ms.quantize_rows_fp4(de, block=32)
    back = ms.dequantize_rows_fp4(*index, block=32)
    assert torch.equal(back, de)  # values of one code's grid are held exactly
    scores, _ = ms.maxsim_fwd(qe, back)
    sim = np.einsum("isk,jtk->ijst", q[..., pick], d[..., pick])
    ref = sim.max(axis=3).sum(axis=2)
    assert np.array_equal(scores.double().cpu().numpy(), ref)
    given = torch.arange(nq).cuda()
    logprob, entropy, best, best_logprob, stats = ms.logprobs_fwd(scores, given, scale=0.05, k=5)
    want, err = logprobs_ref.forward(ref, np.arange(nq)[:, None], None, 0.05, 5)
    head_ref.within(logprob.cpu().numpy()[:, None], want["logprob"], err["logprob"], "f32")
    head_ref.within(entropy.cpu().numpy(), want["entropy"], err["entropy"], "f32")
    assert np.array_equal(best.cpu().numpy(), want["top_idx"])
    head_ref.within(best_logprob.cpu().numpy(), want["top_logprob"], err["top_logprob"], "f32")
    dscores = ms.logprobs_bwd(scores, given, None, stats, entropy, grad_logprob=torch.full((nq,), -1 / nq, device="cuda"), scale=0.05)
    dx, bound = logprobs_ref.backward(want, err, np.arange(nq)[:, None], 0.05, np.full((nq, 1), -1 / nq), None, None, None)
    head_ref.within(dscores.cpu().numpy(), dx, bound + np.abs(dx) * 2.0 ** -24, "f32")  # the given gradient is rounded too
    assert ms.device_status() == 0


def test_example_answers_in_4_bits():
    n = 24
    head = token_head.TokenHead(256, 64, seed=3)
    q, d = token_head.synthetic_pairs(n, 16, 48, 256, seed=5, noise=0.5)
    head4 = head.quantized4()
    given = torch.arange(n, device="cuda")
    logprob, entropy, best, best_logprob = token_head.answer(q, token_head.TokenHead.index4(d, head4), head4, given, k=4)
    assert logprob.shape == (n,) and entropy.shape == (n,) and best.shape == (n, 4) and best_logprob.shape == (n, 4)
    assert torch.equal(best[:, 0].long(), given)  # a topic with little noise survives 4 bits
    first = best_logprob[:, 0]
    assert torch.equal(first, logprob) and (best_logprob.diff(dim=1) <= 0).all()
    assert ((entropy >= 0) & (entropy <= np.log(n) + 1e-5)).all()
    # two products and two quantisations away from the 32-bit head
    plain = torch.nn.functional.normalize(d.float() @ head.weight.detach().t(), dim=-1)
    stored = ms.dequantize_rows_fp4(*token_head.TokenHead.index4(d, head4), block=32, out_dtype=torch.float32)
    assert torch.nn.functional.cosine_similarity(plain, stored, dim=-1).min() > 0.9
    assert ms.device_status() == 0
