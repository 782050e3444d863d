"""The token head end to end (examples/token_head.py): its training gradient
against a plain one, and its INT8 serving path against the 64-bit one."""
import os
import sys

import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import head_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import token_head  # noqa: E402

pytestmark = pytest.mark.gpu


def test_head_gradient_against_plain_form():
    # the head's gradient with the same masks applied by hand, in float64 from the dropped-out hidden states on
    n, lq, ld, hidden, dim = 6, 5, 9, 64, 32
    head = token_head.TokenHead(hidden, dim, p=0.25, seed=3)
    q, d = token_head.synthetic_pairs(n, lq, ld, hidden, seed=2)
    before = head.weight.detach().clone()
    head.train_step(q, d, lr=1.0)
    got = (before - head.weight.detach()).double().cpu()

    w = before.to(torch.bfloat16).double().cpu().requires_grad_()
    def embed(h, stream):
        x, _ = head_ref.dropout(h.double().cpu().numpy().reshape(-1, hidden), 0.25, 3, stream)
        x = torch.from_numpy(x).to(torch.bfloat16).double().reshape(h.shape)
        return torch.nn.functional.normalize(x @ w.t(), dim=-1)
    qe, de = embed(q, 0), embed(d, 1)
    sim = torch.einsum("isk,jtk->ijst", qe, de)
    scores = sim.amax(dim=3).sum(dim=2) / (lq * 0.1)
    loss = torch.nn.functional.cross_entropy(scores, torch.arange(n))
    (ref,) = torch.autograd.grad(loss, w)
    # embeddings, their gradients and the projection's products are bf16 on the GPU: a handful of
    # roundings of 2^-8 each, and a maximum that they may move to another token; the direction holds
    cos = torch.nn.functional.cosine_similarity(got.flatten(), ref.flatten(), dim=0).item()
    assert cos > 0.98
    assert abs(got.norm().item() / ref.norm().item() - 1) < 0.1


def test_int8_index_against_64_bits():
    n, ld, hidden, dim = 7, 33, 256, 128
    head = token_head.TokenHead(hidden, dim, seed=5)
    _, d = token_head.synthetic_pairs(n, 4, ld, hidden, seed=6)
    served = head.quantized()
    q8, scale = token_head.TokenHead.index(d, served)
    assert ms.device_status() == 0
    assert q8.shape == (n, ld, dim) and q8.dtype == torch.int8 and scale.shape == (n, ld)
    got = q8.double().cpu() * scale.double().cpu()[..., None]
    x = d.double().cpu()
    ref = torch.nn.functional.normalize(x @ head.weight.detach().double().cpu().t(), dim=-1)
    # each of the three quantisations moves a value by at most half a step of its row: s / 2
    # (hidden and weights 1/254 of their row's largest, embeddings 1/254 of theirs)
    xs = x.abs().amax(-1, keepdim=True) / 254
    wm = head.weight.detach().double().cpu()
    ws = wm.abs().amax(-1) / 254
    raw = x @ wm.t()
    err = xs * wm.abs().sum(-1) + x.abs().sum(-1, keepdim=True) * ws + hidden * xs * ws     # of the product
    err = err + raw.abs() * 2.0 ** -11                                                       # its rounding to f16
    norm = raw.norm(dim=-1, keepdim=True)
    unit = err / norm + ref.abs() * (err.norm(dim=-1, keepdim=True) / norm)                  # of the unit row
    unit = unit * 1.2 + ref.abs().amax(-1, keepdim=True) / 254 * 1.2                         # second order; the last step
    assert ((got - ref).abs() <= unit).all()
    assert np.allclose(got.norm(dim=-1).numpy(), 1.0, atol=0.02)


def test_example_learns_and_serves():
    losses, hit = token_head.main(n=32, lq=16, ld=40, hidden=512, dim=64, steps=12)
    assert losses[-1] < losses[0]
    assert hit == 1.0
