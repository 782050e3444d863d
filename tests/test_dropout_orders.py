"""Second-order gradients of dropout: on the host with stand-ins for the two
kernels, and on the GPU against the same expression in plain operations."""
import pytest
import torch

import maxsim_scoring_gb300 as ms
from maxsim_scoring_gb300 import ops
from tests import head_ref


def plain(x, p, seed, offset, residual=None):
    keep = torch.from_numpy(head_ref.keep_mask(*x.shape, p, seed, offset)).to(x.device)
    t = round(p * 65536)
    y = x * keep * (65536.0 / (65536 - t))
    return y if residual is None else y + residual


@pytest.fixture
def stand_ins(monkeypatch):
    """The kernels' values without a graph, as the kernels give them."""
    def fwd(x, p, seed, offset=0, residual=None, *, out=None):
        with torch.no_grad():
            return plain(x, p, seed, offset, residual).detach()
    monkeypatch.setattr(ops, "dropout_fwd", fwd)
    monkeypatch.setattr(ops, "dropout_bwd", lambda grad, p, seed, offset=0, *, out=None: fwd(grad, p, seed, offset))


def penalty_gradients(x, r, dropout):
    """Gradients of ||d/dx (sum dropout(x, r)^3 + sum x^3)||^2, which need the second derivative."""
    y = dropout(x, 0.25, 5, 6, r)
    (dx,) = torch.autograd.grad((y ** 3).sum() + (x ** 3).sum(), x, create_graph=True)
    return torch.autograd.grad(dx.square().sum(), (x, r))


def test_second_order_on_the_host(stand_ins):
    g = torch.Generator()
    g.manual_seed(1)
    x, r = (torch.randn(6, 11, generator=g, dtype=torch.float64).requires_grad_() for _ in range(2))
    got, want = penalty_gradients(x, r, ms.dropout), penalty_gradients(x, r, plain)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)
    assert torch.autograd.gradcheck(lambda a, b: ms.dropout(a, 0.5, 3, 4, b), (x, r))
    assert torch.autograd.gradgradcheck(lambda a, b: ms.dropout(a, 0.5, 3, 4, b) ** 2, (x, r))
    (dx,) = torch.autograd.grad(ms.dropout(x, 0.5, 3, 4).sum(), x)      # first order alone: no graph kept
    assert not dx.requires_grad


@pytest.mark.gpu
def test_second_order_on_the_gpu():
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x, r = (torch.randn(40, 101, generator=g, device="cuda").requires_grad_() for _ in range(2))
    got = penalty_gradients(x, r, ms.dropout)
    x64, r64 = (t.detach().double().requires_grad_() for t in (x, r))
    want = penalty_gradients(x64, r64, plain)
    # products and sums of at most a few dozen float32 roundings of values of the sizes below
    y = plain(x64, 0.25, 5, 6, r64).abs() + x64.abs()
    size = 24 * 2 * (y.detach() + 1) ** 3 * 4
    for a, b in zip(got, want):
        assert ((a.double() - b).abs() <= 32 * head_ref.U * size).all()
