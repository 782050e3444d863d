"""Log probabilities, entropies, strongest columns and the gradient on the GPU
against float64 within derived bounds; masks, ties, infinities and empty rows."""
import numpy as np
import pytest
import torch

import maxsim_scoring_gb300 as ms
from tests import head_ref, logprobs_ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, rows, n, dtype, T=1, mask=None, pad=0, spread=3.0, levels=None, offset=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n + pad, generator=g) * spread + 10 * torch.rand(rows, 1, generator=g)
    if levels:
        x = torch.randint(0, levels, (rows, n + pad), generator=g).float()
    flat = torch.zeros(offset + x.numel(), dtype=DT[dtype])
    flat[offset:] = x.to(DT[dtype]).reshape(-1)
    x = flat.cuda()[offset:].view(rows, n + pad)[:, :n]
    t = torch.randint(0, n, (rows, T), generator=g)
    t[torch.rand(rows, T, generator=g) < 0.15] = -1
    m = None
    if mask == "columns":
        m = torch.rand(n, generator=g) < 0.8
    elif mask == "rows":
        m = torch.rand(rows, n, generator=g) < 0.7
        m[rows // 2] = False
    return x, t.cuda(), None if m is None else m.cuda()


def full_mask(m, x):
    return None if m is None else m.expand(x.shape).cpu().numpy().astype(np.uint8)


def compare(x, t, m, scale, k, way="step", seed=0):
    rows, n = x.shape
    ref, err = logprobs_ref.forward(x.double().cpu().numpy(), t.cpu().numpy(), full_mask(m, x), scale, k)
    logprob, entropy, top_idx, top_logprob, stats = ms.logprobs_fwd(x, t, m, scale=scale, k=k)
    head_ref.within(logprob.cpu().numpy(), ref["logprob"], err["logprob"], "f32")
    head_ref.within(entropy.cpu().numpy(), ref["entropy"], err["entropy"], "f32")
    if k:
        assert np.array_equal(top_idx.cpu().numpy(), ref["top_idx"])
        head_ref.within(top_logprob.cpu().numpy(), ref["top_logprob"], err["top_logprob"], "f32")
    else:
        assert top_idx is None and top_logprob is None
    if way != "step":
        return
    g = torch.Generator().manual_seed(seed)
    gl, ge = torch.randn(t.shape, generator=g), torch.randn(rows, generator=g)
    gt = torch.randn(rows, k, generator=g) if k else None
    for use in ((1, 0, 0), (1, 1, 1), (0, 1, 0), (0, 0, 1)):
        if use == (0, 0, 1) and not k:
            continue
        a, b, c = gl if use[0] else None, ge if use[1] else None, gt if use[2] and k else None
        f = lambda v: None if v is None else v.cuda()  # noqa: E731
        d = lambda v: None if v is None else v.double().numpy()  # noqa: E731
        dx = ms.logprobs_bwd(x, t, m, stats, entropy, grad_logprob=f(a), grad_entropy=f(b), top_idx=top_idx, grad_top=f(c), scale=scale)
        want, bound = logprobs_ref.backward(ref, err, t.cpu().numpy(), scale, d(a), d(b), d(c), full_mask(m, x))
        assert dx.dtype == x.dtype and dx.shape == x.shape
        name = {v: s for s, v in DT.items()}[x.dtype]
        head_ref.within(dx.double().cpu().numpy(), want, bound, name)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("mask", [None, "columns", "rows"])
@pytest.mark.parametrize("rows,n,pad,T,k,scale", [
    (1, 1, 0, 1, 1, 1.0), (3, 2, 1, 2, 0, 0.5), (64, 64, 0, 1, 0, 10.0), (5, 100, 3, 3, 5, 1.0), (9, 257, 0, 1, 64, 1.0),
    (17, 1000, 24, 8, 20, 0.7), (4, 2049, 0, 1, 0, 1.0), (4, 2048, 1, 1, 0, 2.0), (3, 4099, 5, 1, 1, 1.0), (2, 20000, 0, 4, 64, 3.0),
    (1, 70001, 0, 1, 20, 1.0), (40, 3000, 1, 256, 2, 0.1), (2, 131072, 0, 1, 5, 1.0)])
def test_against_float64(dtype, mask, rows, n, pad, T, k, scale):
    x, t, m = make(rows * 101 + n, rows, n, dtype, T, mask, pad)
    compare(x, t, m, scale, min(k, n), seed=n)


@pytest.mark.parametrize("n,k", [(7, 7), (300, 64), (5000, 64), (50000, 33), (300000, 64), (300000, 1)])
@pytest.mark.parametrize("levels", [1, 2, 5])
def test_ties(n, k, levels):
    """Rows of few values: the lowest columns among equal ones, whatever threads and blocks they fall to."""
    x, t, _ = make(n + levels, 3, n, "bf16", levels=levels)
    compare(x, t, None, 1.0, k, way="fwd")


@pytest.mark.parametrize("n,step", [(65536, 512 * 8), (65536, 128 * 8), (200000, 512 * 8), (1 << 20, 512 * 4), (30000, 1), (30000, 7)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strongest_in_few_threads(n, step, dtype):
    """Large values a fixed stride apart, ascending and descending: all of them may belong to a few threads."""
    x = torch.zeros(2, n)
    at = torch.arange(0, n, step)
    for e in range(4):
        at2 = (at + e).clamp(max=n - 1)
        x[0, at2] = 5 + torch.linspace(0, 1, len(at2))
        x[1, at2] = 5 - torch.linspace(0, 1, len(at2))
    compare(x.to(DT[dtype]).cuda(), torch.zeros(2, 1, dtype=torch.int64).cuda(), None, 1.0, 64, way="fwd")


def test_masked_places_and_infinities():
    inf, nan = float("inf"), float("nan")
    for n in (40, 3000):
        for dtype in ("f32", "f16", "bf16"):
            low = torch.finfo(DT[dtype]).min
            x, t, _ = make(n, 12, n, dtype, 2)
            t[:, 0], t[:, 1] = 3, n - 1
            m = torch.ones(12, n, dtype=torch.bool, device="cuda")
            x[0, 5], m[0, 5] = nan, False             # what is masked has no effect
            x[1, :], m[1, :] = nan, False
            x[2, 7], m[2, 7] = inf, False
            x[3, :] = -inf                            # nothing left without a mask
            x[4, :] = low                             # the type's lowest value everywhere: uniform
            x[5, : n // 2] = low                      # and as a mask
            x[6, : n - 1] = -inf                      # one column left
            x[7, 3] = -inf                            # the given one has probability zero
            m[8, 3] = False                           # the given one is masked
            x[9, 2] = nan                             # broken rows
            x[10, 2] = inf
            m[11, : n - 2] = False
            compare(x, t, m, 1.0, 5, seed=n)
            compare(x, t, m, 1.0, 0, seed=n)
            compare(x[3:8], t[3:8], None, 0.25, 5, seed=n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores_keep_their_digits(dtype):
    """Scores far from zero: differences decide, and they are exact."""
    x, t, _ = make(3, 20, 5000, dtype, 1, spread=2.0)
    compare((x.float() + 4096).to(x.dtype), t, None, 8.0, 5)
    compare((x.float() - 30000).to(x.dtype), t, None, 0.01, 5)


def test_repeated_targets_and_status():
    x, t, _ = make(5, 30, 700, "f32", 6)
    t[:, 2] = t[:, 0]
    t[:, 5] = t[:, 0]
    t[::2, 4] = t[::2, 1]
    compare(x, t, None, 1.0, 8)
    assert ms.device_status() == 0
    bad = t.clone()
    bad[3, 1], bad[4, 0] = 700, -2
    good = ms.logprobs_fwd(x, t)
    got = ms.logprobs_fwd(x, bad)
    assert ms.device_status() == 6 and ms.device_status() == 0
    assert got[0][3, 1].isnan() and got[0][4, 0].isnan()
    got[0][3, 1], got[0][4, 0] = good[0][3, 1], good[0][4, 0]
    assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
    g = torch.ones(30, 6, device="cuda")
    dx = ms.logprobs_bwd(x, bad, None, got[4], got[1], grad_logprob=g)
    assert ms.device_status() == 6
    bad[3, 1] = bad[4, 0] = -1  # none
    assert torch.equal(dx, ms.logprobs_bwd(x, bad, None, got[4], got[1], grad_logprob=g))


def test_shapes_and_outputs():
    x, t, _ = make(6, 24, 90, "bf16", 1)
    flat = ms.logprobs_fwd(x, t, k=3)
    lead = ms.logprobs_fwd(x.view(2, 3, 4, 90), t.view(2, 3, 4), k=3)
    assert lead[0].shape == (2, 3, 4) and lead[2].shape == (2, 3, 4, 3) and lead[4].shape == (2, 3, 4, 2)
    for a, b in zip(flat, lead):
        assert torch.equal(a.flatten(), b.flatten())
    one = ms.logprobs_fwd(x[0], t[0])
    assert one[0].shape == (1,) and torch.equal(one[0], flat[0][0])
    none = ms.logprobs_fwd(x, None, k=3)
    assert none[0] is None and torch.equal(none[3], flat[3])
    empty = ms.logprobs_fwd(x[:0], t[:0], k=2)
    assert empty[0].shape == (0, 1) and empty[2].shape == (0, 2)
    dx = ms.logprobs_bwd(x, None, None, none[4], none[1], top_idx=none[2], grad_top=torch.ones(24, 3, device="cuda"))
    assert dx.shape == x.shape
    assert not ms.logprobs_bwd(x, t, None, flat[4], flat[1]).any()
    buf = torch.full((26, 90), 9.0, dtype=torch.bfloat16, device="cuda")
    ms.logprobs_bwd(x, t, None, flat[4], flat[1], grad_logprob=torch.ones(24, 1, device="cuda"), out=buf[1:25])
    assert (buf[0] == 9).all() and (buf[25] == 9).all() and not (buf[1:25] == 9).all()
    i32 = ms.logprobs_fwd(x, t.int())
    assert torch.equal(i32[0], flat[0])


def test_gradient_beside_the_logits_but_not_over_them():
    x, t, _ = make(8, 40, 500, "bf16", 2)
    _, h, _, _, st = ms.logprobs_fwd(x, t)
    g = torch.ones(40, 2, device="cuda")
    want = ms.logprobs_bwd(x, t, None, st, h, grad_logprob=g)
    lib, stream = ms._native.lib(), torch.cuda.current_stream().cuda_stream
    flat = torch.empty(40 * 1003, dtype=torch.bfloat16, device="cuda")
    both = flat.view(40, 1003)  # rows of logits, their gradients beside them
    for xs, ds in ((0, 500), (503, 0)):
        both.fill_(9.0)
        both[:, xs:xs + 500] = x
        p = flat.data_ptr()
        rc = lib.maxsim_logprobs_bwd(p + 2 * xs, 1, 40, 500, 1003, t.data_ptr(), 2, None, 0, 1.0, st.data_ptr(), h.data_ptr(), g.data_ptr(),
                                     None, None, None, 0, p + 2 * ds, 1003, stream)
        assert rc == 0
        assert torch.equal(both[:, ds:ds + 500], want) and torch.equal(both[:, xs:xs + 500], x)
    own = x.contiguous()
    with pytest.raises(ms._native.MaxSimError):
        ms.logprobs_bwd(own, t, None, st, h, grad_logprob=g, out=own)


def test_mask_bytes_of_any_value():
    for dtype in ("f32", "bf16"):
        for n, at in ((40, 0), (3000, 0), (3001, 1), (60000, 3)):
            x, t, _ = make(n, 6, n, dtype, 2)
            g = torch.Generator().manual_seed(n)
            values = torch.tensor([0, 1, 2, 127, 128, 129, 254, 255, 16], dtype=torch.uint8)
            m = torch.empty(6 * n + at, dtype=torch.uint8)
            m[at:] = values[torch.randint(0, 9, (6 * n,), generator=g)]
            m = m.cuda()[at:].view(6, n)
            one = ms.logprobs_fwd(x, t, m != 0, k=5)
            got = ms.logprobs_fwd(x, t, m, k=5)
            assert all(torch.equal(a, b) for a, b in zip(one, got))
            g1 = torch.ones(6, 2, device="cuda")
            assert torch.equal(ms.logprobs_bwd(x, t, m != 0, one[4], one[1], grad_logprob=g1),
                               ms.logprobs_bwd(x, t, m, one[4], one[1], grad_logprob=g1))


def test_autograd_against_differences():
    x, t, m = make(7, 6, 50, "f32", 2, "rows", spread=1.0)
    x = x.clone().requires_grad_()
    w = torch.randn(6, 2, device="cuda"), torch.randn(6, device="cuda"), torch.randn(6, 4, device="cuda")

    def loss(x):
        logprob, entropy, top_idx, top = ms.logprobs(x, t, m, scale=1.5, k=4)
        fine = lambda v: torch.where(v == -float("inf"), 0.0, v)  # noqa: E731
        return (fine(logprob) * w[0]).sum() + (entropy * w[1]).sum() + (fine(top) * w[2]).sum()
    (dx,) = torch.autograd.grad(loss(x), x)
    assert not dx[~m].any()
    with torch.no_grad():
        for r, j in ((0, 3), (1, 10), (2, int(t[2, 0].clamp(min=0))), (5, 49)):
            h = 1e-2
            up, down = x.clone(), x.clone()
            up[r, j] += h
            down[r, j] -= h
            # third derivatives are at most 6 * 1.5^3 * the weights' sum; a loss of size 100 is known to 2^-16
            near = (loss(up) - loss(down)) / (2 * h)
            assert abs(near - dx[r, j]) < h * h * 20 * 15 + 100 * 2.0 ** -17 / h
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad(loss(x), x, create_graph=True)
        torch.autograd.grad(g.sum(), x)


def test_autograd_outputs_that_are_left_out():
    x, t, _ = make(8, 6, 70, "bf16", 1)
    x = x.clone().requires_grad_()
    logprob, entropy, top_idx, top = ms.logprobs(x, None)
    assert logprob is None and top_idx is None and top is None and entropy.requires_grad
    (dx,) = torch.autograd.grad(entropy.sum(), x)
    ref = ms.logprobs_fwd(x.detach(), None)
    assert torch.equal(dx, ms.logprobs_bwd(x.detach(), None, None, ref[4], ref[1], grad_entropy=torch.ones(6, device="cuda")))
    logprob, entropy, top_idx, top = ms.logprobs(x, t[:, 0], k=2)
    assert not top_idx.requires_grad
    (dx,) = torch.autograd.grad(top.sum(), x)
    ref = ms.logprobs_fwd(x.detach(), t[:, 0], k=2)
    assert torch.equal(dx, ms.logprobs_bwd(x.detach(), t[:, 0], None, ref[4], ref[1], top_idx=ref[2], grad_top=torch.ones(6, 2, device="cuda")))
    assert ms.logprobs(x.detach(), t[:, 0])[0].requires_grad is False


def test_two_streams_at_once():
    """Calls of all operators on two streams, each with its own data, interleaved."""
    data = [make(s, 300, 9000, "bf16", 1)[:2] for s in (1, 2)]
    want = [ms.logprobs_fwd(x, t, k=7) for x, t in data]
    rows = [torch.randn(700, 512, device="cuda") for _ in data]
    w = ms.quantize_rows_fp4(torch.randn(300, 512, device="cuda"))
    prod = [ms.linear_fp4(*ms.quantize_rows_fp4(r), *w) for r in rows]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((ms.logprobs_fwd(*data[i], k=7), ms.linear_fp4(*ms.quantize_rows_fp4(rows[i]), *w)))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out, y in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])) and torch.equal(y, prod[i])


def test_contrastive_step_through_the_scores():
    """MaxSim scores, the given document's log probability, the gradient back to the token embeddings."""
    g = torch.Generator().manual_seed(11)
    Q, D = (torch.nn.functional.normalize(torch.randn(s, generator=g), dim=-1).bfloat16().cuda() for s in ((16, 32, 128), (16, 64, 128)))
    Q.requires_grad_()
    D.requires_grad_()
    scores = ms.maxsim(Q, D)
    target = torch.arange(16, device="cuda")
    logprob, entropy, top_idx, _ = ms.logprobs(scores, target, scale=0.5, k=3)
    dQ, dD = torch.autograd.grad(-logprob.mean(), (Q, D))
    assert torch.equal(top_idx, ms.maxsim_topk(scores.detach(), 3)[1])
    p = torch.softmax(scores.detach().double() * 0.5, dim=1)
    ds = (0.5 / 16 * (p - torch.eye(16, device="cuda").double())).float()
    dQ2, dD2, _, _ = ms.maxsim_bwd(Q.detach(), D.detach(), ms.maxsim_fwd(Q.detach(), D.detach(), want_argmax=True)[1], ds)
    # gradients of at most a few hundredths, rounded to bf16; the scores' gradient is known to 1e-6 of its size
    assert torch.allclose(dQ.float(), dQ2, rtol=2.0 ** -8 + 1e-4, atol=1e-5 * dQ2.abs().max().item())
    assert torch.allclose(dD.float(), dD2, rtol=2.0 ** -8 + 1e-4, atol=1e-5 * dD2.abs().max().item())


def test_graph_replay():
    xs = [make(s, 33, 5000, "f32", 1)[:2] for s in (1, 2)]
    want = [ms.logprobs_fwd(x, t, k=9) for x, t in xs]
    x, t = xs[0][0].clone(), xs[0][1].clone()
    ge = torch.ones(33, 1, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ms.logprobs_fwd(x, t, k=9)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = ms.logprobs_fwd(x, t, k=9)
            dx = ms.logprobs_bwd(x, t, None, out[4], out[1], grad_logprob=ge)
        for i in (1, 0, 1):
            x.copy_(xs[i][0])
            t.copy_(xs[i][1])
            graph.replay()
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
            assert torch.equal(dx, ms.logprobs_bwd(x, t, None, want[i][4], want[i][1], grad_logprob=ge))
