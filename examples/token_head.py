"""A late-interaction head from hidden states to ranked documents.

Training: dropout on the hidden states, a linear projection to the token
embedding's width, L2 normalisation, MaxSim scores of every (query, document)
pair, an in-batch contrastive loss, its gradient.
Serving: the same head in 8-bit integers. Weights are quantised per channel
once, hidden states per token; the INT8 product gives the embeddings, whose
quantised unit rows are what the INT8 scoring and the top-k take. Or in 4 bits:
weights and hidden states in 4-bit floating point, the index stored in 4 bits a
value and read back for the scoring, the answer as probabilities.

    python examples/token_head.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import maxsim_scoring_gb300 as ms  # noqa: E402


class TokenHead:
    """weight [dim, hidden] f32, trained in bf16 products and served in INT8."""

    def __init__(self, hidden, dim, p=0.1, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.weight = (torch.randn(dim, hidden, generator=g, device=device) * hidden ** -0.5).requires_grad_()
        self.p, self.seed, self.step = p, seed, 0

    def embed(self, hidden, stream):
        """Unit token embeddings [..., dim] in bf16 for training; `stream` tells
        the masks of one step's calls apart."""
        x = ms.dropout(hidden, self.p, self.seed, 2 * self.step + stream)
        return torch.nn.functional.normalize((x @ self.weight.to(x.dtype).t()).float(), dim=-1).to(x.dtype)

    def train_step(self, q_hidden, d_hidden, q_mask=None, d_mask=None, lr=0.5, temperature=0.1):
        """One step on queries [B, Lq, hidden] and their documents [B, Ld, hidden]; returns the loss."""
        q, d = self.embed(q_hidden, 0), self.embed(d_hidden, 1)
        scores = ms.maxsim(q, d, q_mask, d_mask) / (q.shape[1] * temperature)
        loss = torch.nn.functional.cross_entropy(scores, torch.arange(len(scores), device=scores.device))
        (grad,) = torch.autograd.grad(loss, self.weight)
        with torch.no_grad():
            self.weight -= lr * grad
        self.step += 1
        return loss.detach()

    def quantized(self):
        """The head for serving: INT8 weights and their channels' scales."""
        return ms.quantize_rows(self.weight.detach())

    @staticmethod
    def index(hidden, head):
        """INT8 token embeddings [..., dim] and their scales for hidden states [..., hidden]."""
        x, x_scale = ms.quantize_rows(hidden)
        embeddings = ms.linear_int8(x, x_scale, *head, out_dtype=torch.float16)
        return ms.quantize_rows(embeddings, normalize=True)

    def quantized4(self):
        """The head in 4-bit floating point: codes, block scales, row scales."""
        return ms.quantize_rows_fp4(self.weight.detach())

    @staticmethod
    def embed4(hidden, head):
        """Unit token embeddings [..., dim] in bf16 through the 4-bit head."""
        y = ms.linear_fp4(*ms.quantize_rows_fp4(hidden), *head, out_dtype=torch.bfloat16)
        return torch.nn.functional.normalize(y.float(), dim=-1).to(torch.bfloat16)

    @staticmethod
    def index4(hidden, head):
        """Unit token embeddings stored in 4 bits, with a scale for every 32 values."""
        return ms.quantize_rows_fp4(TokenHead.embed4(hidden, head), block=32)


def answer(q_hidden, index, head, given, k, temperature=0.1):
    """Among the documents of a 4-bit index: the log probability of each query's given one, the entropy, and the k
    likeliest with theirs."""
    q, d = TokenHead.embed4(q_hidden, head), ms.dequantize_rows_fp4(*index, block=32, out_dtype=torch.bfloat16)
    scores, _ = ms.maxsim_fwd(q, d)
    return ms.logprobs_fwd(scores, given, scale=1 / (q.shape[1] * temperature), k=k)[:4]


def search(q_hidden, index, head, k):
    """The k best documents of each query by INT8 MaxSim: (scores, indices)."""
    q8, q_scale = TokenHead.index(q_hidden, head)
    scores, _, _ = ms.maxsim_fwd_int8(q8, q_scale, *index)
    return ms.maxsim_topk(scores, k)


def synthetic_pairs(n, lq, ld, hidden, seed, noise=2.0, device="cuda"):
    """Hidden states of n queries and n documents: each pair shares a topic, buried in noise of its own tokens."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    topic = torch.randn(n, 1, 16, generator=g, device=device) @ torch.randn(16, hidden, generator=g, device=device) / 4
    make = lambda length: (topic + noise * torch.randn(n, length, hidden, generator=g, device=device)).to(torch.bfloat16)  # noqa: E731
    return make(lq), make(ld)


def main(n=64, lq=32, ld=180, hidden=1024, dim=128, steps=20):
    head = TokenHead(hidden, dim)
    q, d = synthetic_pairs(n, lq, ld, hidden, seed=1)
    losses = [head.train_step(q, d).item() for _ in range(steps)]
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    served = head.quantized()
    _, best = search(q, TokenHead.index(d, served), served, k=5)
    hit = (best[:, 0].cpu() == torch.arange(n)).float().mean().item()
    print(f"own document first for {hit:.0%} of the queries")
    head4 = head.quantized4()
    logprob, entropy, best, _ = answer(q, TokenHead.index4(d, head4), head4, torch.arange(n, device=q.device), k=5)
    print(f"in 4 bits: own document first for {(best[:, 0].cpu() == torch.arange(n)).float().mean().item():.0%}, "
          f"its log probability {logprob.mean().item():.3f}, entropy {entropy.mean().item():.3f}")
    return losses, hit


if __name__ == "__main__":
    main()
