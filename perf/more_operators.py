"""More operators as they are measured: 4-bit floating-point rows (quantisation, reading back, the linear product) and the log
probabilities of given columns with their gradient.

`run` computes a case's operator in plain torch operations, or with `own` set through the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # hidden states of one query (32 tokens) before the 4-bit head: the smallest call
        {"name": "quantize_query", "op": "quantize", "rows": 32, "cols": 1024, "block": 16, "dtype": "bf16", "pad": 0},
        # token embeddings of 10,000 pages, 128 wide, stored in 4 bits and read back for scoring
        {"name": "quantize_index", "op": "quantize", "rows": 5000000, "cols": 128, "block": 32, "dtype": "f16", "pad": 0},
        # one token through a wide layer: the weights' bytes decide
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "block": 16, "dtype": "bf16", "bias": False},
        # one query (32 tokens) through the 128-wide head: latency decides
        {"name": "linear_query_head", "op": "linear", "M": 32, "N": 128, "K": 1024, "block": 32, "dtype": "f16", "bias": True},
        # odd sizes all round, f32 result
        {"name": "linear_odd", "op": "linear", "M": 999, "N": 1537, "K": 1111, "block": 16, "dtype": "f32", "bias": True},
        # the 128-wide head over the tokens of 1,024 pages: the activations' and the embeddings' bytes decide
        {"name": "linear_index_head", "op": "linear", "M": 1048576, "N": 128, "K": 1024, "block": 16, "dtype": "f16",
         "bias": False},
        # a batch of pages through a wide layer: the arithmetic decides
        {"name": "linear_pages", "op": "linear", "M": 32768, "N": 4096, "K": 4096, "block": 16, "dtype": "bf16", "bias": True},
        # an in-batch contrastive step: 64 queries against their 64 documents, probability of each one's own, gradient
        {"name": "logprobs_batch", "op": "logprobs", "way": "step", "rows": 64, "n": 64, "targets": 1, "k": 0, "dtype": "f32",
         "mask": "none", "scale": 10.0, "pad": 0},
        # a query batch against a corpus of 100,000 documents, the ones in use marked: given documents, 20 best
        {"name": "logprobs_corpus", "op": "logprobs", "way": "fwd", "rows": 32, "n": 100000, "targets": 4, "k": 20,
         "dtype": "f32", "mask": "columns", "scale": 1.0, "pad": 0},
        # logits of 4,096 tokens over a large vocabulary: the given token, entropy, 5 alternatives
        {"name": "logprobs_tokens", "op": "logprobs", "way": "fwd", "rows": 4096, "n": 131072, "targets": 1, "k": 5,
         "dtype": "bf16", "mask": "none", "scale": 1.0, "pad": 0},
        # a training step over an odd vocabulary, each row with its own mask, rows of a wider buffer
        {"name": "logprobs_odd", "op": "logprobs", "way": "step", "rows": 999, "n": 32003, "targets": 1, "k": 8, "dtype": "f16",
         "mask": "rows", "scale": 0.7, "pad": 5},
        # the same for a batch of tokens: the bytes of logits and gradients decide
        {"name": "logprobs_train", "op": "logprobs", "way": "step", "rows": 8192, "n": 32768, "targets": 1, "k": 0,
         "dtype": "bf16", "mask": "none", "scale": 1.0, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "logprobs", "logprobs"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    pad = rng.choice([0, 0, 0, 8, 16, 1, 5])
    block = rng.choice([16, 32])
    if op == "quantize":
        while True:
            rows, cols = _log(rng, 1, 5000000), _log(rng, 1, 16384)
            if rows * (cols + pad) <= 5000000 * 128:
                return {"op": op, "rows": rows, "cols": cols, "block": block, "dtype": dtype, "pad": pad}
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 1 << 20), _log(rng, 1, 8192), _log(rng, 1, 16384)
            if rng.random() < 0.5:  # the sizes of layers as they are mostly built
                n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
            if m * n * k <= 32768 * 4096 * 4096 and m * (k + 4 * n) <= 1 << 32:
                return {"op": op, "M": m, "N": n, "K": k, "block": block, "dtype": dtype, "bias": rng.random() < 0.5}
    while True:
        rows, n = _log(rng, 1, 16384), _log(rng, 2, 1 << 20)
        if rows * (n + pad) <= 1 << 28:
            k = min(n, rng.choice([0, 0, 1, 5, 20, 64]))
            return {"op": op, "way": rng.choice(["fwd", "step"]), "rows": rows, "n": n, "targets": rng.choice([1, 1, 1, 3, 8]),
                    "k": k, "dtype": dtype, "mask": rng.choice(["none", "none", "columns", "rows"]),
                    "scale": rng.choice([0.1, 0.7, 1.0, 1.0, 10.0]), "pad": pad}


def _activations(g, rows, cols, pad, dtype):
    """Activations: a size of its own for every row, every 97th channel ten times the others, rows of a wider buffer."""
    t = torch.randn((rows, cols + pad), generator=g, device="cuda", dtype=torch.float32)
    t *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda", dtype=torch.float32))
    t[:, ::97] *= 10.0
    return t.to(dtype)[:, :cols]


def _round_scale(v):
    """v >= 0 to the nearest of E4M3's values (ties to even), 2**-9 at least."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).float() - 3)
    return (torch.round(v / step) * step).clamp(min=2.0 ** -9)


def _round_code(v):
    """v to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (ties to even), 6 at most."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _plain_quantize(x, block):
    """(codes' values [rows, blocks, block], block scales [rows, blocks], row scales [rows] or None)."""
    rows, cols = x.shape
    blocks = (cols + block - 1) // block
    y = torch.nn.functional.pad(x.float(), (0, blocks * block - cols)).reshape(rows, blocks, block)
    most = y.abs().amax(dim=2)
    if block == 32:
        _, e = torch.frexp(most)
        b = torch.exp2(torch.where(most > 0, e - 3, -127).clamp(min=-127).double())
        return _round_code((y.double() / b[:, :, None]).float()), b.float(), None
    m, e = torch.frexp(most.amax(dim=1))  # 2688 = 0.65625 * 2**12
    s = torch.exp2(torch.where(m > 0, e - 12 + (m > 0.65625).int(), -126).clamp(min=-126).float())
    b = _round_scale((most / s[:, None]) / 6.0)
    return _round_code((y / s[:, None, None]) / b[:, :, None]), b, s


def _pack(codes, b, s, block):
    """The bytes of quantised rows: q [rows, 16-byte pieces], the scales of 4 blocks of 128 rows in 512 bytes, row scales."""
    rows, blocks, _ = codes.shape
    a = codes.abs()
    nibble = (a * 2).where(a < 2, a + 2).where(a < 4, a / 2 + 4).to(torch.uint8)
    nibble += torch.signbit(codes).to(torch.uint8) * 8
    nibble = nibble.reshape(rows, blocks * block)
    nibble = torch.nn.functional.pad(nibble, (0, -(blocks * block) % 32))
    q = (nibble[:, 0::2] + nibble[:, 1::2] * 16).contiguous()
    byte = (torch.log2(b) + 127).round().to(torch.uint8) if block == 32 else b.to(torch.float8_e4m3fn).view(torch.uint8)
    byte = torch.nn.functional.pad(byte, (0, -blocks % 4, 0, -rows % 128))
    byte = byte.reshape(-1, 4, 32, byte.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return q, byte, s


def _unpack(q, byte, s, block):
    """The values of quantised rows [rows, 2 * bytes] in 32 bits, without the row scales."""
    rows = q.shape[0]
    nibble = torch.stack((q & 15, q >> 4), dim=2).reshape(rows, -1)
    c = (nibble & 7).float()
    v = torch.where(c < 4, c / 2, torch.where(c < 6, c - 2, 2 * c - 8))
    v = torch.where(nibble > 7, -v, v)
    b = byte.permute(0, 3, 2, 1, 4).reshape(byte.shape[0] * 128, -1)[:rows]
    b = torch.exp2(b.float() - 127) if block == 32 else b.view(torch.float8_e4m3fn).float()
    return v * b.repeat_interleave(block, dim=1)[:, :v.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "quantize":
        s = {"x": _activations(g, case["rows"], case["cols"], case["pad"], DTYPES[case["dtype"]])}
    elif case["op"] == "linear":
        M, N, K, block = case["M"], case["N"], case["K"], case["block"]
        w = torch.randn((N, K), generator=g, device="cuda") * torch.exp(0.3 * torch.randn((N, 1), generator=g, device="cuda"))
        s = {"x": _pack(*_plain_quantize(_activations(g, M, K, 0, torch.bfloat16), block), block),
             "w": _pack(*_plain_quantize((w * K ** -0.5).to(torch.bfloat16), block), block),
             "bias": torch.randn(N, generator=g, device="cuda") if case["bias"] else None}
    else:
        rows, n, dtype = case["rows"], case["n"], DTYPES[case["dtype"]]
        x = torch.randn((rows, n + case["pad"]), generator=g, device="cuda") * (2.0 / case["scale"])
        x += 8.0 / case["scale"] * torch.rand((rows, 1), generator=g, device="cuda")
        targets = torch.randint(0, n, (rows, case["targets"]), generator=g, device="cuda")
        x.scatter_add_(1, targets, torch.full(targets.shape, 5.0 / case["scale"], device="cuda"))  # what is given is likely
        targets[3::17, 0] = -1  # a token that is not counted
        mask = None
        if case["mask"] != "none":
            shape = (n,) if case["mask"] == "columns" else (rows, n)
            mask = torch.rand(shape, generator=g, device="cuda") < 0.9
            if case["mask"] == "rows":
                mask[5::23] = False  # padding: a row whose mask leaves nothing
        s = {"x": x.to(dtype)[:, :n], "targets": targets, "mask": mask,
             "g": torch.randn((rows, case["targets"]), generator=g, device="cuda") / rows,
             "g_entropy": 0.01 * torch.randn(rows, generator=g, device="cuda") / rows}
    s["case"] = case
    return s


def _plain_logprobs(s, scale, k, step):
    x, targets = s["x"].float(), s["targets"]
    rows, n = x.shape
    if s["mask"] is not None:
        x = torch.where(s["mask"], x, -math.inf)
    most = x.amax(dim=1, keepdim=True)
    empty = most == -math.inf
    d = (x - torch.where(empty, 0.0, most)) * scale
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    logp = d - torch.log(total)
    logp = torch.where(empty, -math.inf, logp)
    p = torch.where(empty, 0.0, e / total)
    terms = p * torch.where(p > 0, logp, 0.0)
    entropy = -terms.sum(dim=1)
    given = targets >= 0
    logprob = torch.where(given, logp.gather(1, targets.clamp(min=0)), 0.0)
    out = {"logprob": logprob, "entropy": entropy}
    if k:
        best, at = torch.sort(x, dim=1, descending=True, stable=True)
        listed_ = best[:, :k] > -math.inf
        out["top_idx"] = torch.where(listed_, at[:, :k], -1).int()
        out["top_logprob"] = torch.where(listed_, logp.gather(1, at[:, :k]), -math.inf)
    if step:
        c = torch.where(given & (logprob > -math.inf), s["g"], 0.0)
        gh = s["g_entropy"][:, None]
        dx = -p * c.sum(dim=1, keepdim=True) - gh * (terms + p * entropy[:, None])
        dx.scatter_add_(1, targets.clamp(min=0), c)
        out["dx"] = (dx * scale).to(s["x"].dtype)
    return out


def run(state):
    case = state["case"]
    if own:
        import maxsim_scoring_gb300 as ms
        if case["op"] == "quantize":
            q, block_scale, scale = ms.quantize_rows_fp4(state["x"], block=case["block"])
            return ms.dequantize_rows_fp4(q, block_scale, scale, block=case["block"], cols=case["cols"],
                                          out_dtype=DTYPES[case["dtype"]])
        if case["op"] == "linear":
            return ms.linear_fp4(*state["x"], *state["w"], state["bias"], block=case["block"], out_dtype=DTYPES[case["dtype"]])
        logprob, entropy, top_idx, top_logprob, stats = ms.logprobs_fwd(
            state["x"], state["targets"], state["mask"], scale=case["scale"], k=case["k"])
        out = {"logprob": logprob, "entropy": entropy}
        if case["k"]:
            out["top_idx"], out["top_logprob"] = top_idx, top_logprob
        if case["way"] == "step":
            out["dx"] = ms.logprobs_bwd(state["x"], state["targets"], state["mask"], stats, entropy, grad_logprob=state["g"],
                                        grad_entropy=state["g_entropy"], scale=case["scale"])
        return out
    if case["op"] == "quantize":
        codes, b, s = _plain_quantize(state["x"], case["block"])
        v = (codes * b[:, :, None]).reshape(codes.shape[0], -1)[:, :case["cols"]]
        return (v if s is None else v * s[:, None]).to(state["x"].dtype)
    if case["op"] == "linear":
        y = _unpack(*state["x"], case["block"]) @ _unpack(*state["w"], case["block"]).t()
        if case["block"] == 16:
            y = y * state["x"][2][:, None] * state["w"][2][None, :]
        if state["bias"] is not None:
            y = y + state["bias"]
        return y.to(DTYPES[case["dtype"]])
    return _plain_logprobs(state, case["scale"], case["k"], case["way"] == "step")


def work(case):
    if case["op"] == "quantize":  # to 4 bits and back
        n, blocks = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // case["block"])
        return {"bytes": 2 * n * BYTES[case["dtype"]] + 2 * (n // 2 + blocks), "flops": 4 * n}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        rows = (M + N) * ((K + 1) // 2 + -(-K // case["block"]) + (4 if case["block"] == 16 else 0))
        return {"bytes": rows + (4 * N if case["bias"] else 0) + M * N * BYTES[case["dtype"]], "flops": 2 * M * N * K}
    n = case["rows"] * case["n"]
    mask = {"none": 0, "columns": case["n"], "rows": n}[case["mask"]]
    step = case["way"] == "step"
    return {"bytes": n * BYTES[case["dtype"]] * (2 if step else 1) + mask + case["rows"] * (12 * case["targets"] + 4 + 8 * case["k"]),
            "flops": (12 if step else 6) * n}


def exact(case, seed):
    """The definitions in float64."""
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x, block = s["x"].double(), case["block"]
        if x.numel() > 1 << 30:
            return None
        lead = x.new_zeros(x.shape[0], -x.shape[1] % block)
        groups = torch.cat((x, lead), dim=1).unflatten(1, (-1, block))
        size = torch.linalg.vector_norm(groups, ord=math.inf, dim=2)
        if block == 32:
            unit = _largest_power(size / 4, -127)
        else:
            row = torch.linalg.vector_norm(size, ord=math.inf, dim=1, keepdim=True)
            power = _largest_power(row / 2688, -126)
            power = torch.where(power * 2688 < row, power * 2, power)
            table = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
            unit = _nearest(size / (6 * power), table).clamp(min=2.0 ** -9) * power
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
        v = _nearest(groups.abs() / unit.unsqueeze(2), table) * groups.sign() * unit.unsqueeze(2)
        return v.flatten(1)[:, :x.shape[1]]
    if case["op"] == "linear":
        if case["M"] * case["N"] * case["K"] > 1 << 39:
            return None
        code = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
        sides = []
        for q, byte, row in (s["x"], s["w"]):
            pairs = torch.stack((q % 16, q // 16), dim=-1).flatten(1)
            r = torch.arange(q.shape[0], device="cuda").unsqueeze(1)
            j = torch.arange(-(-pairs.shape[1] // case["block"]), device="cuda")
            byte = byte[r // 128, j // 4, r % 32, r // 32 % 4, j % 4]
            unit = _powers(byte.device)[byte.long() + 23] if row is None else byte.view(
                torch.float8_e4m3fn).double() * row.double().unsqueeze(1)
            at = torch.arange(pairs.shape[1], device="cuda") // case["block"]
            sides.append(code[pairs.long()].mul_(unit[:, at]))
        y = torch.einsum("mk,nk->mn", *sides)
        return y if s["bias"] is None else y.add_(s["bias"].double())
    y = s["x"].double().mul(case["scale"])
    if s["mask"] is not None:
        y = y.masked_fill(~s["mask"], -math.inf)
    total = torch.logsumexp(y, dim=1, keepdim=True)
    logp = (y - total).nan_to_num(nan=-math.inf, neginf=-math.inf)
    p = logp.exp()
    surprise = -logp.masked_fill(p == 0, 0.0)
    entropy = (p * surprise).sum(dim=1)
    t = s["targets"]
    out = {"logprob": logp.gather(1, t.clamp(min=0)).masked_fill(t < 0, 0.0), "entropy": entropy}
    if case["k"]:
        out["top_idx"], out["top_logprob"] = None, logp.topk(case["k"], dim=1).values
    if case["way"] == "step":
        g = s["g"].double().masked_fill((t < 0) | (out["logprob"] == -math.inf), 0.0)
        hot = torch.zeros_like(p).scatter_add_(1, t.clamp(min=0), g)
        out["dx"] = case["scale"] * (hot - p * g.sum(1, True) + s["g_entropy"].double()[:, None] * p * (surprise - entropy[:, None]))
    return out


def _powers(device):
    return torch.tensor([2.0 ** i for i in range(-150, 129)], dtype=torch.float64, device=device)


def _largest_power(v, least):
    """The largest power of two that is not above v (in float64), 2**least at least."""
    table = _powers(v.device)[least + 150:]
    return table[(torch.searchsorted(table, v.contiguous(), right=True) - 1).clamp(min=0)]


def _nearest(v, table):
    """v >= 0 to the nearest value of an ascending table (in float64), to the even place where two are as near."""
    hi = torch.searchsorted(table, v.contiguous()).clamp(1, len(table) - 1)
    up, down = table[hi] - v, v - table[hi - 1]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), table[hi], table[hi - 1])
