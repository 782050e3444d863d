"""The token head's operators as they are measured: row quantisation to INT8, the INT8 linear product and dropout.

`run` computes a case's operator in plain torch operations, or with `own` set through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

FLT_MIN = 1.1754943508222875e-38  # smallest normal float32
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # one query's 32 token embeddings, normalised and quantised for the INT8 scoring: the smallest call
        {"name": "quantize_query", "op": "quantize", "rows": 32, "cols": 128, "dtype": "f16", "normalize": True, "pad": 0},
        # hidden states of a batch of pages (8 x 1024 tokens) on their way into the INT8 product
        {"name": "quantize_hidden", "op": "quantize", "rows": 8192, "cols": 1024, "dtype": "bf16", "normalize": False,
         "pad": 0},
        # token embeddings of 10,000 pages in f32, 128 wide, quantised into an index
        {"name": "quantize_index", "op": "quantize", "rows": 5000000, "cols": 128, "dtype": "f32", "normalize": True,
         "pad": 0},
        # one token through a wide layer: the weights' bytes decide
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16", "bias": False, "pad": 0},
        # one query (32 tokens) through the 128-wide head: latency decides
        {"name": "linear_query_head", "op": "linear", "M": 32, "N": 128, "K": 1024, "dtype": "f16", "bias": True, "pad": 0},
        # odd sizes all round, rows of a wider buffer, f32 result
        {"name": "linear_odd", "op": "linear", "M": 999, "N": 1537, "K": 1111, "dtype": "f32", "bias": True, "pad": 5},
        # a batch of 64 queries through an encoder layer
        {"name": "linear_batch", "op": "linear", "M": 2048, "N": 4096, "K": 1024, "dtype": "bf16", "bias": True, "pad": 0},
        # the 128-wide head over the tokens of 1,024 pages: the activations' bytes decide
        {"name": "linear_index_head", "op": "linear", "M": 1048576, "N": 128, "K": 1024, "dtype": "f16", "bias": False,
         "pad": 0},
        # a batch of pages through a wide layer: the arithmetic decides
        {"name": "linear_pages", "op": "linear", "M": 32768, "N": 4096, "K": 4096, "dtype": "bf16", "bias": True, "pad": 0},
        # hidden states of one training query: the smallest call
        {"name": "dropout_query", "op": "dropout", "way": "fwd", "rows": 32, "cols": 1024, "dtype": "bf16", "p": 0.1,
         "residual": False, "pad": 0},
        # a training batch with the residual added, rows of a wider buffer, odd width
        {"name": "dropout_residual", "op": "dropout", "way": "fwd", "rows": 16384, "cols": 1023, "dtype": "bf16", "p": 0.1,
         "residual": True, "pad": 1},
        # the gradient of a large batch
        {"name": "dropout_grad", "op": "dropout", "way": "bwd", "rows": 262144, "cols": 1024, "dtype": "f16", "p": 0.1,
         "residual": False, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "dropout"])
    pad = rng.choice([0, 0, 0, 8, 16, 1, 5])
    dtype = rng.choice(["f16", "bf16", "f32"])
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 1 << 20), _log(rng, 1, 8192), _log(rng, 1, 8192)
            if rng.random() < 0.5:  # the sizes of layers as they are mostly built
                n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
            if m * n * k <= 32768 * 4096 * 4096 and m * (k + 4 * n) <= 1 << 32:
                return {"op": op, "M": m, "N": n, "K": k, "dtype": dtype, "bias": rng.random() < 0.5, "pad": pad}
    if op == "quantize":
        while True:
            rows, cols = _log(rng, 1, 5000000), _log(rng, 1, 16384)
            if rows * cols <= 5000000 * 128:
                return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "normalize": rng.random() < 0.5, "pad": pad}
    while True:
        rows, cols, residual = _log(rng, 1, 262144), _log(rng, 1, 16384), rng.random() < 0.5
        way = rng.choice(["fwd", "bwd"])
        if rows * cols * BYTES[dtype] * (3 if residual and way == "fwd" else 2) <= 262144 * 1024 * 4:
            return {"op": op, "way": way, "rows": rows, "cols": cols, "dtype": dtype, "p": rng.choice([0.05, 0.1, 0.25, 0.5]),
                    "residual": residual and way == "fwd", "pad": pad}


def _rows(g, rows, cols, pad, dtype):
    """Activations: a size of its own for every row, every 97th channel ten times the others, rows of a wider buffer."""
    t = torch.randn((rows, cols + pad), generator=g, device="cuda", dtype=torch.float32)
    t *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda", dtype=torch.float32))
    t[:, ::97] *= 10.0
    return t.to(DTYPES[dtype])[:, :cols]


def _codes(g, rows, cols, pad):
    t = torch.randint(-127, 128, (rows, cols + pad), generator=g, device="cuda", dtype=torch.int8)
    return t[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "quantize":
        s = {"x": _rows(g, case["rows"], case["cols"], case["pad"], case["dtype"])}
    elif case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s = {"x": _codes(g, M, K, case["pad"]), "w": _codes(g, N, K, 0),
             "x_scale": 0.01 + 0.05 * torch.rand(M, generator=g, device="cuda"),
             "w_scale": 0.001 + 0.001 * torch.rand(N, generator=g, device="cuda"),
             "bias": torch.randn(N, generator=g, device="cuda") if case["bias"] else None}
    else:
        s = {"x": _rows(g, case["rows"], case["cols"], case["pad"], case["dtype"]),
             "residual": _rows(g, case["rows"], case["cols"], 0, case["dtype"]) if case["residual"] else None,
             "seed": 0x9E3779B97F4A7C15 ^ (seed * 1000003), "offset": 3 * seed + 1}
    s["case"] = case
    return s


def _philox(block, seed, offset):
    """Philox4x32 with ten rounds: the four 32-bit words (in int64) of every counter (block, offset)."""
    low = 0xFFFFFFFF
    c0, c1 = block & low, block >> 32
    c2, c3 = torch.full_like(block, offset & low), torch.full_like(block, offset >> 32)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products, kept modulo 2^64
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _plain_keep(rows, cols, p, seed, offset, device):
    block = torch.arange((rows * cols + 7) // 8, device=device, dtype=torch.int64)
    words = torch.stack(_philox(block, seed, offset), dim=1)
    halves = torch.stack((words & 0xFFFF, words >> 16), dim=2)
    return (halves >= round(p * 65536)).reshape(-1)[:rows * cols].reshape(rows, cols)


def _plain_quantize(x, normalize):
    x = x.float()
    s = (x.abs().amax(dim=1, keepdim=True) / 127.0).clamp(min=FLT_MIN)
    y = x / s
    q = y.round().clamp(-127, 127).to(torch.int8)
    if not normalize:
        return q, s[:, 0]
    norm = y.square().sum(dim=1).sqrt()
    return q, torch.where(norm > 0, 1.0 / norm, torch.full_like(norm, FLT_MIN))


def _plain_linear(s, dtype):
    y = s["x"].float() @ s["w"].float().t()
    y = y * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(dtype)


def _plain_dropout(s, p):
    x = s["x"]
    rows, cols = x.shape
    drop = round(p * 65536)
    keep = _plain_keep(rows, cols, p, s["seed"], s["offset"], x.device)
    y = torch.where(keep, x.float() * (65536.0 / (65536 - drop) if drop < 65536 else 0.0), torch.zeros((), device=x.device))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype)


def run(state):
    case = state["case"]
    if own:
        import maxsim_scoring_gb300 as ms
        if case["op"] == "quantize":
            return ms.quantize_rows(state["x"], normalize=case["normalize"])
        if case["op"] == "linear":
            return ms.linear_int8(state["x"], state["x_scale"], state["w"], state["w_scale"], state["bias"],
                                  out_dtype=DTYPES[case["dtype"]])
        if case["way"] == "bwd":
            return ms.dropout_bwd(state["x"], case["p"], state["seed"], state["offset"])
        return ms.dropout_fwd(state["x"], case["p"], state["seed"], state["offset"], residual=state["residual"])
    if case["op"] == "quantize":
        return _plain_quantize(state["x"], case["normalize"])
    if case["op"] == "linear":
        return _plain_linear(state, DTYPES[case["dtype"]])
    return _plain_dropout(state, case["p"])


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (BYTES[case["dtype"]] + 1) + 4 * case["rows"], "flops": (4 if case["normalize"] else 2) * n}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * M + 4 * N * (2 if case["bias"] else 1) + M * N * BYTES[case["dtype"]],
                "flops": 2 * M * N * K}
    n = case["rows"] * case["cols"]
    return {"bytes": n * BYTES[case["dtype"]] * (3 if case["residual"] else 2), "flops": 2 * n}


def exact(case, seed):
    """The definition in float64 (the codes of a quantised row have no other value than the definition's in float32)."""
    if case["op"] == "quantize":
        x = prepare(case, seed)["x"].double()
        largest = torch.linalg.vector_norm(x, ord=math.inf, dim=1)
        if case["normalize"]:
            # the unit row's codes times this scale: the row over its norm, in units of its step
            length = torch.linalg.vector_norm(x, dim=1)
            return None, torch.where(length > 0, torch.clamp(largest / 127, min=FLT_MIN) / length, FLT_MIN)
        return None, torch.clamp(largest / 127, min=FLT_MIN)
    if case["op"] == "linear":
        s = prepare(case, seed)
        if case["M"] * case["N"] * case["K"] > 1 << 38:
            return None
        left = s["x"].double() * s["x_scale"].double().unsqueeze(1)
        right = s["w"].double() * s["w_scale"].double().unsqueeze(1)
        y = torch.einsum("mk,nk->mn", left, right)
        return y if s["bias"] is None else y.add_(s["bias"].double())
    if case["rows"] * case["cols"] > 1 << 25:
        return None
    s = prepare(case, seed)
    n = case["rows"] * case["cols"]
    ctr = [np.arange((n + 7) // 8, dtype=np.uint64), None, None, None]
    ctr[1], ctr[0] = ctr[0] >> np.uint64(32), ctr[0] & np.uint64(0xFFFFFFFF)
    ctr[2] = np.full_like(ctr[0], s["offset"] % 2**32)
    ctr[3] = np.full_like(ctr[0], s["offset"] // 2**32)
    for r in range(10):
        key = [(s["seed"] + r * 0x9E3779B9) % 2**32, (s["seed"] // 2**32 + r * 0xBB67AE85) % 2**32]
        p0, p1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(p1 >> np.uint64(32)) ^ ctr[1] ^ np.uint64(key[0]), p1 & np.uint64(0xFFFFFFFF),
               (p0 >> np.uint64(32)) ^ ctr[3] ^ np.uint64(key[1]), p0 & np.uint64(0xFFFFFFFF)]
    bits = np.stack(ctr, axis=1).astype("<u4").view("<u2").reshape(-1)[:n].reshape(case["rows"], case["cols"])
    least = int(np.rint(case["p"] * 65536))
    x = s["x"].double().cpu().numpy()
    y = np.where(bits < least, 0.0, x * (65536 / (65536 - least)))
    return y if s["residual"] is None else y + s["residual"].double().cpu().numpy()
