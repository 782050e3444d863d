"""Plain reference of the log probabilities and their gradient (numpy, float64),
with bounds for a computation in float32."""
import numpy as np

U = 2.0 ** -24


def forward(x, targets, mask, scale, k):
    """dict of outputs and of their bounds for float64 x [rows, n], targets [rows, T], mask [rows, n] or None.

    A difference from the maximum, its factor (rounded) and the product lose 4 U
    of it; an exponential 2^-22 and as much as its argument is off; a sum of n
    terms at most n U of itself, W's terms as much of their own sum. A logarithm
    is off by 2 units of its last place and by its argument's relative error."""
    rows, n = x.shape
    y = x if mask is None else np.where(mask != 0, x, -np.inf)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = y.max(axis=1, initial=-np.inf)
        empty = m == -np.inf
        broken = np.isnan(y).any(axis=1) | (m == np.inf)
        d = scale * (y - np.where(empty, 0.0, m)[:, None])
        e = np.exp(d)
        total = e.sum(axis=1)
        L = np.log(total)
        lp = np.where(empty[:, None], -np.inf, d - L[:, None])
        p = np.where(empty[:, None], 0.0, e / total[:, None])
        dd = np.where(p > 0, d, 0.0)
        D = (p * np.abs(dd)).sum(axis=1)
        H = np.where(empty, 0.0, L + (p * -dd).sum(axis=1))
        H = np.where(broken, np.nan, H)
        lp = np.where(broken[:, None], np.nan, lp)
        plain = ~(empty | broken)
        L, D, total = np.where(plain, L, 0.0), np.where(plain, D, 0.0), np.where(plain, total, 1.0)
        rel = 2.0 ** -21 + 2 * n * U + 8 * U * D              # of the sum, and of a probability near the maximum
        lp_err = 5 * U * np.abs(np.where(np.isfinite(d), d, 0.0)) + (rel + 4 * U * np.abs(L))[:, None]
        H_err = 2 * rel * (1 + D) + 4 * U * (np.abs(L) + D) + 4 * U * D * np.abs(np.log(np.maximum(total, 1)))
    given = targets >= 0
    r = np.arange(rows)[:, None]
    out = {"logprob": np.where(given, lp[r, np.where(given, targets, 0)], 0.0), "entropy": H, "p": p, "lp": lp}
    err = {"logprob": np.where(given, lp_err[r, np.where(given, targets, 0)], 0.0), "entropy": H_err, "rel": rel, "lp": lp_err}
    # an inactive column's log probability is minus infinity whatever the row
    if mask is not None:
        off = given & (mask[r, np.where(given, targets, 0)] == 0)
        out["logprob"] = np.where(off, -np.inf, out["logprob"])
    if k:
        z = np.where(np.isnan(y), -np.inf, y)
        order = np.argsort(-z, axis=1, kind="stable")[:, :k]
        listed = np.take_along_axis(z, order, 1) > -np.inf
        out["top_idx"] = np.where(listed, order, -1)
        out["top_logprob"] = np.where(listed, np.take_along_axis(lp, order, 1), -np.inf)
        err["top_logprob"] = np.take_along_axis(lp_err, order, 1)
    return out, err


def backward(out, err, targets, scale, g, g_entropy, g_top, mask):
    """(gradient, bound) in float64."""
    p, lp, H = out["p"], out["lp"], out["entropy"]
    rows, n = p.shape
    hot, mag, total, size = np.zeros((rows, n)), np.zeros((rows, n)), np.zeros(rows), np.zeros(rows)
    def add(columns, values):
        for r in range(rows):
            for j, v in zip(columns[r], values[r]):
                if j >= 0 and lp[r, j] > -np.inf and (mask is None or mask[r, j]):
                    hot[r, j] += v
                    mag[r, j] += abs(v)
                    total[r] += v
                    size[r] += abs(v)
    if g is not None:
        add(targets, g)
    if g_top is not None:
        add(out["top_idx"], g_top)
    gh = np.zeros(rows) if g_entropy is None else g_entropy
    with np.errstate(invalid="ignore"):
        l0 = np.where(p > 0, lp, 0.0)
        dx = hot - p * (total[:, None] + gh[:, None] * (l0 + H[:, None]))
        rel_p = err["rel"][:, None] + 2.0 ** -21 + err["lp"]
        inner = size[:, None] * (targets.shape[1] + 80) * U + np.abs(gh)[:, None] * (
            err["lp"] + err["entropy"][:, None] + 6 * U * (np.abs(l0) + np.abs(H)[:, None]))
        whole = size[:, None] + np.abs(gh)[:, None] * (np.abs(l0) + np.abs(H)[:, None])
        # an exponential below 2^-126 is 0, and so may a product of one be
        bound = 2.0 ** -125 * (1 + whole) + p * (rel_p * whole + inner + 6 * U * whole) + (targets.shape[1] + 80) * U * mag + 4 * U * np.abs(dx)
    if mask is not None:
        dx, bound = np.where(mask != 0, dx, 0.0), np.where(mask != 0, bound, 0.0)
    return scale * dx, scale * bound
