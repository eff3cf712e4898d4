"""Float64 NumPy statement of what stands around the expert passes in a training
step: the router with its losses and gradient, the routing weights' gradient, the
RMS norm with the residual's addition and its 8-bit output, and AdamW with 32-bit
or 8-bit moments. Test infrastructure; shares no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np

F8_MAX = 448.0
F8_STEP = 2.0 ** -9
AMAX_MIN = 2.0 ** -100


def takes_part(logits, mask=None):
    """Tokens with at least one logit above -inf (a NaN is one) that are not masked out."""
    x = np.asarray(logits, dtype=np.float64)
    use = ((x > -np.inf) | np.isnan(x)).any(1)
    return use if mask is None else use & (np.asarray(mask) != 0)


def topk(logits, K):
    """The K largest of every row, descending; NaN ranks as -inf, ties to the lower id."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x) + 0.0
    return np.argsort(-x, axis=1, kind="stable")[:, :K].astype(np.int32)


def softmax_rows(logits, use):
    """(p, lse) of the rows in use; zero rows elsewhere."""
    x = np.asarray(logits, dtype=np.float64)
    p, lse = np.zeros_like(x), np.zeros(x.shape[0])
    for t in np.nonzero(use)[0]:
        top = np.max(x[t])
        with np.errstate(invalid="ignore"):
            ex = np.exp(x[t] - top)
            p[t] = ex / ex.sum()
            lse[t] = top + np.log(ex.sum())
    return p, lse


def route(logits, K, renorm=False, balance_coef=0.0, z_coef=0.0, mask=None, idx=None):
    """topk_idx, alpha, counts, prob_sum, loss [2]. ``idx`` fixes the choices."""
    T, E = np.asarray(logits).shape
    use = takes_part(logits, mask)
    idx = topk(logits, K) if idx is None else idx
    p, lse = softmax_rows(logits, use)
    alpha = np.take_along_axis(p, idx.astype(np.int64), 1)
    if renorm:
        s = alpha.sum(1, keepdims=True)
        alpha = alpha / np.where(use[:, None], s, 1.0)
    counts = np.bincount(idx[use].reshape(-1), minlength=E).astype(np.int32)
    prob_sum = p.sum(0)
    n = max(1, int(use.sum()))
    loss = np.array([balance_coef * E / (n * n * K) * float(counts @ prob_sum),
                     z_coef / n * float((lse ** 2).sum())])
    return {"topk_idx": idx, "alpha": alpha, "counts": counts, "prob_sum": prob_sum,
            "loss": loss, "use": use, "p": p, "lse": lse}


def route_bwd(logits, idx, counts, dalpha, dloss=(1.0, 1.0), renorm=False, balance_coef=0.0,
              z_coef=0.0, mask=None):
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    K = idx.shape[1]
    use = takes_part(x, mask)
    p, lse = softmax_rows(x, use)
    n = max(1.0, counts.sum() / K)
    cost = dloss[0] * balance_coef * E * np.asarray(counts, dtype=np.float64) / (n * n * K)
    out = np.zeros_like(x)
    for t in np.nonzero(use)[0]:
        dp = cost.copy()
        chosen = idx[t].astype(np.int64)
        da = np.zeros(K) if dalpha is None else np.asarray(dalpha, dtype=np.float64)[t]
        if not renorm:
            dp[chosen] += da
        out[t] = p[t] * (dp - p[t] @ dp) + p[t] * dloss[1] * 2 * z_coef * lse[t] / n
        if renorm:
            a = p[t, chosen] / p[t, chosen].sum()
            out[t, chosen] += a * (da - a @ da)
    return out


def gate_grad(g, y, inv, K):
    g, y = np.asarray(g, dtype=np.float64), np.asarray(y, dtype=np.float64)
    T = g.shape[0]
    return np.einsum("td,tkd->tk", g, y[np.asarray(inv)].reshape(T, K, -1))


def e4m3_grid():
    """The non-negative e4m3 values: subnormals m 2^-9, then (8 + m) 2^(e - 10)."""
    vals = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        for m in range(8):
            if not (e == 15 and m == 7):  # that code is NaN
                vals.append((8 + m) * 2.0 ** (e - 10))
    return np.array(vals)


def e4m3(v):
    """Nearest e4m3 value (ties to the even code), saturating."""
    grid = e4m3_grid()
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), F8_MAX)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(v), np.nan, np.sign(v) * grid[pick])


def add_rmsnorm(x, res, w, eps, q_cols=None):
    h = np.asarray(x, dtype=np.float64)
    if res is not None:
        h = h + np.asarray(res, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None] * np.asarray(w, dtype=np.float64)
    out = {"h": h, "rstd": rstd, "y": y}
    if q_cols is not None:
        D = h.shape[1]
        cols = q_cols or D
        scale = np.stack([np.maximum(np.abs(y[:, c:c + cols]).max(1), AMAX_MIN) / F8_MAX
                          for c in range(0, D, cols)], 1)
        out["q_scale"] = scale
        out["q"] = e4m3(y / np.repeat(scale, cols, axis=1)[:, :D])
    return out


def add_rmsnorm_bwd(dy, dh, h, w, rstd):
    dy, h = np.asarray(dy, dtype=np.float64), np.asarray(h, dtype=np.float64)
    rs = np.asarray(rstd, dtype=np.float64)[:, None]
    xhat = h * rs
    wdy = dy * np.asarray(w, dtype=np.float64)
    dx = rs * (wdy - xhat * (wdy * xhat).mean(1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, dtype=np.float64)
    return dx, (dy * xhat).sum(0)


def quantise_blocks(v, root=False, block=256):
    """(e4m3 values, scales) of the blocks of a vector; root: positive stays positive."""
    v = np.asarray(v, dtype=np.float64)
    n = v.shape[0]
    nb = -(-n // block)
    b = np.zeros(nb * block)
    b[:n] = v
    b = b.reshape(nb, block)
    scale = np.maximum(np.abs(b).max(1), AMAX_MIN) / F8_MAX
    s = b / scale[:, None]
    if root:
        s = np.where(b > 0, np.maximum(s, F8_STEP), s)
    return e4m3(s).reshape(-1)[:n], scale


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """New (p, m, v)."""
    p, g = np.asarray(p, dtype=np.float64), np.asarray(g, dtype=np.float64) * grad_scale
    m = beta1 * np.asarray(m, dtype=np.float64) + (1 - beta1) * g
    v = beta2 * np.asarray(v, dtype=np.float64) + (1 - beta2) * g * g
    mhat, vhat = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p * (1 - lr * weight_decay) - lr * mhat / (np.sqrt(vhat) + eps), m, v
