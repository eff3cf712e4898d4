"""Float64 NumPy statement of the operators for training under tight memory: the router
over groups of experts with its gradient and the bias's step, the saved state in 8 bits
and what the backward pass rebuilds from it, the norms around a block with their
gradients. Test infrastructure; shares no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np

from .step_oracle import AMAX_MIN, F8_MAX, e4m3, takes_part


def scores(logits, fn):
    """s of every logit, and s / sum_e s (0 where that sum is 0)."""
    x = np.asarray(logits, dtype=np.float64)
    s, share = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        row, top = x[t], np.fmax.reduce(x[t])
        if top == -np.inf and not np.isnan(row).any():
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            if fn == "softmax":
                ex = np.exp(row - top)
                s[t] = share[t] = ex / ex.sum()
                continue
            s[t] = np.where(row >= 0, 1 / (1 + np.exp(-row)), np.exp(row) / (1 + np.exp(row)))
            m = min(top, 0.0)  # the shares of very low logits
            f = np.where(row >= 0, 1 / (1 + np.exp(-row)), np.exp(row - m) / (1 + np.exp(row)))
            s[t] = np.where(row == np.inf, 1.0, s[t])
            f = np.where(row == np.inf, 1.0, f)
            share[t] = f / f.sum() if f.sum() != 0 else 0.0
    return s, share


def choose(logits, K, fn="sigmoid", bias=None, groups=1, top_groups=1, group_top=2):
    """The K choices of every token, by sorting tuples."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    s, _ = scores(x, fn)
    v = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    size = E // groups
    out = np.zeros((T, K), dtype=np.int32)
    for t in range(T):
        opened = x[t] > -np.inf
        ranked = []
        for g in range(groups):
            mine = sorted((v[t, e] for e in range(g * size, (g + 1) * size) if opened[e]),
                          reverse=True)[:group_top]
            ranked.append((-sum(mine) if mine else np.inf, g))
        kept = {g for _, g in sorted(ranked)[:top_groups]}
        key = x[t] if bias is None else v[t]
        order = sorted((-key[e] if opened[e] else np.inf, e) for e in range(E)
                       if e // size in kept)
        out[t] = [e for _, e in order[:K]]
    return out


def choose_rows(logits, K, fn="sigmoid", bias=None, groups=1, top_groups=1, group_top=2):
    """What ``choose`` gives, for all tokens at once by stable sorts."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    s, _ = scores(x, fn)
    v = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    opened = x > -np.inf
    best = -np.sort(np.where(opened, -v, np.inf).reshape(T, groups, E // groups))[..., :group_top]
    score = np.where(best[..., 0] > -np.inf, np.where(best > -np.inf, best, 0.0).sum(-1), -np.inf)
    rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1)
    dropped = np.repeat(rank >= top_groups, E // groups, axis=1)
    key = np.where(opened, -(x if bias is None else v), np.inf)
    return np.lexsort((key, dropped), axis=1)[:, :K].astype(np.int32)


def group_route(logits, K, fn="sigmoid", bias=None, groups=1, top_groups=1, group_top=2,
                renorm=True, scale=1.0, balance_coef=0.0, mask=None, idx=None):
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    use = takes_part(x, mask)
    if idx is None:
        idx = choose(x, K, fn, bias, groups, top_groups, group_top)
    s, share = scores(x, fn)
    share = np.where(use[:, None], share, 0.0)
    alpha = np.take_along_axis(s, idx.astype(np.int64), 1)
    if renorm:
        for t in range(T):
            row = x[t, idx[t]]
            top = np.fmax.reduce(row)
            if fn == "sigmoid" and top < 0 and top > -np.inf:  # ratios of very low scores
                w = np.exp(row - top) / (1 + np.exp(row))
            elif fn == "softmax" and np.isfinite(row).any() and np.isfinite(s[t]).all():
                w = np.exp(row - top)
            else:
                w = alpha[t]
            total = w.sum()
            alpha[t] = w / total if total != 0 else 0.0
    alpha = np.where(use[:, None], alpha * scale, 0.0)
    counts = np.bincount(idx[use].reshape(-1), minlength=E).astype(np.int32)
    prob_sum = share.sum(0)
    n = max(1, int(use.sum()))
    loss = balance_coef * E / (n * n * K) * float(counts @ prob_sum)
    return {"topk_idx": idx, "alpha": alpha, "counts": counts, "prob_sum": prob_sum,
            "loss": np.array([loss]), "use": use, "s": s, "share": share}


def group_route_bwd(logits, idx, counts, dalpha, dloss=1.0, fn="sigmoid", renorm=True, scale=1.0,
                    balance_coef=0.0, mask=None):
    """Two chains kept apart: weights -> scores -> logits, and shares -> logits."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    K = idx.shape[1]
    use = takes_part(x, mask)
    s, share = scores(x, fn)
    n = max(1.0, counts.sum() / K)
    cost = dloss * balance_coef * E * np.asarray(counts, dtype=np.float64) / (n * n * K)
    out = np.zeros_like(x)
    for t in np.nonzero(use)[0]:
        # d share_e / d x_f = share_e (1 - s_e) [e = f] - share_e share_f (1 - s_f) (sigmoid),
        # the same without the (1 - s) for the softmax
        with np.errstate(over="ignore"):
            less = 1 / (1 + np.exp(x[t])) if fn == "sigmoid" else np.ones(E)
        out[t] = share[t] * less * (cost - share[t] @ cost)
        if dalpha is None:
            continue
        c = idx[t].astype(np.int64)
        da = np.asarray(dalpha, dtype=np.float64)[t] * scale
        if renorm:
            a = group_route(x[t:t + 1], K, fn, renorm=True, idx=idx[t:t + 1])["alpha"][0]
            out[t, c] += a * less[c] * (da - a @ da)
        else:
            out[t, c] += s[t, c] * less[c] * da
            if fn == "softmax":
                out[t] -= s[t] * (s[t, c] @ da)
    return out


def bias_step(bias, counts, rate):
    counts = np.asarray(counts, dtype=np.int64)
    lack = counts.sum() - counts.size * counts
    return np.asarray(bias, dtype=np.float64) + rate * np.sign(lack)


def quantise_rows(v, cols):
    """(e4m3 values, scales) of each ``cols`` columns of the rows (0: of a row)."""
    v = np.asarray(v, dtype=np.float64)
    width = v.shape[1]
    cols = cols or width
    amax = np.stack([np.fmax(np.fmax.reduce(np.abs(v[:, c:c + cols]), axis=1), AMAX_MIN)
                     for c in range(0, width, cols)], 1)
    with np.errstate(invalid="ignore"):
        # 448 v is exact: a quotient that lies between two codes is one, and goes to the even
        # one, where v over a rounded scale would fall to either side
        return e4m3(v * F8_MAX / np.repeat(amax, cols, axis=1)[:, :width]), amax / F8_MAX


def phi(a, b):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a)) * b


def pack(ab, cols):
    ab = np.asarray(ab, dtype=np.float64)
    H = ab.shape[1] // 2
    (qa, sa), (qb, sb) = quantise_rows(ab[:, :H], cols), quantise_rows(ab[:, H:], cols)
    return (np.concatenate([qa, qb], 1), np.concatenate([sa, sb], 1),
            (phi(ab[:, :H], ab[:, H:]) ** 2).sum(1))


def decode(q, scale, cols):
    q = np.asarray(q, dtype=np.float64)
    return q * np.repeat(np.asarray(scale, dtype=np.float64), cols or q.shape[1],
                         axis=1)[:, :q.shape[1]]


def unpack(q, scale, cols):
    """[a | b] and phi of a packed state."""
    H, G = q.shape[1] // 2, scale.shape[1] // 2
    a, b = decode(q[:, :H], scale[:, :G], cols), decode(q[:, H:], scale[:, G:], cols)
    return np.concatenate([a, b], 1), phi(a, b)


def block_norm(block, res, w, w_post=None, gate=None, gate_kind=None, res_scale=1.0, eps=0.0,
               q_cols=None):
    u = np.asarray(block, dtype=np.float64)
    out = {}
    if w_post is not None:
        out["block_rstd"] = 1.0 / np.sqrt((u * u).mean(1) + eps)
        u = u * out["block_rstd"][:, None] * np.asarray(w_post, dtype=np.float64)
    if gate is not None:
        g = np.asarray(gate, dtype=np.float64)
        u = u * (g[:, None] if gate_kind == "token" else g[None, :])
    h = res_scale * np.asarray(res, dtype=np.float64) + u
    out["h"], out["rstd"] = h, 1.0 / np.sqrt((h * h).mean(1) + eps)
    out["y"] = h * out["rstd"][:, None] * np.asarray(w, dtype=np.float64)
    if q_cols is not None:
        out["q"], out["q_scale"] = quantise_rows(out["y"], q_cols)
    return out


def block_norm_bwd(dy, dh, h, block, w, rstd, w_post=None, gate=None, gate_kind=None,
                   block_rstd=None, res_scale=1.0):
    dy, h, o = (np.asarray(v, dtype=np.float64) for v in (dy, h, block))
    rs = np.asarray(rstd, dtype=np.float64)[:, None]
    xhat, wdy = h * rs, dy * np.asarray(w, dtype=np.float64)
    dhs = rs * (wdy - xhat * (wdy * xhat).mean(1, keepdims=True))
    if dh is not None:
        dhs = dhs + np.asarray(dh, dtype=np.float64)
    out = {"dres": res_scale * dhs, "dw": (dy * xhat).sum(0), "dhs": dhs}
    g = 1.0
    if gate is not None:
        g = np.asarray(gate, dtype=np.float64)
        g = g[:, None] if gate_kind == "token" else g[None, :]
    if w_post is not None:
        wp, rb = np.asarray(w_post, dtype=np.float64), np.asarray(block_rstd, np.float64)[:, None]
        ohat = o * rb
        u = ohat * wp
        out["dw_post"] = (g * dhs * ohat).sum(0)
        k = wp * g * dhs
        out["dblock"] = rb * (k - ohat * (k * ohat).mean(1, keepdims=True))
    else:
        u = o
        out["dblock"] = g * dhs
    if gate is not None:
        out["dgate"] = (dhs * u).sum(1 if gate_kind == "token" else 0)
    return out
