"""float64 oracle of the attention gradient, the router over experts with its gradient, and the
sampler: plain numpy, straight from the definitions, row by row where that is simplest.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np


def _f64(x) -> np.ndarray:
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, dtype=np.float64)


# ------------------------------------------------------------------ attention
def attention_probs(q, k, lse, scale, causal) -> np.ndarray:
    """P[s, i, j] = e^(scale q_i . k_j - L_i) over the keys that query i sees, else 0; a row
    whose L is -inf sees none."""
    q, k, lse = _f64(q), _f64(k), _f64(lse)
    s = scale * np.einsum("bid,bjd->bij", q, k)
    n = q.shape[1]
    seen = np.isfinite(lse)[:, :, None] & np.ones((n, n), dtype=bool)
    if causal:
        seen &= np.tri(n, dtype=bool)
    with np.errstate(over="ignore", invalid="ignore"):
        return np.where(seen, np.exp(np.where(seen, s - np.where(seen, lse[:, :, None], 0.0), 0.0)),
                        0.0)


def attention_backward(q, k, v, o, lse, dout, scale, causal=False, dlse=None):
    """(dq, dk, dv), all [bh, n, d]."""
    p = attention_probs(q, k, lse, scale, causal)
    q, k, v, o, do = (_f64(t) for t in (q, k, v, o, dout))
    delta = (o * do).sum(-1)
    if dlse is not None:
        delta = delta - _f64(dlse)
    dp = np.einsum("bid,bjd->bij", do, v)
    ds = p * (dp - delta[:, :, None])
    return (scale * np.einsum("bij,bjd->bid", ds, k), scale * np.einsum("bij,bid->bjd", ds, q),
            np.einsum("bij,bid->bjd", p, do))


# ------------------------------------------------------------------ router
def route_scores(x, score) -> np.ndarray:
    """s of every logit; 0 where the logit is -inf."""
    x = _f64(x)
    there = x > -np.inf
    z = np.where(there, x, 0.0)
    if score == "sigmoid":
        s = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        return np.where(there, s, 0.0)
    m = np.where(there.any(1), np.where(there, x, -np.inf).max(1, initial=-np.inf), 0.0)
    e = np.where(there, np.exp(z - m[:, None]), 0.0)
    d = e.sum(1, keepdims=True)
    return e / np.where(d > 0, d, 1.0)


def route(x, K, score="softmax", bias=None, groups=1, topk_groups=None, group_top=1, renorm=True,
          scale=1.0):
    """(weights [rows, K], experts int32 [rows, K]): one row at a time, by full sorts."""
    x = _f64(x)
    rows, experts = x.shape
    topk_groups = groups if topk_groups is None else topk_groups
    s = route_scores(x, score)
    b = np.zeros(experts) if bias is None else _f64(bias)
    size = experts // groups
    weights, idx = np.zeros((rows, K)), np.zeros((rows, K), dtype=np.int32)
    for r in range(rows):
        c = np.where(x[r] > -np.inf, s[r] + b, -np.inf)
        value = []
        for g in range(groups):
            best = sorted(c[g * size:(g + 1) * size], reverse=True)
            value.append(sum(best[:group_top]))
        order = sorted(range(groups), key=lambda g: (-value[g], g))[:topk_groups]
        allowed = [e for g in order for e in range(g * size, (g + 1) * size)]
        rank = x[r] if bias is None else c
        chosen = sorted(allowed, key=lambda e: (-rank[e], e))[:K]
        idx[r] = chosen
        w = s[r][chosen]
        if renorm:
            # ratios of scores: relative to the largest chosen logit, so that none underflows
            z = x[r][chosen]
            live = z > -np.inf
            if live.any():
                log_s = np.where(live, z, 0.0)
                if score == "sigmoid":
                    log_s = np.minimum(log_s, 0) - np.log1p(np.exp(-np.abs(log_s)))
                e = np.where(live, np.exp(log_s - log_s[live].max()), 0.0)
                w = e / e.sum()
            else:
                w = np.zeros(K)
        weights[r] = w * scale
    return weights, idx


def route_backward(x, idx, dweights, score="softmax", renorm=True, scale=1.0):
    """dx [rows, experts], slot by slot through the Jacobian of the weights."""
    x, dw = _f64(x), _f64(dweights)
    idx = np.asarray(idx.cpu() if hasattr(idx, "cpu") else idx)
    rows, experts = x.shape
    s = route_scores(x, score)
    dx = np.zeros_like(x)
    for r in range(rows):
        slots = [(int(e), scale * dw[r, k]) for k, e in enumerate(idx[r])
                 if 0 <= e < experts and x[r, e] > -np.inf]
        if not slots:
            continue
        e = np.array([a for a, _ in slots])
        g = np.array([b for _, b in slots])
        if renorm:
            z = x[r][e]
            log_s = z if score == "softmax" else np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))
            w = np.exp(log_s - log_s.max())
            w /= w.sum()
            t = w * (g - (g * w).sum())
            if score == "sigmoid":
                t = t * (1 - s[r][e])
            np.add.at(dx[r], e, t)
        elif score == "sigmoid":
            np.add.at(dx[r], e, g * s[r][e] * (1 - s[r][e]))
        else:
            np.add.at(dx[r], e, g * s[r][e])
            dx[r] -= s[r] * (g * s[r][e]).sum()
    return dx


# ------------------------------------------------------------------ sampler
def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(column, probability, kept columns) of one row of logits."""
    x = np.where(np.isnan(x), -np.inf, x)
    if not (x > -np.inf).any():
        return -1, 0.0, np.array([], dtype=np.int64)
    if not temperature > 0:
        at = int(np.argmax(x))
        return at, 1.0, np.array([at])
    m = x.max()
    with np.errstate(invalid="ignore"):
        z = np.where(x == m, 0.0, x - m) / temperature
    w = np.where(x > -np.inf, np.exp(np.where(np.isnan(z), 0.0, z)), 0.0)
    kept = np.argsort(-x, kind="stable")
    kept = kept[x[kept] > -np.inf]
    if 0 < top_k < len(x):
        kept = kept[:top_k]
    if top_p < 1:
        run = np.cumsum(w[kept])
        reach = np.flatnonzero(run >= max(top_p, 0.0) * run[-1])
        kept = kept[:max(1, int(reach[0]) + 1)]
    if min_p > 0:
        kept = kept[w[kept] >= min(min_p, 1.0)]
    kept = np.sort(kept)
    run = np.cumsum(w[kept])
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    at = 0 if u == 0 else int(np.flatnonzero(run > u * run[-1])[0])
    return int(kept[at]), w[kept[at]] / run[-1], kept


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(columns int32 [rows], probabilities [rows]); settings are numbers or arrays."""
    x, u = _f64(x), _f64(u)
    rows = len(x)

    def column(v):
        if not np.isscalar(v):
            return _f64(v)
        return np.full(rows, float(np.float32(v)))

    t, k, p, mp = column(temperature), column(top_k), column(top_p), column(min_p)
    got = [sample_row(x[r], u[r], t[r], int(k[r]), p[r], mp[r]) for r in range(rows)]
    return np.array([g[0] for g in got], dtype=np.int32), np.array([g[1] for g in got])
