"""float64 oracle of the decode loop's operators: a paged key-value cache (append with rotation,
attention of one new token, reordering) and beam search's selection.  Plain numpy, token by token
and page by page, straight from the definitions.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

from .operators import _f64


def _ints(x) -> np.ndarray:
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").numpy()
    return np.asarray(x, dtype=np.int64)


def place(table, pages, page_size, b, pos):
    """(page, slot) of a sequence's position, or None where the table has none of the pool's."""
    if pos < 0 or pos // page_size >= table.shape[1]:
        return None
    page = int(table[b, pos // page_size])
    return (page, pos % page_size) if 0 <= page < pages else None


def rotate(x, pos, inv_freq, interleaved):
    """One token's heads [heads, d] turned by its position."""
    if inv_freq is None:
        return x.copy()
    a = pos * _f64(inv_freq)
    half, out = len(a), x.copy()
    one = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    two = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    out[:, one] = x[:, one] * np.cos(a) - x[:, two] * np.sin(a)
    out[:, two] = x[:, two] * np.cos(a) + x[:, one] * np.sin(a)
    return out


def new_tokens(lengths, starts, tokens):
    """(token, sequence, position) of the tokens that take part."""
    lengths = _ints(lengths)
    for b in range(len(lengths)):
        lo, hi = (b, b + 1) if starts is None else (int(starts[b]), int(starts[b + 1]))
        for t in range(max(lo, 0), min(hi, tokens)):
            if lengths[b] - hi + t >= 0:
                yield t, b, int(lengths[b]) - hi + t


def append(k_cache, v_cache, table, lengths, k, v, q=None, starts=None, inv_freq=None,
           interleaved=False, q_out=None):
    """(k_cache, v_cache, q_out) behind the append; rows of q_out that take no part are q_out's."""
    k_cache, v_cache, k, v, table = _f64(k_cache), _f64(v_cache), _f64(k), _f64(v), _ints(table)
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    if q is not None:
        q = _f64(q)
        q_out = np.zeros_like(q) if q_out is None else _f64(q_out).copy()
    starts = None if starts is None else _ints(starts)
    for t, b, pos in new_tokens(lengths, starts, len(k)):
        if q is not None:
            q_out[t] = rotate(q[t], pos, inv_freq, interleaved)
        at = place(table, len(k_cache), k_cache.shape[2], b, pos)
        if at is not None:
            k_cache[at[0], :, at[1]] = rotate(k[t], pos, inv_freq, interleaved)
            v_cache[at[0], :, at[1]] = v[t]
    return k_cache, v_cache, q_out


def keys_of(cache, table, lengths, b):
    """The places of sequence b's keys, [n, 2]."""
    size = cache.shape[2]
    length = max(0, min(int(_ints(lengths)[b]), table.shape[1] * size))
    places = (place(table, len(cache), size, b, p) for p in range(length))
    return np.array([p for p in places if p is not None], dtype=np.int64).reshape(-1, 2)


def attention(q, k_cache, v_cache, table, lengths, scale):
    """(O, L, A) with A = sum of the weights times |v|, which bounds O's rounding errors."""
    q, table = _f64(q), _ints(table)
    seqs, heads, d = q.shape
    group = heads // k_cache.shape[1]
    out, weighted = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((seqs, heads), -np.inf)
    for b in range(seqs):
        at = keys_of(k_cache, table, lengths, b)
        if not len(at):
            continue
        # (only the pages in use are widened: the rest may hold anything)
        k, v = (_f64(c[at[:, 0], :, at[:, 1]]) for c in (k_cache, v_cache))
        for h in range(heads):
            s = scale * (k[:, h // group] @ q[b, h])
            w = np.exp(s - s.max())
            lse[b, h] = s.max() + np.log(w.sum())
            w /= w.sum()
            out[b, h], weighted[b, h] = w @ v[:, h // group], w @ np.abs(v[:, h // group])
    return out, lse, weighted


def reorder(k_cache, v_cache, table, lengths, parents, out_table, page_size):
    """(k_cache, v_cache, out_table, out_lengths); the caches are [layers, pages, ...]."""
    new_k, new_v, new_table = k_cache.copy(), v_cache.copy(), _ints(out_table).copy()
    table, lengths, parents = _ints(table), _ints(lengths), _ints(parents)
    beams, pages = parents.shape[1], k_cache.shape[1]
    out_lengths = np.zeros(len(table), dtype=np.int64)
    for j, parent in enumerate(parents.reshape(-1)):
        if not 0 <= parent < beams:
            continue
        p = j // beams * beams + int(parent)
        out_lengths[j] = length = max(0, min(int(lengths[p]), table.shape[1] * page_size))
        full, rest = divmod(length, page_size)
        new_table[j, :full] = table[p, :full]
        if rest:
            here, there = int(table[p, full]), int(new_table[j, full])
            if 0 <= here < pages and 0 <= there < pages:
                new_k[:, there, :, :rest] = k_cache[:, here, :, :rest]
                new_v[:, there, :, :rest] = v_cache[:, here, :, :rest]
    return new_k, new_v, new_table, out_lengths


# ------------------------------------------------------------------ beam search
def beam_values(x, scores, ended=None, pad=0):
    """c of every continuation, [groups, beams, cols]; -inf where there is none."""
    scores = _f64(scores)
    groups, beams = scores.shape
    x = _f64(x).reshape(groups, beams, -1)
    x = np.where(np.isnan(x), -np.inf, x)
    c = np.full(x.shape, -np.inf)
    for g in range(groups):
        for i in range(beams):
            row, s = x[g, i], scores[g, i]
            if not s > -np.inf:
                continue
            if ended is not None and bool(ended[g][i]):
                c[g, i, pad] = s
                continue
            m = row.max()
            if m == -np.inf:
                continue
            there = row == m if m == np.inf else row > -np.inf
            z = np.zeros(there.sum()) if m == np.inf else row[there] - m
            c[g, i, there] = s + z - np.log(np.exp(z).sum())
    return c


def beam_select(x, scores, K, ended=None, pad=0):
    """(values, parents, tokens), [groups, K]."""
    c = beam_values(x, scores, ended, pad)
    groups, _, cols = c.shape
    values = np.full((groups, K), -np.inf)
    parents, tokens = (np.full((groups, K), -1, dtype=np.int64) for _ in range(2))
    for g in range(groups):
        flat = c[g].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:K]
        order = order[flat[order] > -np.inf]
        n = len(order)
        values[g, :n], parents[g, :n], tokens[g, :n] = flat[order], order // cols, order % cols
    return values, parents, tokens
