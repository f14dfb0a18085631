"""The row operators in plain numpy, 64 bits, one item after another where
that is affordable.  Shares no code with the library."""

import numpy as np

U_LO, U_HI = 2.0 ** -25, 1.0 - 2.0 ** -24
# Relative error of one rounding to nearest (half a unit in the last place at
# most: 24, 8 and 11 significant bits), and the smallest step near zero.
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def capacity(tokens, topk, experts, align):
    pairs = tokens * topk
    return pairs + min(pairs, experts) * (align - 1)


def plan(ids, experts, align, rows):
    """-> offsets, counts, slots, pairs."""
    flat = ids.reshape(-1)
    offsets = np.zeros(experts + 1, np.int64)
    counts = np.zeros(experts, np.int64)
    slots = np.full(flat.size, -1, np.int64)
    pairs = np.full(rows, -1, np.int64)
    at = 0
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        offsets[e], counts[e] = at, mine.size
        slots[mine] = at + np.arange(mine.size)
        pairs[at:at + mine.size] = mine
        at += -(-mine.size // align) * align
    offsets[experts] = at
    return offsets, counts, slots.reshape(ids.shape), pairs


def dispatch(x, pairs, topk):
    out = np.zeros((pairs.size, x.shape[1]))
    has = pairs >= 0
    out[has] = x[pairs[has] // topk]
    return out


def combine(y, slots, weights):
    """-> out, and the sum of the terms' magnitudes."""
    out = np.zeros((slots.shape[0], y.shape[1]))
    size = np.zeros_like(out)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            s = slots[t, j]
            if 0 <= s < y.shape[0]:
                term = (1.0 if weights is None else float(weights[t, j])) * y[s]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_grad(g, y, slots, pairs, weights):
    """-> dy, dweights, and the sum of the magnitudes of each dot's terms."""
    dy = np.zeros((pairs.size, g.shape[1]))
    dw = np.zeros(slots.shape)
    size = np.zeros(slots.shape)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            s = slots[t, j]
            if 0 <= s < pairs.size:
                dy[s] = (1.0 if weights is None else float(weights[t, j])) * g[t]
                dw[t, j] = g[t] @ y[s]
                size[t, j] = np.abs(g[t]) @ np.abs(y[s])
    return dy, dw, size


def embedding(table, ids, scale):
    out = np.zeros((ids.size, table.shape[1]))
    has = (ids >= 0) & (ids < table.shape[0])
    out[has] = table[ids[has]] * float(np.float32(scale))
    return out


def embedding_grad(g, ids, vocab, scale):
    """-> dtable, the sum of the magnitudes, the number of terms per row."""
    out = np.zeros((vocab, g.shape[1]))
    size = np.zeros_like(out)
    count = np.zeros(vocab)
    for i, v in enumerate(ids):
        if 0 <= v < vocab:
            out[v] += float(np.float32(scale)) * g[i]
            size[v] += abs(float(np.float32(scale))) * np.abs(g[i])
            count[v] += 1
    return out, size, count


def kept_tokens(x, t, top_k, top_p, min_p):
    """One row's kept tokens in their order, their z and w."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, float(np.finfo(np.float32).max)))
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if order.size == 0:
        return order, None, None
    z = (x[order] - x[order[0]]) / t
    w = np.exp(z)
    if 0 < top_k < order.size:
        order, z, w = order[:top_k], z[:top_k], w[:top_k]
    n = order.size
    if top_p < 1:
        total, before, n = w.sum(), 0.0, 0
        while n < order.size and (n == 0 or before < top_p * total):
            before += w[n]
            n += 1
    keep = np.arange(order.size) < n
    if min_p > 0:
        keep &= w >= min(min_p, 1.0)
    keep &= w > 1e-45
    return order[keep], z[keep], w[keep]


def sample(x, u, t, top_k, top_p, min_p):
    """One row -> (token, logprob, z of the token)."""
    if not t > 0:
        order, _, _ = kept_tokens(x, 1.0, 0, 1.0, 0.0)
        return (int(order[0]), 0.0, 0.0) if order.size else (-1, -np.inf, 0.0)
    order, z, w = kept_tokens(x, t, top_k, top_p, min_p)
    if order.size == 0:
        return -1, -np.inf, 0.0
    u = np.clip(np.where(np.isnan(u[order]), 0.0, u[order]), U_LO, U_HI)
    score = z - np.log(-np.log(u))
    best = min(np.flatnonzero(score == score.max()), key=lambda i: order[i])
    return int(order[best]), float(z[best] - np.log(w.sum())), float(z[best])
