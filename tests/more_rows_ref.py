"""Routing, verification of drafts and cache eviction in plain numpy, 64 bits,
one item after another.  Shares no code with the library."""

import numpy as np

U_LO, U_HI = 2.0 ** -25, 1.0 - 2.0 ** -24
MOST = float(np.finfo(np.float32).max)
E24 = 2.0 ** -24


def clean(x):
    """Logits as the operators read them."""
    x = np.asarray(x, np.float64)
    return np.where(np.isnan(x), -np.inf, np.minimum(x, MOST))


def softmax(x):
    """-> p, the distance of each logit from the largest (0 where there is none)."""
    m = x.max(-1, keepdims=True)
    z = x - np.where(m > -np.inf, m, 0.0)
    w = np.where(x > -np.inf, np.exp(np.maximum(z, -800.0)), 0.0)
    total = w.sum(-1, keepdims=True)
    return w / np.where(total > 0, total, 1.0), np.where(w > 0, -z, 0.0)


def route(logits, topk, normalize, mask):
    """-> ids, weights, counts, load, loss, p, |z|."""
    x = clean(logits)
    if mask is not None:
        x = np.where(mask[:, None], x, -np.inf)
    tokens, experts = x.shape
    p, z = softmax(x)
    ids = np.full((tokens, topk), -1, np.int64)
    weights = np.zeros((tokens, topk))
    counts = np.zeros(experts + 1, np.int64)
    for t in range(tokens):
        order = np.lexsort((np.arange(experts), -x[t]))[:topk]
        order = order[x[t, order] > -np.inf]
        ids[t, :order.size] = order
        weights[t, :order.size] = p[t, order] / (p[t, order].sum() if normalize else 1.0)
        counts[order] += 1
        counts[experts] += order.size > 0
    n, pairs = counts[experts], counts[:experts].sum()
    load = p.sum(0) / max(n, 1)
    loss = experts * float(counts[:experts] @ load) / max(pairs, 1)
    return ids, weights, counts, load, loss, p, z


def route_grad(logits, ids, counts, dweights, dloss, normalize):
    """-> dx, and the sum of the magnitudes of its terms."""
    x = clean(logits)
    tokens, experts = x.shape
    n, pairs = counts[experts], counts[:experts].sum()
    a = np.zeros(experts)
    if dloss is not None and n > 0:
        a = float(dloss) * experts / n * counts[:experts] / max(pairs, 1)
    out, size = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(tokens):
        if not 0 <= ids[t, 0] < experts:
            continue
        p, _ = softmax(x[t])
        out[t] = p * (a - p @ a)
        size[t] = p * (np.abs(a) + p @ np.abs(a))
        if dweights is None:
            continue
        chosen = [(int(e), float(g)) for e, g in zip(ids[t], dweights[t]) if 0 <= e < experts]
        w = np.array([p[e] for e, _ in chosen])
        g = np.array([g for _, g in chosen])
        if normalize:
            w = w / w.sum()
        inner, bound = w @ g, w @ np.abs(g)
        for (e, _), wj, gj in zip(chosen, w, g):
            out[t, e] += wj * (gj - inner) if normalize else wj * gj
            size[t, e] += wj * (abs(gj) + bound)
        if not normalize:
            out[t] -= p * inner
            size[t] += p * bound
    return out, size


def verify(logits, drafts, accept, uniform, draft_logits, temperature, slack=2.0 ** -16):
    """One sequence -> tokens, accepted, logprobs, whether every decision is clear by more than `slack`."""
    k, vocab = len(drafts), logits.shape[1]
    tokens, logprobs = np.full(k + 1, -1, np.int64), np.full(k + 1, -np.inf)
    sure = True
    for j in range(k + 1):
        x = clean(logits[j])
        if x.max() == -np.inf:
            return tokens, j, logprobs, sure
        d = int(drafts[j]) if j < k else -1
        real = 0 <= d < vocab
        if uniform is None or not temperature > 0:
            best = int(np.argmax(x))
            tokens[j], logprobs[j] = best, 0.0
            if real and d == best:
                continue
            return tokens, j, logprobs, sure
        p, _ = softmax(x / temperature)
        q = np.zeros(vocab)
        if real:
            if draft_logits is None:
                q[d] = 1.0
            else:
                q, _ = softmax(clean(draft_logits[j]) / temperature)
            u = min(max(0.0 if np.isnan(accept[j]) else float(accept[j]), U_LO), U_HI)
            sure &= abs(u * q[d] - p[d]) > slack * p[d]
            if u * q[d] < p[d]:
                tokens[j], logprobs[j] = d, np.log(p[d])
                continue
        r = np.maximum(p - q, 0.0)
        v = np.clip(np.where(np.isnan(uniform), 0.0, uniform.astype(np.float64)), U_LO, U_HI)
        ratio = r / -np.log(v)
        best = int(np.argmax(ratio))
        # each r is off by up to slack of p and q
        low = (r[best] - slack * (p[best] + q[best])) / -np.log(v[best])
        others = np.delete((r + slack * (p + q)) / -np.log(v), best)
        sure &= others.size == 0 or low > others.max()
        tokens[j], logprobs[j] = best, np.log(p[best]) if p[best] > 0 else -np.inf
        return tokens, j, logprobs, sure
    return tokens, k, logprobs, sure


def score(weights, scores, heads, decay, lengths, queries):
    """-> out, the sum of the magnitudes of its terms."""
    batch, query_heads, count, length = weights.shape
    group = query_heads // heads
    out, size = np.zeros((batch, heads, length)), np.zeros((batch, heads, length))
    for b in range(batch):
        n = length if lengths is None else min(max(int(lengths[b]), 0), length)
        m = count if queries is None else min(max(int(queries[b]), 0), count)
        for h in range(heads):
            w = weights[b, h * group:(h + 1) * group, :m, :n].reshape(group * m, n)
            out[b, h, :n] = w.sum(0)
            size[b, h, :n] = np.abs(w).sum(0)
            if scores is not None:
                out[b, h, :n] += float(np.float32(decay)) * scores[b, h, :n]
                size[b, h, :n] += np.abs(float(np.float32(decay)) * scores[b, h, :n])
    return out, size


def kept(scores, n, budget, sinks, recent):
    """One head's kept positions."""
    if n <= budget:
        return np.arange(n)
    middle = np.arange(sinks, n - recent)
    s = scores[middle].astype(np.float64)
    s = np.where(np.isnan(s), -np.inf, s)
    best = middle[np.lexsort((middle, -s))[:budget - sinks - recent]]
    return np.sort(np.concatenate([np.arange(sinks), best, np.arange(n - recent, n)])).astype(np.int64)
