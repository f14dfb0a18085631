"""Cases of the language-model operators of libgc, with their plain forms.

Three operators, all of them a partition, a sort or a selection with rows or
scores attached:

* tokens sorted by expert and back ("exchange", "exchange_grad"): every token
  names top-k experts; its row is copied to each expert's block of rows, and
  the experts' results come back as a weighted sum per token.  The gradient
  goes the other way through the same slots.
* embedding lookup with scaling ("embed") and its gradient by sorted tokens
  ("embed_grad").
* sampling with temperature, top-k, top-p and min-p from given uniform random
  numbers ("sample").

A case is a dict of plain values.  ``own`` selects what ``run`` does: the plain
form in elementary torch operations, or the library's entry points.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
IDS = {"i32": torch.int32, "i64": torch.int64}

# Uniforms are clamped to [U_LO, U_HI] before their logarithms are taken.
U_LO, U_HI = 2.0 ** -25, 1.0 - 2.0 ** -24


def listed():
    return [
        # One step of a small serving batch: what counts is the latency of the calls.
        {"name": "exchange_decode", "op": "exchange", "tokens": 16, "width": 2048, "experts": 64, "topk": 4,
         "align": 1, "drop": 0.0, "pad": 0, "dtype": "bf16", "ids": "i64"},
        # A prompt of odd length on one of several expert groups: the ids that live elsewhere are dropped, the
        # width is odd, the input rows are a slice of wider ones, the experts' blocks start at multiples of 16.
        {"name": "exchange_ragged", "op": "exchange", "tokens": 1531, "width": 1001, "experts": 60, "topk": 3,
         "align": 16, "drop": 0.3, "pad": 5, "dtype": "f16", "ids": "i32"},
        # The largest forward pass: a training batch, blocks aligned for a tiled grouped product.
        {"name": "exchange_train", "op": "exchange", "tokens": 16384, "width": 2048, "experts": 128, "topk": 8,
         "align": 128, "drop": 0.0, "pad": 0, "dtype": "bf16", "ids": "i64"},
        # The gradient of a small layer kept in 32 bits.
        {"name": "exchange_grad_small", "op": "exchange_grad", "tokens": 700, "width": 1024, "experts": 8, "topk": 2,
         "align": 1, "drop": 0.0, "pad": 0, "dtype": "f32", "ids": "i64"},
        # The largest gradient pass.
        {"name": "exchange_grad_train", "op": "exchange_grad", "tokens": 8192, "width": 4096, "experts": 64, "topk": 8,
         "align": 16, "drop": 0.02, "pad": 0, "dtype": "bf16", "ids": "i64"},
        # The last sampled tokens of a serving batch looked up in a large table: latency.
        {"name": "embed_decode", "op": "embed", "tokens": 96, "vocab": 128000, "width": 4096, "scale": 64.0,
         "outside": 0.0, "dtype": "bf16", "ids": "i32"},
        # A training batch's tokens, a tenth of them padding.
        {"name": "embed_train", "op": "embed", "tokens": 65536, "vocab": 128000, "width": 2048, "scale": 1.0,
         "outside": 0.1, "dtype": "bf16", "ids": "i64"},
        # The gradient of a small table in 32 bits, odd token count and width.
        {"name": "embed_grad_small", "op": "embed_grad", "tokens": 2047, "vocab": 32768, "width": 515, "scale": 22.5,
         "outside": 0.05, "dtype": "f32", "ids": "i64"},
        # The gradient of a large table from a training batch, summed in 32 bits; frequent tokens own thousands of rows.
        {"name": "embed_grad_train", "op": "embed_grad", "tokens": 32768, "vocab": 128000, "width": 2048, "scale": 1.0,
         "outside": 0.1, "dtype": "bf16", "ids": "i64"},
        # One user's next token.
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 32768, "filters": "all", "masked": 0.0, "pad": 0,
         "dtype": "f32"},
        # A serving batch whose users ask for different filters, an odd vocabulary, some tokens forbidden.
        {"name": "sample_mixed", "op": "sample", "rows": 63, "vocab": 100003, "filters": "mixed", "masked": 0.3,
         "pad": 5, "dtype": "bf16"},
        # A large batch, top-k and top-p.
        {"name": "sample_batch", "op": "sample", "rows": 512, "vocab": 128000, "filters": "all", "masked": 0.0,
         "pad": 0, "dtype": "f32"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3 * 1024 else n


def _width(rng):
    w = _spread(rng, 64, 8192)
    n = w if rng.random() < 0.3 else max(64, w // 64 * 64)
    return n - 64 if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["exchange", "exchange_grad", "embed", "embed_grad", "sample", "sample"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    ids = rng.choice(["i32", "i64"])
    if op in ("exchange", "exchange_grad"):
        experts = _spread(rng, 2, 512)
        topk = min(experts, _spread(rng, 1, 10))
        width = _width(rng)
        align = rng.choice([1, 1, 8, 16, 64, 128])
        # no more bytes than the listed training cases
        most = min(16384, max(1, 256_000_000 // (topk * width * SIZE[dtype])))
        tokens = _spread(rng, 1, most)
        if min(experts, tokens * topk) * align * width * SIZE[dtype] > 128_000_000:
            align = 1
        return {"op": op, "tokens": tokens, "width": width, "experts": experts, "topk": topk, "align": align,
                "drop": rng.choice([0.0, 0.0, 0.1, 0.5]), "pad": rng.choice([0, 0, 8, 3]), "dtype": dtype, "ids": ids}
    if op in ("embed", "embed_grad"):
        width = _width(rng)
        vocab = _spread(rng, 256, min(262144, 1_000_000_000 // (4 * width)))
        tokens = _spread(rng, 1, min(65536, 268_000_000 // (SIZE[dtype] * width)))
        return {"op": op, "tokens": tokens, "vocab": vocab, "width": width, "scale": rng.choice([1.0, 8.0, 45.25]),
                "outside": rng.choice([0.0, 0.1, 0.4]), "dtype": dtype, "ids": ids}
    vocab = _spread(rng, 256, 262144)
    rows = _spread(rng, 1, min(512, 65_000_000 // vocab))
    return {"op": op, "rows": rows, "vocab": vocab, "filters": rng.choice(["mixed", "all", "none", "top_k", "top_p", "min_p"]),
            "masked": rng.choice([0.0, 0.0, 0.3, 0.99]), "pad": rng.choice([0, 0, 8, 3]), "dtype": dtype}


def _rand(gen, rows, width, dtype, pad=0):
    """Normal rows of a type; with `pad`, a slice of wider ones."""
    x = torch.randn(rows, width + pad, generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    return x[:, :width] if pad else x


def _capacity(c):
    """Rows that hold every token of any routing: each expert with a token may waste align - 1 rows."""
    pairs = c["tokens"] * c["topk"]
    return pairs + min(c["experts"], pairs) * (c["align"] - 1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[c["dtype"]]
    if c["op"] in ("exchange", "exchange_grad"):
        t, k, e = c["tokens"], c["topk"], c["experts"]
        # a router's scores: some experts are more popular than others
        scores = torch.randn(t, e, generator=gen, device="cuda") + 0.5 * torch.randn(e, generator=gen, device="cuda")
        top, ids = torch.topk(scores, k, dim=1)
        weights = torch.softmax(top, dim=1)
        if c["drop"]:
            ids = ids.masked_fill(torch.rand(t, k, generator=gen, device="cuda") < c["drop"], -1)
        s = {"case": c, "ids": ids.to(IDS[c["ids"]]).contiguous(), "weights": weights.contiguous(),
             "x": _rand(gen, t, c["width"], dtype, c["pad"]),  # the tokens' rows, or the gradient of their sums
             "ys": _rand(gen, _capacity(c), c["width"], dtype)}  # the experts' results
        if c["op"] == "exchange_grad":
            # the forward pass's plan, and the gradient that the experts hand back
            s["offsets"], s["counts"], s["slots"], s["pairs"] = _plan(s["ids"], e, c["align"], _capacity(c))
            s["dxs"] = _rand(gen, _capacity(c), c["width"], dtype)
        return s
    if c["op"] in ("embed", "embed_grad"):
        n, v = c["tokens"], c["vocab"]
        # token frequencies fall like 1 / rank
        u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(v + 1)) - 1).long().clamp_(0, v - 1)
        if c["outside"]:
            ids = ids.masked_fill(torch.rand(n, generator=gen, device="cuda") < c["outside"], -1)
        s = {"case": c, "ids": ids.to(IDS[c["ids"]])}
        s["rows"] = _rand(gen, v if c["op"] == "embed" else n, c["width"], dtype)
        return s
    b, v = c["rows"], c["vocab"]
    # a bulk of unlikely tokens and a few dozen that the context favours
    x = 2.0 * torch.randn(b, v + c["pad"], generator=gen, device="cuda")
    x = x[:, :v]
    at = torch.randint(v, (b, 40), generator=gen, device="cuda")
    x.scatter_add_(1, at, 12.0 * torch.rand(b, 40, generator=gen, device="cuda") ** 2)
    if c["masked"]:
        x.masked_fill_(torch.rand(b, v, generator=gen, device="cuda") < c["masked"], -math.inf)
    if c["pad"]:
        wide = torch.zeros(b, v + c["pad"], device="cuda", dtype=dtype)
        wide[:, :v] = x
        x = wide[:, :v]
    else:
        x = x.to(dtype)
    params = _filters(c)
    s = {"case": c, "logits": x, "uniform": torch.rand(b, v, generator=gen, device="cuda")}
    s.update({n: torch.tensor(p, device="cuda", dtype=torch.int32 if n == "top_k" else torch.float32)
              for n, p in params.items()})
    return s


# What the users of a mixed batch ask for: temperature, top-k, top-p, min-p (0, 1 and 0 switch a filter off).
MIXED = [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (0.8, 0, 0.9, 0.0),
         (1.0, 0, 1.0, 0.05), (0.9, 50, 0.95, 0.0), (0.6, 20, 0.8, 0.1), (1.2, 0, 0.95, 0.0)]
ALONE = {"all": (0.8, 50, 0.9, 0.02), "none": (1.0, 0, 1.0, 0.0), "top_k": (0.8, 100, 1.0, 0.0),
         "top_p": (1.0, 0, 0.95, 0.0), "min_p": (1.1, 0, 1.0, 0.03)}


def _filters(c):
    each = [MIXED[r % len(MIXED)] if c["filters"] == "mixed" else ALONE[c["filters"]] for r in range(c["rows"])]
    return dict(zip(("temperature", "top_k", "top_p", "min_p"), map(list, zip(*each))))


# ------------------------------------------------------------------ plain forms


def _plan(ids, experts, align, capacity):
    """Pairs (token, choice) sorted by expert, stably: block starts, counts, each pair's row, each row's pair."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    kept = (flat >= 0) & (flat < experts)
    key = torch.where(kept, flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    counts.index_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(counts, 0) - counts  # of each expert in the sorted pairs
    counts = counts[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum((counts + align - 1) // align * align, 0)
    sorted_key = key[order]
    row = offsets[sorted_key] + torch.arange(n, device=ids.device) - first[sorted_key]
    row = torch.where(sorted_key < experts, row, torch.full_like(row, -1))
    slots = torch.empty(n, dtype=torch.int64, device=ids.device)
    slots[order] = row
    pairs = torch.full((capacity + 1,), -1, dtype=torch.int64, device=ids.device)
    pairs[torch.where(row >= 0, row, torch.full_like(row, capacity))] = order
    return (offsets.int(), counts.int(), slots.int().reshape(ids.shape), pairs[:capacity].int())


def _gather(rows, index):
    """float32 rows[index], zeros where the index is -1."""
    got = rows[index.clamp(min=0).long()].float()
    return got.masked_fill_((index < 0).unsqueeze(-1), 0.0)


def _exchange(s):
    c = s["case"]
    offsets, counts, slots, pairs = _plan(s["ids"], c["experts"], c["align"], _capacity(c))
    token = torch.where(pairs >= 0, pairs // c["topk"], pairs)
    xs = _gather(s["x"], token).to(s["x"].dtype)
    out = (_gather(s["ys"], slots) * s["weights"].unsqueeze(-1)).sum(1).to(s["ys"].dtype)
    return {"rows": xs, "offsets": offsets, "counts": counts, "slots": slots, "pairs": pairs, "out": out}


def _exchange_grad(s):
    c = s["case"]
    token = torch.where(s["pairs"] >= 0, s["pairs"] // c["topk"], s["pairs"])
    w = s["weights"].reshape(-1)[s["pairs"].clamp(min=0).long()]
    d_rows = (_gather(s["x"], token) * w.unsqueeze(-1)).to(s["x"].dtype)
    d_weights = (_gather(s["ys"], s["slots"]) * s["x"].float().unsqueeze(1)).sum(-1)
    d_x = _gather(s["dxs"], s["slots"]).sum(1).to(s["dxs"].dtype)
    return {"d_rows": d_rows, "d_weights": d_weights, "d_x": d_x}


def _embed(s):
    return (_gather(s["rows"], s["ids"]) * s["case"]["scale"]).to(s["rows"].dtype)


def _embed_grad(s):
    c = s["case"]
    kept = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
    at = torch.where(kept, s["ids"], torch.full_like(s["ids"], c["vocab"])).long()
    d = torch.zeros(c["vocab"] + 1, c["width"], dtype=torch.float32, device=at.device)
    d.index_add_(0, at, s["rows"].float())
    return d[: c["vocab"]] * c["scale"]


def _sample(s):
    x = s["logits"].float()
    b, v = x.shape
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x).clamp(max=torch.finfo(torch.float32).max)
    m = x.amax(1, keepdim=True)
    greedy = ~(s["temperature"] > 0)
    t = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"]).unsqueeze(1)
    z = torch.where(x > -math.inf, (x - m) / t, x)
    w = torch.exp(z)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    rank = torch.arange(v, device=x.device)
    k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], v)).unsqueeze(1)
    ws = torch.where(rank < k, w.gather(1, order), torch.zeros_like(w))
    upto = torch.cumsum(ws, 1)
    before = torch.cat([torch.zeros_like(upto[:, :1]), upto[:, :-1]], 1)
    p = s["top_p"].unsqueeze(1)
    keep = (rank < k) & ((p >= 1) | (before < p * ws.sum(1, keepdim=True)) | (rank == 0)) & (ws >= s["min_p"].unsqueeze(1))
    keep = keep & (ws > 0)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    g = -torch.log(-torch.log(s["uniform"].clamp(U_LO, U_HI)))
    score = torch.where(kept, z + g, torch.full_like(z, -math.inf))
    token = torch.where(greedy, order[:, 0], score.argmax(1))
    mass = torch.where(kept, w, torch.zeros_like(w)).sum(1)
    logprob = z.gather(1, token.unsqueeze(1)).squeeze(1) - torch.log(mass)
    logprob = torch.where(greedy, torch.zeros_like(logprob), logprob)
    empty = m.squeeze(1) == -math.inf
    token = torch.where(empty, torch.full_like(token, -1), token)
    return {"tokens": token.int(), "logprobs": torch.where(empty, torch.full_like(logprob, -math.inf), logprob)}


PLAIN = {"exchange": _exchange, "exchange_grad": _exchange_grad, "embed": _embed, "embed_grad": _embed_grad,
         "sample": _sample}


# ------------------------------------------------------------------ the library's calls


def _own(s):
    from partition_pass_tile_gb300 import gc
    c = s["case"]
    if c["op"] == "exchange":
        rows, plan = gc.expert_dispatch(s["x"], s["ids"], c["experts"], align=c["align"])
        out = gc.expert_combine(s["ys"], plan.slots, s["weights"])
        return {"rows": rows, "offsets": plan.offsets, "counts": plan.counts, "slots": plan.slots,
                "pairs": plan.pairs, "out": out}
    if c["op"] == "exchange_grad":
        d_rows, d_weights = gc.expert_combine_grad(s["x"], s["ys"], s["slots"], s["pairs"], s["weights"])
        return {"d_rows": d_rows, "d_weights": d_weights, "d_x": gc.expert_dispatch_grad(s["dxs"], s["slots"])}
    if c["op"] == "embed":
        return gc.embedding(s["rows"], s["ids"], scale=c["scale"])
    if c["op"] == "embed_grad":
        return gc.embedding_grad(s["rows"], s["ids"], c["vocab"], scale=c["scale"], out_dtype=torch.float32)
    tokens, logprobs = gc.sample(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
                                 top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": tokens, "logprobs": logprobs}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    size = SIZE[c["dtype"]]
    if c["op"] in ("exchange", "exchange_grad"):
        t, k, h, r = c["tokens"], c["topk"], c["width"], _capacity(c)
        used = int(t * k * (1.0 - c["drop"]))  # pairs that reach an expert
        if c["op"] == "exchange":
            ids = t * k * (8 if c["ids"] == "i64" else 4)
            plan = 4 * (t * k + r + 2 * c["experts"] + 1)
            rows = size * h * (t + r + used + t)  # tokens in, rows out, results in, sums out
            return {"bytes": ids + plan + rows + 4 * t * k, "flops": 2 * used * h}
        rows = size * h * (t + used + r + used + t)  # gradient and results in, rows out; rows in, tokens out
        return {"bytes": rows + 4 * (2 * t * k + t * k + r), "flops": 4 * used * h}
    if c["op"] in ("embed", "embed_grad"):
        n, v, d = c["tokens"], c["vocab"], c["width"]
        used = n * (1.0 - c["outside"])
        ids = n * (8 if c["ids"] == "i64" else 4)
        if c["op"] == "embed":
            # distinct tokens: the sum over ids of the chance that it occurs, with frequencies like 1 / rank
            i = np.arange(1, v + 1)
            distinct = float(np.sum(-np.expm1(-used * np.log1p(1.0 / i) / math.log(v + 1))))
            return {"bytes": int(ids + size * d * (n + distinct)), "flops": n * d}
        return {"bytes": int(ids + size * d * used + 4 * d * v), "flops": int(used * d + v * d)}
    b, v = c["rows"], c["vocab"]
    each = _filters(c)
    # every logit once; the random numbers of rows without a filter, and of at most top-k tokens elsewhere
    free = sum(t > 0 and k == 0 and p >= 1 and q == 0 for t, k, p, q in zip(*each.values()))
    return {"bytes": b * v * size + 4 * v * free + 4 * sum(each["top_k"]) + 24 * b, "flops": 4 * b * v}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_plan(ids, experts, align, capacity):
    """The pairs placed one expert at a time."""
    flat = ids.reshape(-1).cpu().numpy()
    slots = np.full(flat.size, -1, dtype=np.int64)
    pairs = np.full(capacity, -1, dtype=np.int64)
    at = 0
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        slots[mine] = at + np.arange(mine.size)
        pairs[at:at + mine.size] = mine
        at += -(-mine.size // align) * align
    return slots.reshape(ids.shape), pairs


def _exact_sum(rows, slots, weights=None):
    """sum_j weights[:, j] * rows[slots[:, j]] in 64 bits, one choice after another."""
    out = torch.zeros(slots.shape[0], rows.shape[1], dtype=torch.float64, device=rows.device)
    for j in range(slots.shape[1]):
        at = torch.nonzero(slots[:, j] >= 0).squeeze(1)
        part = rows[slots[at, j].long()].double()
        out[at] += part if weights is None else part * weights[at, j].double().unsqueeze(1)
    return out


def _exact_sample(x, u, t, k, p, q):
    """One row: (token, log probability)."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    m = x.max()
    if m == -np.inf:
        return -1, -np.inf
    if not t > 0:
        return int(np.argmax(x)), 0.0
    likely = np.flatnonzero(x >= np.partition(x, x.size - k)[x.size - k]) if 0 < k < x.size else np.arange(x.size)
    order = likely[np.argsort(-x[likely], kind="stable")]
    order = order[: k if k > 0 else x.size]
    order = order[x[order] > -np.inf]
    z = (x[order] - m) / t
    w = np.exp(z)
    before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
    keep = (before < p * w.sum()) if p < 1 else np.ones(w.size, bool)
    keep[0] = True
    keep &= w >= q
    z, w, at = z[keep], w[keep], order[keep]
    score = z - np.log(-np.log(np.clip(u[at], U_LO, U_HI)))
    best = np.flatnonzero(score == score.max())
    best = best[np.argmin(at[best])]
    return int(at[best]), float(z[best] - np.log(w.sum()))


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "exchange":
        slots, _ = _exact_plan(s["ids"], c["experts"], c["align"], _capacity(c))
        out = _exact_sum(s["ys"], torch.from_numpy(slots).cuda(), s["weights"])
        # the rows are copies and the plan is whole numbers
        return {"rows": None, "offsets": None, "counts": None, "slots": None, "pairs": None, "out": out}
    if c["op"] == "exchange_grad":
        slots, pairs = _exact_plan(s["ids"], c["experts"], c["align"], _capacity(c))
        slots, pairs = torch.from_numpy(slots).cuda(), torch.from_numpy(pairs).cuda()
        d_rows = torch.zeros(pairs.numel(), c["width"], dtype=torch.float64, device="cuda")
        d_weights = torch.zeros(c["tokens"], c["topk"], dtype=torch.float64, device="cuda")
        g = s["x"].double()
        for j in range(c["topk"]):
            at = torch.nonzero(slots[:, j] >= 0).squeeze(1)
            to = slots[at, j]
            d_rows[to] = s["weights"][at, j].double().unsqueeze(1) * g[at]
            d_weights[at, j] = torch.linalg.vecdot(g[at], s["ys"][to].double())
        return {"d_rows": d_rows, "d_weights": d_weights, "d_x": _exact_sum(s["dxs"], slots)}
    if c["op"] == "embed":
        ids = s["ids"].long()
        out = torch.zeros(ids.numel(), c["width"], dtype=torch.float64, device="cuda")
        at = torch.nonzero((ids >= 0) & (ids < c["vocab"])).squeeze(1)
        out[at] = s["rows"][ids[at]].double() * c["scale"]
        return out
    if c["op"] == "embed_grad":
        out = torch.zeros(c["vocab"], c["width"], dtype=torch.float64, device="cuda")
        ids = s["ids"].long()
        at = torch.nonzero((ids >= 0) & (ids < c["vocab"])).squeeze(1)
        out.index_put_((ids[at],), c["scale"] * s["rows"][at].double(), accumulate=True)
        return out
    x = s["logits"].double().cpu().numpy()
    u = s["uniform"].double().cpu().numpy()
    if x.size > 80_000_000:
        return None
    got = [_exact_sample(x[r], u[r], *(np.float64(s[n][r].item()) if n != "top_k" else int(s[n][r].item())
                                       for n in ("temperature", "top_k", "top_p", "min_p"))) for r in range(c["rows"])]
    return {"tokens": np.array([t for t, _ in got], dtype=np.int32), "logprobs": np.array([p for _, p in got])}
