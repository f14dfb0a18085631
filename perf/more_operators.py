"""Cases of the operators around routing, drafting and the cache, with their plain forms.

* "route", "route_grad": every token's top-k experts with their weights, the
  experts' counts and mean probabilities and the balance loss, and the gradient
  of weights and loss with respect to the router's logits.
* "verify": drafted tokens accepted or replaced against the target's
  probabilities, from given uniform random numbers.
* "score": attention weights added to the scores of a cache's positions.
* "evict": the positions with the highest scores kept, in their order, with
  their rows of keys and values.

A case is a dict of plain values.  ``own`` selects what ``run`` does: the plain
form in elementary torch operations, or the library's entry points.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
MOST = torch.finfo(torch.float32).max

# Uniforms are clamped to [U_LO, U_HI].
U_LO, U_HI = 2.0 ** -25, 1.0 - 2.0 ** -24


def listed():
    return [
        # One step of a serving batch: latency.
        {"name": "route_decode", "op": "route", "tokens": 24, "experts": 64, "topk": 4, "normalize": True,
         "masked": 0.0, "forbidden": 0.0, "pad": 0, "dtype": "f32"},
        # A padded batch of prompts, an odd number of experts, some of them closed to some tokens, the logits a slice of
        # wider rows.
        {"name": "route_ragged", "op": "route", "tokens": 4099, "experts": 60, "topk": 6, "normalize": False,
         "masked": 0.2, "forbidden": 0.1, "pad": 5, "dtype": "f16"},
        # The largest routing pass: a training batch of many small experts, logits kept in 32 bits.
        {"name": "route_train", "op": "route", "tokens": 131072, "experts": 256, "topk": 8, "normalize": True,
         "masked": 0.0, "forbidden": 0.0, "pad": 0, "dtype": "f32"},
        # The gradient of a small layer.
        {"name": "route_grad_small", "op": "route_grad", "tokens": 1000, "experts": 8, "topk": 2, "normalize": True,
         "masked": 0.1, "forbidden": 0.0, "pad": 0, "dtype": "bf16"},
        # The gradient of the training batch.
        {"name": "route_grad_train", "op": "route_grad", "tokens": 131072, "experts": 256, "topk": 8, "normalize": True,
         "masked": 0.0, "forbidden": 0.0, "pad": 0, "dtype": "f32"},
        # One user's next tokens, drafted by a small model: latency.
        {"name": "verify_one", "op": "verify", "sequences": 1, "drafts": 4, "vocab": 32768, "drafted": "model",
         "agree": 0.8, "ragged": False, "greedy": 0.0, "pad": 0, "dtype": "f32"},
        # Drafts found in the text so far (no draft probabilities), of different lengths; a third of the users decode
        # greedily; an odd vocabulary.
        {"name": "verify_lookup", "op": "verify", "sequences": 29, "drafts": 7, "vocab": 100003, "drafted": "lookup",
         "agree": 0.6, "ragged": True, "greedy": 0.33, "pad": 5, "dtype": "bf16"},
        # A large serving batch.
        {"name": "verify_batch", "op": "verify", "sequences": 192, "drafts": 5, "vocab": 128000, "drafted": "model",
         "agree": 0.8, "ragged": False, "greedy": 0.0, "pad": 0, "dtype": "bf16"},
        # The weights of one decoded token of every sequence, odd lengths.
        {"name": "score_decode", "op": "score", "batch": 6, "heads": 8, "group": 4, "queries": 1, "length": 5003,
         "ragged": True, "decay": 1.0, "dtype": "f32"},
        # The last queries of long prompts.
        {"name": "score_prompt", "op": "score", "batch": 4, "heads": 8, "group": 4, "queries": 64, "length": 16384,
         "ragged": False, "decay": 0.99, "dtype": "bf16"},
        # Caches of different lengths that have outgrown their budget by a little, rows of odd width.
        {"name": "evict_ragged", "op": "evict", "batch": 3, "heads": 4, "length": 1411, "width": 72, "value_width": 57,
         "budget": 1024, "sinks": 4, "recent": 128, "ragged": True, "order": "head", "dtype": "f16"},
        # Long prompts cut down to what decoding keeps; the prompt's cache has its heads innermost.
        {"name": "evict_prompt", "op": "evict", "batch": 16, "heads": 8, "length": 32768, "width": 128,
         "value_width": 128, "budget": 2048, "sinks": 4, "recent": 512, "ragged": False, "order": "token",
         "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "verify", "verify", "score", "evict", "evict"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op in ("route", "route_grad"):
        experts = _spread(rng, 2, 1024)
        if rng.random() < 0.5:
            experts = max(2, experts // 8 * 8)
        return {"op": op, "tokens": _spread(rng, 1, min(131072, 33_554_432 // experts)), "experts": experts,
                "topk": min(experts, _spread(rng, 1, 12)), "normalize": rng.random() < 0.5,
                "masked": rng.choice([0.0, 0.0, 0.1, 0.4]), "forbidden": rng.choice([0.0, 0.0, 0.2]),
                "pad": rng.choice([0, 0, 8, 3]), "dtype": dtype}
    if op == "verify":
        vocab = _spread(rng, 256, 262144)
        drafts = _spread(rng, 1, 12)
        drafted = rng.choice(["model", "model", "lookup"])
        rows = 2 * drafts + 1 if drafted == "model" else drafts + 1
        return {"op": op, "sequences": _spread(rng, 1, min(256, max(1, 250_000_000 // (rows * vocab * SIZE[dtype])))),
                "drafts": drafts, "vocab": vocab, "drafted": drafted, "agree": rng.choice([0.3, 0.6, 0.8, 0.95]),
                "ragged": rng.random() < 0.3, "greedy": rng.choice([0.0, 0.0, 0.5, 1.0]),
                "pad": rng.choice([0, 0, 8, 3]), "dtype": dtype}
    if op == "score":
        heads, group = _spread(rng, 1, 16), rng.choice([1, 2, 4, 5, 8])
        length = _spread(rng, 16, 65536)
        queries = rng.choice([1, 1, _spread(rng, 2, 256)])
        heads = min(heads, max(1, 250_000_000 // (group * queries * length * SIZE[dtype])))
        most = max(1, 250_000_000 // (heads * group * queries * length * SIZE[dtype]))
        return {"op": op, "batch": _spread(rng, 1, min(64, most)), "heads": heads, "group": group, "queries": queries,
                "length": length, "ragged": rng.random() < 0.5, "decay": rng.choice([1.0, 1.0, 0.9]), "dtype": dtype}
    heads, length = _spread(rng, 1, 16), _spread(rng, 64, 65536)
    width = rng.choice([64, 80, 128, 128, 192, 256, _spread(rng, 32, 256)])
    value_width = rng.choice([width, width, 64, 33])
    budget = max(8, int(length * rng.choice([0.06, 0.25, 0.5, 0.9])))
    # a cache that is rewritten whole costs no more than the largest case's bytes
    row = (width + value_width) * SIZE[dtype]
    heads = min(heads, max(1, 400_000_000 // (budget * 2 * row + length * 4)))
    return {"op": "evict", "batch": _spread(rng, 1, min(32, max(1, 400_000_000 // (heads * (budget * 2 * row + length * 4))))),
            "heads": heads, "length": length, "width": width, "value_width": value_width, "budget": budget,
            "sinks": rng.choice([0, 4]), "recent": rng.choice([0, 1, budget // 8, budget // 2]),
            "ragged": rng.random() < 0.4, "order": rng.choice(["head", "token"]), "dtype": dtype}


def _slice(x, pad, dtype):
    """x in a type; with `pad`, a slice of rows that much wider."""
    if not pad:
        return x.to(dtype)
    wide = torch.zeros(*x.shape[:-1], x.shape[-1] + pad, device=x.device, dtype=dtype)
    wide[..., : x.shape[-1]] = x
    return wide[..., : x.shape[-1]]


def _temperatures(c):
    greedy = round(c["greedy"] * c["sequences"])
    return [0.0 if i < greedy else (0.7, 1.0, 0.9, 1.3)[i % 4] for i in range(c["sequences"])]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    if c["op"] in ("route", "route_grad"):
        t, e, k = c["tokens"], c["experts"], c["topk"]
        x = 1.5 * normal(t, e) + 0.5 * normal(e)  # some experts are more popular than others
        if c["forbidden"]:
            x.masked_fill_(uniform(t, e) < c["forbidden"], -math.inf)
        s = {"case": c, "logits": _slice(x, c["pad"], dtype), "mask": uniform(t) >= c["masked"] if c["masked"] else None}
        if c["op"] == "route_grad":
            ids, _, counts, _, _ = _routing(s["logits"], k, c["normalize"], s["mask"])
            s.update(ids=ids, counts=counts, dweights=normal(t, k), dloss=uniform(1) + 0.5)
        return s
    if c["op"] == "verify":
        b, k, v = c["sequences"], c["drafts"], c["vocab"]
        # a bulk of unlikely tokens and a few dozen that the context favours
        x = 2.0 * normal(b, k + 1, v)
        x.scatter_add_(2, torch.randint(v, (b, k + 1, 40), generator=gen, device="cuda"), 12.0 * uniform(b, k + 1, 40) ** 2)
        temperature = torch.tensor(_temperatures(c), device="cuda")
        t = torch.where(temperature > 0, temperature, 0.01).view(b, 1, 1)
        follows = uniform(b, k, 1) < c["agree"]  # positions at which the draft says what the target says, nearly
        if c["drafted"] == "model":
            d = torch.where(follows, x[:, :k] + 0.2 * normal(b, k, v), x[:, :k].roll(v // 3 + 1, 2))
            d = _slice(d, c["pad"], dtype)
        else:
            d = None
        x = _slice(x, c["pad"], dtype)
        # what the draft model drew, or for drafts without one what the target might draw, or anything
        like = x[:, :k] if d is None else d
        ids = torch.empty(b, k, dtype=torch.int64, device="cuda")
        for j in range(k):
            ids[:, j] = (like[:, j].float() / t[:, 0] - torch.log(-torch.log(uniform(b, v).clamp(U_LO, U_HI)))).argmax(1)
        if d is None:
            ids = torch.where(follows[..., 0], ids, torch.randint(v, (b, k), generator=gen, device="cuda"))
        if c["ragged"]:
            n = torch.randint(k + 1, (b, 1), generator=gen, device="cuda")
            ids = torch.where(torch.arange(k, device="cuda") < n, ids, -1)
        return {"case": c, "logits": x, "draft_logits": d, "drafts": ids.int(), "accept": uniform(b, k),
                "uniform": uniform(b, v), "temperature": temperature}
    b, h, n = c["batch"], c["heads"], c["length"]
    lengths = None
    if c["ragged"]:
        lengths = torch.randint(n // 2, n + 1, (b,), generator=gen, device="cuda").int()
        lengths[0] = n
    if c["op"] == "score":
        x = 1.5 * normal(b, h * c["group"], c["queries"], n)
        s = {"case": c, "weights": torch.softmax(x, 3).to(dtype), "scores": torch.exp(normal(b, h, n)), "lengths": lengths}
        return s
    # scores that were summed from weights of 8 bits: many small ones are equal
    scores = torch.exp(1.5 * normal(b, h, n)).bfloat16().float()
    shapes = [(b, n, h, w) if c["order"] == "token" else (b, h, n, w) for w in (c["width"], c["value_width"])]
    rows = [normal(*s).to(dtype) for s in shapes]
    if c["order"] == "token":
        rows = [r.transpose(1, 2) for r in rows]
    positions = torch.arange(n, device="cuda", dtype=torch.int32) + torch.randint(100, (b, h, 1), generator=gen, device="cuda").int()
    m = c["budget"]
    # the cache that decoding works in, empty
    kept = {"keys": torch.zeros(b, h, m, c["width"], dtype=dtype, device="cuda"),
            "values": torch.zeros(b, h, m, c["value_width"], dtype=dtype, device="cuda"),
            "scores": torch.zeros(b, h, m, device="cuda"),
            "positions": torch.zeros(b, h, m, dtype=torch.int32, device="cuda"),
            "lengths": torch.zeros(b, dtype=torch.int32, device="cuda")}
    return {"case": c, "keys": rows[0], "values": rows[1], "scores": scores, "positions": positions,
            "lengths": lengths, "kept": kept}


# ------------------------------------------------------------------ plain forms


def _clean(x):
    """float32 logits: NaN is a forbidden token, +inf the largest finite value."""
    x = x.float()
    return torch.where(torch.isnan(x), -math.inf, x).clamp(max=MOST)


def _routing(logits, topk, normalize, mask):
    """ids, weights, counts, load, loss."""
    x = _clean(logits)
    if mask is not None:
        x = x.masked_fill(~mask.unsqueeze(1), -math.inf)
    experts = x.shape[1]
    order = torch.sort(x, dim=1, descending=True, stable=True)
    chosen = order.values[:, :topk] > -math.inf
    ids = torch.where(chosen, order.indices[:, :topk], -1).int()
    p = _probabilities(x)
    w = torch.where(chosen, p.gather(1, order.indices[:, :topk]), 0.0)
    if normalize:
        w = torch.where(chosen, w / w.sum(1, keepdim=True), 0.0)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=x.device)
    counts.index_add_(0, torch.where(chosen, order.indices[:, :topk], experts).reshape(-1),
                      torch.ones(chosen.numel(), dtype=torch.int64, device=x.device))
    counts = counts[:experts]
    routed = chosen[:, 0].sum()
    load = p.sum(0, dtype=torch.float64) / routed.clamp(min=1)
    loss = experts * (counts.double() / counts.sum().clamp(min=1) * load).sum()
    return ids, w, torch.cat([counts, routed.view(1)]).int(), load.float(), loss.float().view(1)


def _probabilities(x):
    """Softmax of cleaned logits; zeros for a row without any."""
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    return w / torch.where(m > -math.inf, w.sum(-1, keepdim=True), 1.0)


def _route(s):
    c = s["case"]
    return dict(zip(("ids", "weights", "counts", "load", "loss"), _routing(s["logits"], c["topk"], c["normalize"], s["mask"])))


def _route_grad(s):
    c = s["case"]
    routed = s["ids"][:, :1] >= 0
    p = _probabilities(torch.where(routed, _clean(s["logits"]), -math.inf))
    counts = s["counts"][:-1].double()
    share = (counts / counts.sum().clamp(min=1)).float()
    a = s["dloss"] * c["experts"] / s["counts"][-1].clamp(min=1) * share  # gradient of a probability
    chosen = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    w = torch.where(chosen, p.gather(1, at), 0.0)
    g = torch.where(chosen, s["dweights"], 0.0)
    if c["normalize"]:
        w = torch.where(chosen, w / w.sum(1, keepdim=True), 0.0)
        g = w * (g - (w * g).sum(1, keepdim=True))
        d = p * (a - (p * a).sum(1, keepdim=True))
    else:
        d = p * (a - (p * a).sum(1, keepdim=True) - (w * g).sum(1, keepdim=True))
        g = w * g
    d.scatter_add_(1, at, g)
    return d.to(s["logits"].dtype)


def _weights(x, t):
    """Of cleaned logits: their exp((x - max) / t), its sum in 64 bits, and the scaled differences."""
    m = x.amax(-1, keepdim=True)
    z = (x - torch.where(m > -math.inf, m, 0.0)) / t
    w = torch.exp(z)
    return w, w.sum(-1, keepdim=True, dtype=torch.float64), z


def _first_largest(x):
    """Index of the largest value of each row, the lowest of equal ones."""
    i = torch.arange(x.shape[-1], device=x.device, dtype=torch.int32)
    return torch.where(x == x.amax(-1, keepdim=True), i, x.shape[-1]).amin(-1).long()


def _verify(s):
    x = _clean(s["logits"])
    b, k, v = x.shape[0], x.shape[1] - 1, x.shape[2]
    temperature = s["temperature"]
    greedy = ~(temperature > 0).unsqueeze(1)
    t = torch.where(greedy, 1.0, temperature.unsqueeze(1)).unsqueeze(2)
    w, total, z = _weights(x, t)
    first = _first_largest(x)
    drafts = s["drafts"].long()
    real = (drafts >= 0) & (drafts < v)
    at = drafts.clamp(0, v - 1).unsqueeze(2)
    p_at = (w[:, :k].gather(2, at) / total[:, :k])[..., 0]
    u = s["accept"].clamp(U_LO, U_HI).double()
    if s["draft_logits"] is None:
        q_at = torch.ones_like(p_at)
    else:
        y = _clean(s["draft_logits"])
        wq, totalq, _ = _weights(y, t)
        q_at = (wq.gather(2, at) / totalq)[..., 0]
    ok = real & torch.where(greedy, drafts == first[:, :k], u * q_at < p_at)
    a = torch.cumprod(ok.long(), 1).sum(1)  # accepted drafts
    row = torch.arange(b, device=x.device)
    p = (w[row, a] / total[row, a]).float()
    j = a.clamp(max=k - 1)
    rejected = (a < k) & real[row, j]
    if s["draft_logits"] is None:
        q = torch.zeros_like(p).scatter_(1, at[row, j], 2.0)
    else:
        q = (wq[row, j] / totalq[row, j]).float()
    r = torch.where(rejected.unsqueeze(1), (p - q).clamp(min=0.0), p)
    r = torch.where(r.amax(1, keepdim=True) > 0, r, p)
    score = r / -torch.log(s["uniform"].clamp(U_LO, U_HI))
    drawn = torch.where(greedy[:, 0], first[row, a], _first_largest(score))
    place = torch.arange(k + 1, device=x.device)
    tokens = torch.where(place < a.unsqueeze(1), torch.cat([drafts, drafts[:, :1]], 1), -1)
    tokens = torch.where(place == a.unsqueeze(1), drawn.unsqueeze(1), tokens)
    logprobs = (z.gather(2, tokens.clamp(min=0).unsqueeze(2)).double() - torch.log(total))[..., 0].float()
    logprobs = torch.where(greedy, 0.0, logprobs).masked_fill(tokens < 0, -math.inf)
    return {"tokens": tokens.int(), "accepted": a.int(), "logprobs": logprobs}


def _score(s):
    c = s["case"]
    b, h, n = s["scores"].shape
    w = s["weights"].float().reshape(b, h, c["group"] * c["queries"], n)
    out = s["scores"] * c["decay"] + w.sum(2)
    if s["lengths"] is not None:
        out = torch.where(torch.arange(n, device=out.device) < s["lengths"].view(b, 1, 1), out, 0.0)
    return out


def _evict(s):
    c = s["case"]
    b, h, n = s["scores"].shape
    m = min(c["budget"], n)
    dev = s["scores"].device
    length = torch.full((b,), n, device=dev) if s["lengths"] is None else s["lengths"].long()
    i = torch.arange(n, device=dev).view(1, 1, n)
    last = length.view(b, 1, 1)
    # always kept, in competition, behind the end
    kind = torch.where(i >= last, 2, torch.where((i < c["sinks"]) | (i >= last - c["recent"]), 0, 1)).expand(b, h, n)
    value = torch.where(torch.isnan(s["scores"]), -math.inf, s["scores"])
    order = torch.sort(value, dim=2, descending=True, stable=True).indices
    order = order.gather(2, torch.sort(kind.gather(2, order), dim=2, stable=True).indices)[..., :m]
    new = length.clamp(max=c["budget"])
    there = torch.arange(m, device=dev) < new.view(b, 1, 1)
    at = torch.sort(torch.where(there, order, n), dim=2).values
    there = at < n
    at = at.clamp(max=n - 1)
    kept = s["kept"]
    for name in ("keys", "values"):
        rows = s[name].gather(2, at.unsqueeze(3).expand(b, h, m, s[name].shape[3]))
        kept[name][:, :, :m] = torch.where(there.unsqueeze(3), rows, kept[name][:, :, :m])
    kept["scores"].zero_()
    kept["scores"][:, :, :m] = torch.where(there, s["scores"].gather(2, at), 0.0)
    kept["positions"].fill_(-1)
    kept["positions"][:, :, :m] = torch.where(there, s["positions"].gather(2, at), -1)
    kept["lengths"].copy_(new)
    return kept


PLAIN = {"route": _route, "route_grad": _route_grad, "verify": _verify, "score": _score, "evict": _evict}


# ------------------------------------------------------------------ the library's calls


def _own(s):
    from partition_pass_tile_gb300 import gc
    c = s["case"]
    if c["op"] == "route":
        r = gc.expert_route(s["logits"], c["topk"], normalize=c["normalize"], mask=s["mask"])
        return {"ids": r.ids, "weights": r.weights, "counts": r.counts, "load": r.load, "loss": r.loss}
    if c["op"] == "route_grad":
        return gc.expert_route_grad(s["logits"], s["ids"], s["counts"], dweights=s["dweights"], dloss=s["dloss"],
                                    normalize=c["normalize"])
    if c["op"] == "verify":
        tokens, accepted, logprobs = gc.sample_verify(s["logits"], s["drafts"], s["accept"], s["uniform"],
                                                      draft_logits=s["draft_logits"], temperature=s["temperature"])
        return {"tokens": tokens, "accepted": accepted, "logprobs": logprobs}
    if c["op"] == "score":
        return gc.cache_score(s["weights"], s["scores"], decay=c["decay"], lengths=s["lengths"])
    kept = gc.cache_evict(s["keys"], s["values"], s["scores"], c["budget"], sinks=c["sinks"], recent=c["recent"],
                          positions=s["positions"], lengths=s["lengths"], out=gc.KeptCache(**s["kept"]))
    return kept._asdict()


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    size = SIZE[c["dtype"]]
    if c["op"] in ("route", "route_grad"):
        t, e, k = c["tokens"], c["experts"], c["topk"]
        row = t * k * 8 + (t if c["masked"] else 0)  # ids and weights, or the weights' gradient
        if c["op"] == "route":
            return {"bytes": t * e * size + row + 8 * e, "flops": 5 * t * e}
        return {"bytes": 2 * t * e * size + row + 4 * e, "flops": 8 * t * e}
    if c["op"] == "verify":
        # Rows up to the first rejection.  Of the positions at which the draft follows the target, about 95 in 100 are
        # accepted where a model drew the draft, 42 in 100 where the target's own draw stands for it, all if greedy.
        b, k, v = c["sequences"], c["drafts"], c["vocab"]
        sampled = sum(t > 0 for t in _temperatures(c))
        model = c["drafted"] == "model"
        target = drafted = 0.0
        for each, rate, reads in ((sampled, 0.95 if model else 0.42, model), (b - sampled, 0.95 if model else 1.0, False)):
            for n in range(k + 1) if c["ragged"] else [k]:
                share = each / (k + 1 if c["ragged"] else 1)
                passed = [(rate * c["agree"]) ** j for j in range(n + 1)]
                target += share * sum(passed)
                drafted += share * sum(passed[:-1]) * reads
        rows = target + drafted
        return {"bytes": int(rows * v * size + 4 * v * sampled + b * k * 16), "flops": int(4 * rows * v)}
    mean = 0.75 if c["ragged"] else 1.0
    if c["op"] == "score":
        n = c["batch"] * c["heads"] * c["length"]
        rows = c["group"] * c["queries"]
        return {"bytes": int(n * mean * (rows * size + 4) + 4 * n), "flops": int(n * mean * rows)}
    each = c["batch"] * c["heads"]
    n = c["length"] * mean
    m = min(n, c["budget"])
    return {"bytes": int(each * (4 * n + m * (2 * (c["width"] + c["value_width"]) * size + 12))), "flops": int(each * n)}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_softmax(x):
    """Rows of numpy logits -> probabilities, zeros for a row without any."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, MOST))
    m = x.max(-1, keepdims=True)
    w = np.exp(x - np.where(m > -np.inf, m, 0.0))
    return np.where(m > -np.inf, w / w.sum(-1, keepdims=True), 0.0)


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    t, e, k = c["tokens"], c["experts"], c["topk"]
    if s["mask"] is not None:
        x[~s["mask"].cpu().numpy()] = -np.inf
    p = _exact_softmax(x)
    rank = np.argsort(-x, axis=1, kind="stable")[:, :k]
    live = np.take_along_axis(x, rank, 1) > -np.inf
    w = np.take_along_axis(p, rank, 1) * live
    if c["normalize"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    counts = np.bincount(rank[live], minlength=e)
    routed = max(1, int(live[:, 0].sum()))
    load = p.sum(0) / routed
    return rank, live, w, p, counts, routed, load, e * float(counts @ load) / max(1, int(counts.sum()))


def _exact_verify(s, b):
    """One sequence: its log probabilities."""
    c = s["case"]
    k = c["drafts"]
    t = float(np.float32(_temperatures(c)[b]))
    out = np.full(k + 1, -np.inf)
    drafts = s["drafts"][b].tolist()

    def row(name, j):
        y = s[name][b, j].double()
        y = torch.where(torch.isnan(y), -math.inf, y).clamp(max=MOST)
        return y if t <= 0 else torch.log_softmax(y / t, 0)

    for j in range(k + 1):
        lp = row("logits", j)
        d = drafts[j] if j < k else -1
        if t <= 0:
            out[j] = 0.0
            if d == int((lp == lp.max()).nonzero()[0]):
                continue
            return out
        lq = None
        if d >= 0:
            if s["draft_logits"] is not None:
                lq = row("draft_logits", j)
            u = min(max(float(s["accept"][b, j]), U_LO), U_HI)
            if math.log(u) + (0.0 if lq is None else float(lq[d])) < float(lp[d]):
                out[j] = float(lp[d])
                continue
        r = lp.exp()
        if d >= 0:
            if lq is None:
                r[d] = 0.0
            else:
                r = (r - lq.exp()).clamp(min=0.0)
        r = r / -torch.log(s["uniform"][b].double().clamp(U_LO, U_HI))
        out[j] = float(lp[int(r.argmax())])
        return out
    return out


def _exact_evict(s):
    c = s["case"]
    b, h, n = s["scores"].shape
    scores, positions = s["scores"].cpu().numpy(), s["positions"].cpu().numpy()
    lengths = [n] * b if s["lengths"] is None else s["lengths"].tolist()
    m = c["budget"]
    out = {"scores": np.zeros((b, h, m), np.float32), "positions": None, "lengths": None}
    for name in ("keys", "values"):
        out[name] = torch.zeros(b, h, m, s[name].shape[3], dtype=s[name].dtype, device="cuda")
    for x in range(b):
        for y in range(h):
            size = lengths[x]
            if size <= m:
                at = np.arange(size)
            else:
                middle = np.arange(c["sinks"], size - c["recent"])
                best = middle[np.lexsort((middle, -scores[x, y, middle]))[: m - c["sinks"] - c["recent"]]]
                at = np.sort(np.concatenate([np.arange(c["sinks"]), best, np.arange(size - c["recent"], size)]))
            out["scores"][x, y, : at.size] = scores[x, y, at]
            rows = torch.from_numpy(at).cuda()
            for name in ("keys", "values"):
                out[name][x, y, : at.size] = s[name][x, y, rows]
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "route":
        _, _, w, _, _, _, load, loss = _exact_route(s)
        return {"ids": None, "weights": w, "counts": None, "load": load, "loss": np.array([loss])}
    if c["op"] == "route_grad":
        rank, live, w, p, counts, routed, _, _ = _exact_route(s)
        g = s["dweights"].double().cpu().numpy() * live
        a = float(s["dloss"]) * c["experts"] / routed * counts / max(1, counts.sum())
        d = p * (a - p @ a.reshape(-1, 1))
        inner = (w * g).sum(1, keepdims=True)
        every = np.arange(c["tokens"])
        for j in range(c["topk"]):
            d[every, rank[:, j]] += w[:, j] * (g[:, j] - (inner[:, 0] if c["normalize"] else 0.0))
        return d if c["normalize"] else d - p * inner
    if c["op"] == "verify":
        return {"tokens": None, "accepted": None, "logprobs": np.stack([_exact_verify(s, b) for b in range(c["sequences"])])}
    if c["op"] == "score":
        b, h, n = s["scores"].shape
        out = s["scores"].double() * float(np.float32(c["decay"]))
        for g in range(c["group"]):
            for q in range(c["queries"]):
                out += s["weights"][:, g::c["group"], q].double()
        if s["lengths"] is not None:
            for x, size in enumerate(s["lengths"].tolist()):
                out[x, :, size:] = 0.0
        return out
    return _exact_evict(s)
