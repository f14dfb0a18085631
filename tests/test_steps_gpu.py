"""Runs of the row operators one after another, as a model calls them."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import more_rows_ref as ref
from partition_pass_tile_gb300 import gc

pytestmark = pytest.mark.gpu


def test_training_step_of_experts():
    # route -> dispatch -> a matrix per expert -> combine, and back, against
    # autograd in 64 bits.  Each gradient is a few sums of at most 64 terms
    # and 32 products: 1e-4 of the largest magnitude is a hundred times the
    # sum of their roundings (300 * 2^-24 = 2e-5).
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens, width, experts, topk, align = 200, 32, 12, 3, 8

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    h, router, expert, d_out = normal(tokens, width), normal(width, experts), normal(experts, width, width) / 6, normal(tokens, width)
    mask = torch.rand(tokens, generator=g, device="cuda") > 0.1
    coefficient = torch.full((1,), 0.5, device="cuda")

    scores = h @ router
    r = gc.expert_route(scores, topk, normalize=False, mask=mask)
    rows, plan = gc.expert_dispatch(h, r.ids, experts, align=align)
    assert torch.equal(plan.counts, r.counts[:experts])
    at = plan.offsets.tolist()
    y = torch.zeros_like(rows)
    for e in range(experts):
        y[at[e]:at[e + 1]] = rows[at[e]:at[e + 1]] @ expert[e]
    out = gc.expert_combine(y, plan.slots, r.weights)
    d_y, d_weights = gc.expert_combine_grad(d_out, y, plan.slots, plan.pairs, r.weights)
    d_rows = torch.zeros_like(rows)
    for e in range(experts):
        d_rows[at[e]:at[e + 1]] = d_y[at[e]:at[e + 1]] @ expert[e].T
    d_scores = gc.expert_route_grad(scores, r.ids, r.counts, dweights=d_weights, dloss=coefficient, normalize=False)
    d_h = gc.expert_dispatch_grad(d_rows, plan.slots) + d_scores @ router.T
    d_router = h.T @ d_scores

    h64, r64 = h.double().requires_grad_(), router.double().requires_grad_()
    p = torch.softmax(h64 @ r64, 1) * mask.unsqueeze(1)
    ids = r.ids.long().clamp(min=0)
    w = p.gather(1, ids) * (r.ids >= 0)
    each = torch.einsum("tw,ewv->tev", h64, expert.double())
    out64 = (w.unsqueeze(2) * each.gather(1, ids.unsqueeze(2).expand(-1, -1, width))).sum(1)
    counts = r.counts[:experts].double()
    loss64 = experts * (counts / counts.sum() * p.sum(0) / mask.sum()).sum()
    ((out64 * d_out.double()).sum() + 0.5 * loss64).backward()
    for got, want in ((out, out64), (r.loss, loss64.view(1)), (d_h, h64.grad), (d_router, r64.grad)):
        want = want.detach()
        assert float((got.double() - want).abs().max()) <= 1e-4 * float(want.abs().max())


def test_decoding_steps_with_a_bounded_cache():
    # Two sequences decode into caches of 24 positions: the weights of each new
    # token's attention are added to the scores, and a cache that is full is cut
    # down to 16, beside a cache kept in numpy.
    rng = np.random.default_rng(9)
    batch, heads, group, room, budget, sinks, recent, width = 2, 2, 3, 24, 16, 2, 4, 8
    keys, values = (torch.zeros(batch, heads, room, width, device="cuda") for _ in range(2))
    scores = torch.zeros(batch, heads, room, device="cuda")
    positions = torch.full((batch, heads, room), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
    text = {}                                                      # (b, position) -> row
    known = [[[] for _ in range(heads)] for _ in range(batch)]   # positions kept, by the plain form
    total = [[np.zeros(0) for _ in range(heads)] for _ in range(batch)]
    written = [0, 0]
    evictions = 0
    for step in range(60):
        # a sequence takes up to three tokens at a step, as verification lets it
        take = [int(rng.integers(1, 4)) for _ in range(batch)]
        for b in range(batch):
            n = int(lengths[b])
            for k in range(take[b]):
                row = torch.from_numpy(rng.standard_normal(width).astype(np.float32)).cuda()
                text[b, written[b]] = row
                for h in range(heads):
                    keys[b, h, n + k], values[b, h, n + k] = row, row + h
                    positions[b, h, n + k] = written[b]
                    known[b][h].append(written[b])
                    total[b][h] = np.append(total[b][h], 0.0)
                written[b] += 1
        lengths += torch.tensor(take, dtype=torch.int32, device="cuda")
        # three queries at most, the others' weights are padding
        x = 2 * torch.randn(batch, heads * group, 3, room, device="cuda")
        x.masked_fill_(torch.arange(room, device="cuda") >= lengths.view(-1, 1, 1, 1), -np.inf)
        w = torch.softmax(x, 3)
        queries = torch.tensor(take, dtype=torch.int32, device="cuda")
        for b in range(batch):
            w[b, :, take[b]:] = float("nan")
        gc.cache_score(w, scores, decay=0.95, lengths=lengths, queries=queries, out=scores)
        for b in range(batch):
            for h in range(heads):
                n = len(known[b][h])
                add = w[b, h * group:(h + 1) * group, :take[b], :n].double().sum((0, 1)).cpu().numpy()
                total[b][h] = float(np.float32(0.95)) * total[b][h] + add
                got = scores[b, h].double().cpu().numpy()
                # the roundings of at most 60 steps of 10 additions
                assert np.all(np.abs(got[:n] - total[b][h]) <= 660 * 2.0 ** -24 * total[b][h]) and not got[n:].any()
        if int(lengths.max()) <= room - 3:
            continue
        evictions += 1
        before = scores.cpu().numpy()
        kept = gc.cache_evict(keys, values, scores, budget, sinks=sinks, recent=recent, positions=positions, lengths=lengths)
        for b in range(batch):
            for h in range(heads):
                at = ref.kept(before[b, h], len(known[b][h]), budget, sinks, recent)
                known[b][h] = [known[b][h][i] for i in at]
                total[b][h] = total[b][h][at]
        for mine, got in ((keys, kept.keys), (values, kept.values), (scores, kept.scores), (positions, kept.positions)):
            mine[:, :, :budget] = got
        scores[:, :, budget:] = 0
        lengths = kept.lengths
        for b in range(batch):
            for h in range(heads):
                n = len(known[b][h])
                assert positions[b, h, :n].tolist() == known[b][h] and int(lengths[b]) == n
                want = torch.stack([text[b, q] for q in known[b][h]])
                assert torch.equal(keys[b, h, :n], want) and torch.equal(values[b, h, :n], want + h)
    assert evictions >= 3


def test_verified_tokens_feed_the_next_step():
    # sample -> verify -> the next drafts' input, on one stream without the host in between, captured and replayed
    g = torch.Generator(device="cuda").manual_seed(1)
    n, k, vocab, width = 6, 3, 900, 48
    table = torch.randn(vocab, width, generator=g, device="cuda")
    ids = torch.randint(vocab, (n,), generator=g, device="cuda")
    u, accept = torch.rand(k + 1, n, vocab, generator=g, device="cuda"), torch.rand(n, k, generator=g, device="cuda")

    def step():
        text, guesses = [ids.int()], []
        for j in range(k):
            guesses.append(gc.embedding(table, text[-1], scale=0.1) @ table.T)
            text.append(gc.sample(guesses[-1], u[j])[0])
        h = gc.embedding(table, torch.stack(text, 1).reshape(-1), scale=0.11)
        logits = (h @ table.T).view(n, k + 1, vocab)
        return text, torch.stack(guesses, 1), logits, gc.sample_verify(logits, torch.stack(text[1:], 1), accept, u[k],
                                                                       draft_logits=torch.stack(guesses, 1))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        text, guesses, logits, (tokens, accepted, _) = step()
    compared = 0
    for _ in range(3):
        ids.copy_(torch.randint(vocab, (n,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        drafts = torch.stack(text[1:], 1).cpu().numpy()
        for b in range(n):
            want, a, _, sure = ref.verify(logits[b].double().cpu().numpy(), drafts[b], accept[b].cpu().numpy(),
                                          u[k, b].cpu().numpy(), guesses[b].double().cpu().numpy(), 1.0)
            if sure:
                compared += 1
                assert tokens[b].tolist() == want.tolist() and int(accepted[b]) == a
    assert compared >= 15


def test_example_drafts():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "language_model_step.py")
    spec = importlib.util.spec_from_file_location("language_model_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Model(vocab=300, width=64, experts=40, topk=4, align=8)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(300, (90,), generator=g, device="cuda")
    loss, d_logits, saved = model.loss(ids, (ids * 7 + 3) % 300)
    grads = model.backward(d_logits, saved)
    # along the router's gradient, against a central difference, as the example's other test does it
    d = grads["router"] / grads["router"].norm()
    ends = []
    for h in (1e-3, -1e-3):
        model.params["router"] += h * d
        ends.append(model.loss(ids, (ids * 7 + 3) % 300)[0].double().item())
        model.params["router"] -= h * d
    assert abs((ends[0] - ends[1]) / 2e-3 - grads["router"].norm().item()) <= 0.02 * grads["router"].norm().item() + 2e-3
    tokens, accepted = model.drafted(ids, g)
    assert tokens.shape == (90, 4) and accepted.shape == (90,)
    for row, a in zip(tokens.tolist(), accepted.tolist()):
        assert 0 <= a <= 3 and all(0 <= t < 300 for t in row[:a + 1]) and row[a + 1:] == [-1] * (3 - a)


def test_calls_on_two_streams_at_once():
    # every operator twice, on streams of their own, with nothing waited for in between
    g = torch.Generator(device="cuda").manual_seed(4)
    scores = torch.randn(5000, 64, generator=g, device="cuda")
    logits, drafted = (torch.randn(40, n, 9000, generator=g, device="cuda") for n in (4, 3))
    drafts = drafted.argmax(2).int()
    accept, uniform = torch.rand(40, 3, generator=g, device="cuda"), torch.rand(40, 9000, generator=g, device="cuda")
    w, keys = torch.rand(3, 8, 4, 6000, generator=g, device="cuda"), torch.randn(3, 2, 6000, 32, generator=g, device="cuda")

    def all_of(stream=None):
        r = gc.expert_route(scores, 4, stream=stream)
        d = gc.expert_route_grad(scores, r.ids, r.counts, dweights=r.weights, dloss=r.loss, stream=stream)
        v = gc.sample_verify(logits, drafts, accept, uniform, draft_logits=drafted, stream=stream)
        s = gc.cache_score(w, None, heads=2, stream=stream)
        k = gc.cache_evict(keys, None, s, 900, 4, 50, stream=stream)
        return [*r, d, *v, s, *(t for t in k if t is not None)]
    want = all_of()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [all_of(s) for s in streams]
        torch.cuda.synchronize()
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(want, one))
