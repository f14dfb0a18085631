"""Scores of a cache and eviction on the GPU against plain 64-bit forms (more_rows_ref.py).

A score is a float32 sum of n terms: off by at most (n + 2) 2^-24 of the sum of
their magnitudes (the decay's product and the last addition are one rounding).
Kept rows, scores and positions are copies."""

import numpy as np
import pytest
import torch

import more_rows_ref as ref
from partition_pass_tile_gb300 import gc

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def lengths_of(rng, batch, length, how):
    if how is None:
        return None, None
    n = {"some": lambda: rng.integers(0, length + 1, batch), "ends": lambda: rng.choice([0, 1, length], batch),
         "outside": lambda: rng.choice([-5, length + 7, length, 2 ** 31 - 1, -2 ** 31], batch)}[how]()
    return torch.from_numpy(n.astype(np.int32)).cuda(), n


# batch, heads, group, queries, length, dtype, lengths, counted, decay, scores, pad
SCORE = [
    (1, 1, 1, 1, 1, "f32", None, None, 1.0, True, 0),
    (1, 2, 4, 1, 33, "bf16", None, None, 1.0, True, 0),
    (3, 2, 5, 1, 1003, "f32", "some", None, 0.9, True, 0),
    (2, 3, 1, 7, 256, "f16", "ends", "some", 0.5, True, 8),
    (2, 1, 8, 16, 4096, "bf16", None, None, 1.0, False, 0),
    (4, 2, 2, 33, 515, "bf16", "outside", "outside", 1.0, True, 5),
    (1, 1, 3, 300, 77, "f32", None, None, 0.99, False, 1),
    (2, 2, 2, 0, 40, "f16", "some", None, 0.5, True, 0),
    (5, 4, 1, 2, 8, "bf16", "ends", "ends", 1.0, True, 0),
    (1, 2, 2, 1000, 2000, "bf16", "some", "some", 1.0, True, 0),
]


@pytest.mark.parametrize("batch,heads,group,queries,length,dtype,lengths,counted,decay,with_scores,pad", SCORE)
def test_score(batch, heads, group, queries, length, dtype, lengths, counted, decay, with_scores, pad):
    rng = np.random.default_rng(length * 7 + queries)
    w = torch.from_numpy(rng.random((batch, heads * group, queries, length + pad)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    w = w[..., pad // 2:pad // 2 + length]
    s64 = rng.random((batch, heads, length)).astype(np.float32) if with_scores else None
    s = torch.from_numpy(s64).cuda() if with_scores else None
    n, n_host = lengths_of(rng, batch, length, lengths)
    m, m_host = lengths_of(rng, batch, max(queries, 1), counted)
    want, size = ref.score(w.double().cpu().numpy(), s64, heads, decay, n_host, m_host)
    got = gc.cache_score(w, s, heads=heads, decay=decay, lengths=n, queries=m)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= (group * queries + 2) * 2.0 ** -24 * size)
    if with_scores:
        # in place, within a longer buffer whose rest stays
        wide = torch.full((batch, heads, length + 3), 7.0, device="cuda")
        wide[..., 1:1 + length] = s
        gc.cache_score(w, wide[..., 1:1 + length], decay=decay, lengths=n, queries=m, out=wide[..., 1:1 + length])
        assert torch.equal(wide[..., 1:1 + length], got)
        assert bool((wide[..., 0] == 7).all()) and bool((wide[..., 1 + length:] == 7).all())


def test_masked_weights_do_not_leak():
    w = torch.full((2, 4, 5, 64), float("nan"), device="cuda")
    w[0, :, :3, :20] = 0.25
    w[1, :, :1, :64] = 0.5
    s = torch.full((2, 2, 64), float("inf"), device="cuda")
    s[0, :, :20] = 1.0
    s[1] = 2.0
    out = gc.cache_score(w, s, lengths=torch.tensor([20, 64], dtype=torch.int32, device="cuda"),
                         queries=torch.tensor([3, 1], dtype=torch.int32, device="cuda"))
    assert bool((out[0, :, :20] == 2.5).all()) and not out[0, :, 20:].any() and bool((out[1] == 3.0).all())


def test_score_of_broadcast_and_transposed_weights():
    # heads innermost but one, and one row of weights for every query
    w = torch.rand(2, 6, 4, 100, device="cuda")
    s = torch.zeros(2, 3, 100, device="cuda")
    turned = w.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(gc.cache_score(w, s), gc.cache_score(turned, s))
    same = w[:, :, :1].expand(2, 6, 4, 100)
    assert torch.equal(gc.cache_score(same, s), gc.cache_score(same.contiguous(), s))


def cache_of(rng, batch, heads, length, width, dtype, order, pad=0):
    shape = (batch, length, heads, width + pad) if order == "token" else (batch, heads, length, width + pad)
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DTYPES[dtype]).cuda()[..., :width]
    return t.transpose(1, 2) if order == "token" else t


def scores_of(rng, batch, heads, length, how):
    s = np.exp(2 * rng.standard_normal((batch, heads, length))).astype(np.float32)
    if how == "equal":
        s[:] = 0.5
    elif how == "few":
        s = rng.integers(0, 4, s.shape).astype(np.float32) * np.where(rng.random(s.shape) < 0.5, -1, 1).astype(np.float32)
    elif how == "wild":
        s = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38, 1.0], np.float32), s.shape)
    elif how == "near":
        s = (1 + rng.integers(0, 3, s.shape) * 2.0 ** -23).astype(np.float32)
    return s


# batch, heads, length, width, value width, budget, sinks, recent, dtype, lengths, order, scores, pad
EVICT = [
    (1, 1, 1, 1, None, 1, 0, 0, "f32", None, "head", "any", 0),
    (1, 1, 2, 8, 8, 1, 0, 0, "bf16", None, "head", "any", 0),
    (1, 2, 100, 64, 64, 10, 2, 3, "bf16", None, "head", "any", 0),
    (2, 3, 100, 33, 7, 40, 40, 0, "f16", "some", "token", "any", 1),
    (2, 3, 100, 33, None, 40, 0, 40, "f32", "ends", "token", "few", 0),
    (3, 2, 513, 80, 64, 200, 4, 100, "f16", "some", "head", "equal", 0),
    (2, 4, 1411, 72, 57, 1024, 4, 128, "f16", "some", "head", "few", 3),
    (4, 1, 2048, 128, 128, 2047, 0, 1, "bf16", "outside", "token", "near", 0),
    (1, 3, 5000, 16, 16, 1, 0, 0, "bf16", None, "head", "any", 0),
    (1, 3, 5000, 16, 16, 1, 1, 0, "bf16", None, "head", "any", 0),
    (1, 2, 20000, 256, 192, 3000, 4, 500, "f32", None, "head", "any", 0),
    (2, 1, 9000, 24, 24, 4000, 3, 10, "bf16", None, "token", "wild", 0),
    (1, 1, 70001, 8, 8, 60000, 5, 7, "f16", None, "head", "few", 0),
    (40, 16, 300, 32, 32, 100, 4, 10, "bf16", "some", "token", "any", 0),
    (2, 2, 64, 128, 128, 500, 4, 10, "bf16", "some", "head", "any", 0),
    # a CTA's share of more positions than it holds at a time, one CTA to a head, and 32 positions to a thread
    (1, 1, 300001, 4, None, 200, 4, 10, "bf16", None, "head", "any", 0),
    (1, 2, 270000, 4, None, 150000, 4, 10, "bf16", None, "head", "few", 0),
    (8, 20, 9000, 8, None, 700, 2, 64, "bf16", "some", "token", "any", 0),
    (1, 3, 40000, 8, 16, 39000, 0, 0, "bf16", None, "token", "wild", 0),
]


@pytest.mark.parametrize("batch,heads,length,width,vwidth,budget,sinks,recent,dtype,lengths,order,how,pad", EVICT)
def test_evict(batch, heads, length, width, vwidth, budget, sinks, recent, dtype, lengths, order, how, pad):
    rng = np.random.default_rng(length * 3 + budget)
    k = cache_of(rng, batch, heads, length, width, dtype, order, pad)
    v = None if vwidth is None else cache_of(rng, batch, heads, length, vwidth, dtype, order, pad)
    s64 = scores_of(rng, batch, heads, length, how)
    s = torch.from_numpy(s64).cuda()
    positions = torch.from_numpy(rng.integers(0, 10 ** 6, s64.shape).astype(np.int32)).cuda()
    n, n_host = lengths_of(rng, batch, length, lengths)
    n_host = [length] * batch if n_host is None else [min(max(int(x), 0), length) for x in n_host]
    mine = gc.KeptCache(torch.full((batch, heads, budget, width + 4), 7.0, dtype=DTYPES[dtype], device="cuda")[..., 2:2 + width],
                        None if v is None else torch.full((batch, budget, heads, vwidth), 7.0, dtype=DTYPES[dtype], device="cuda").transpose(1, 2),
                        torch.full((batch, heads, budget), 7.0, device="cuda"),
                        torch.full((batch, heads, budget), 7, dtype=torch.int32, device="cuda"),
                        torch.full((batch,), 7, dtype=torch.int32, device="cuda"))
    got = gc.cache_evict(k, v, s, budget, sinks, recent, positions=positions, lengths=n, out=mine)
    new = gc.cache_evict(k, v, s, budget, sinks, recent, lengths=n)
    assert got.lengths.tolist() == [min(x, budget) for x in n_host] and torch.equal(new.lengths, got.lengths)
    where = np.full((batch, heads, budget), length, np.int64)
    for b in range(batch):
        for h in range(heads):
            at = ref.kept(s64[b, h], n_host[b], budget, sinks, recent)
            where[b, h, :at.size] = at
    there = torch.from_numpy(where < length).cuda()
    at = torch.from_numpy(np.minimum(where, length - 1)).cuda()
    assert torch.equal(got.positions, torch.where(there, positions.gather(2, at), -1))
    assert torch.equal(new.positions, torch.where(there, at, -1).int())
    kept = torch.where(there, s.gather(2, at), 0.0)
    for r in (got, new):
        assert torch.equal(r.scores.view(torch.int32), kept.view(torch.int32))  # bits: NaN among them
    for name, full in (("keys", k), ("values", v)):
        if full is None:
            assert getattr(got, name) is None
            continue
        rows = full.gather(2, at.unsqueeze(3).expand(-1, -1, -1, full.size(3)))
        # behind the new length: as they were, and zeros in new tensors
        assert torch.equal(getattr(got, name), torch.where(there.unsqueeze(3), rows, torch.full_like(rows, 7.0)))
        assert torch.equal(getattr(new, name), torch.where(there.unsqueeze(3), rows, torch.zeros_like(rows)))


def test_evict_offsets_past_32_bits():
    # 2^31 elements and more between the rows of two sequences
    big = torch.empty((1 << 32) + 4096, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((2, 1, 50, 64), (1 << 32, 0, 64, 1))
    k.copy_(torch.randn(2, 1, 50, 64, device="cuda"))
    s = torch.rand(2, 1, 50, device="cuda")
    got = gc.cache_evict(k, None, s, 10)
    for b in range(2):
        at = torch.from_numpy(ref.kept(s[b, 0].cpu().numpy(), 50, 10, 0, 0)).cuda()
        assert torch.equal(got.keys[b, 0], k[b, 0, at])


def test_score_offsets_past_32_bits():
    big = torch.empty((1 << 32) + 4096, dtype=torch.bfloat16, device="cuda")
    w = big.as_strided((2, 1, 3, 64), (1 << 32, 0, 64, 1))
    w.copy_(torch.rand(2, 1, 3, 64, device="cuda"))
    s = torch.rand(2, 1, 64, device="cuda")
    assert torch.equal(gc.cache_score(w, s), gc.cache_score(w.contiguous(), s))


def test_evict_nothing():
    k, s = torch.empty(0, 2, 10, 8, device="cuda"), torch.empty(0, 2, 10, device="cuda")
    assert gc.cache_evict(k, k, s, 4).keys.shape == (0, 2, 4, 8)
    k, s = torch.empty(2, 3, 0, 8, device="cuda"), torch.empty(2, 3, 0, device="cuda")
    got = gc.cache_evict(k, None, s, 4)
    assert not got.keys.any() and not got.scores.any() and bool((got.positions == -1).all()) and not got.lengths.any()
    assert gc.cache_score(torch.empty(2, 6, 1, 0, device="cuda"), s).shape == (2, 3, 0)


def test_streams_graphs_and_two_workspaces():
    rng = np.random.default_rng(1)
    k, v = (cache_of(rng, 4, 4, 6000, 64, "bf16", "head") for _ in range(2))
    w = torch.rand(4, 8, 3, 6000, device="cuda")
    s = torch.rand(4, 4, 6000, device="cuda")

    def both(stream=None):
        total = gc.cache_score(w, s, stream=stream)
        return total, gc.cache_evict(k, v, total, 1000, 4, 64, stream=stream)
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and all(torch.equal(a, b) for a, b in zip(want[1], got[1]))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = both()
        graphs.append((graph, out))
    for _ in range(3):
        s.copy_(torch.rand_like(s))
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = both()
        for _, out in graphs:
            assert torch.equal(want[0], out[0]) and all(torch.equal(a, b) for a, b in zip(want[1], out[1]))


def test_refusals():
    k, s = torch.zeros(2, 3, 20, 8, device="cuda"), torch.zeros(2, 3, 20, device="cuda")
    out = gc.cache_evict(k, k.clone(), s, 5)
    for call in (lambda: gc.cache_evict(k, k[:, :, :19], s, 5), lambda: gc.cache_evict(k, k.half(), s, 5),
                 lambda: gc.cache_evict(k, None, s[:, :, :19], 5), lambda: gc.cache_evict(k, None, s.half(), 5),
                 lambda: gc.cache_evict(k, None, s, 0), lambda: gc.cache_evict(k, None, s, 5, sinks=3, recent=3),
                 lambda: gc.cache_evict(k, None, s, 5, sinks=-1), lambda: gc.cache_evict(k.transpose(2, 3), None, s, 5),
                 lambda: gc.cache_evict(k, None, s, 5, positions=s), lambda: gc.cache_evict(k, None, s, 6, out=out),
                 lambda: gc.cache_evict(k, None, s, 5, lengths=torch.zeros(3, dtype=torch.int32, device="cuda")),
                 lambda: gc.cache_score(torch.zeros(2, 4, 1, 20, device="cuda"), s),
                 lambda: gc.cache_score(torch.zeros(2, 6, 1, 20, device="cuda"), None),
                 lambda: gc.cache_score(torch.zeros(2, 6, 1, 19, device="cuda"), s),
                 lambda: gc.cache_score(torch.zeros(2, 6, 20, 1, device="cuda").transpose(2, 3), s, out=s[:, :, :5])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gc.cache_evict(k.double(), None, s, 5),
                 lambda: gc.cache_evict(k, None, s, 5, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    both = torch.zeros(2, 3, 5, 16, device="cuda")
    for call in (lambda: gc.cache_evict(k, None, s, 5, out=out._replace(keys=k[:, :, :5])),
                 lambda: gc.cache_evict(k, k, s, 5, out=out._replace(keys=both[..., :8], values=both[..., 8:])),
                 lambda: gc.cache_evict(k, None, s, 5, out=out._replace(keys=both[:1].expand(2, 3, 5, 16)[..., :8]))):
        with pytest.raises(gc.GcError):
            call()
