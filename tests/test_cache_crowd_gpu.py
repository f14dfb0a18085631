"""Eviction on the GPU at sizes that take each of its selection kernels with
more CTAs than SMs, and with scores that are not numbers."""

import numpy as np
import pytest
import torch

import more_rows_ref as ref
from partition_pass_tile_gb300 import gc

pytestmark = pytest.mark.gpu


def kept_of(scores, lengths, budget, sinks, recent):
    """[batch, heads, length] scores -> kept positions in the plain form, `length` where none is."""
    batch, heads, length = scores.shape
    where = np.full((batch, heads, budget), length, np.int64)
    for b in range(batch):
        for h in range(heads):
            at = ref.kept(scores[b, h], lengths[b], budget, sinks, recent)
            where[b, h, :at.size] = at
    return where


def check(k, s, lengths, budget, sinks, recent):
    batch, heads, length = s.shape
    n = [length] * batch if lengths is None else lengths
    got = gc.cache_evict(k, None, s, budget, sinks, recent,
                         lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    where = kept_of(s.cpu().numpy(), n, budget, sinks, recent)
    there = torch.from_numpy(where < length).cuda()
    at = torch.from_numpy(np.minimum(where, length - 1)).cuda()
    assert torch.equal(got.positions, torch.where(there, at, -1).int())
    assert torch.equal(got.scores.view(torch.int32), torch.where(there, s.gather(2, at), 0.0).view(torch.int32))
    rows = k.gather(2, at.unsqueeze(3).expand(-1, -1, -1, k.size(3)))
    assert torch.equal(got.keys, torch.where(there.unsqueeze(3), rows, torch.zeros_like(rows)))
    assert got.lengths.tolist() == [min(x, budget) for x in n]


# batch, heads, length, budget, sinks, recent: 4, 8, 16 and 32 positions to a thread, one, two and eight CTAs to a head
CROWDED = [(20, 8, 4000, 900, 4, 100), (20, 8, 5001, 1200, 4, 64), (10, 16, 8192, 8000, 0, 1), (160, 1, 16000, 300, 2, 20),
           (16, 10, 30000, 700, 4, 128), (16, 10, 40001, 800, 0, 0), (20, 1, 200000, 5000, 4, 64)]


@pytest.mark.parametrize("batch,heads,length,budget,sinks,recent", CROWDED)
@pytest.mark.parametrize("how", ["any", "few", "ragged"])
def test_more_heads_than_sms(batch, heads, length, budget, sinks, recent, how):
    rng = np.random.default_rng(length + budget)
    s = np.exp(2 * rng.standard_normal((batch, heads, length))).astype(np.float32)
    if how == "few":
        s = np.floor(s)
    k = torch.from_numpy(rng.standard_normal((batch, heads, length, 2)).astype(np.float32)).cuda()
    lengths = [int(rng.integers(0, length + 1)) for _ in range(batch)] if how == "ragged" else None
    check(k, torch.from_numpy(s).cuda(), lengths, budget, sinks, recent)


@pytest.mark.parametrize("length", [3000, 70000])
def test_nearly_all_scores_equal(length):
    # fresh positions, weights of 0: one value, and a few others
    rng = np.random.default_rng(length)
    s = np.zeros((2, 4, length), np.float32)
    s[:, :, rng.integers(0, length, 50)] = rng.random(50).astype(np.float32)
    s[1, 2:] = 0.25
    k = torch.from_numpy(rng.standard_normal((2, 4, length, 4)).astype(np.float32)).cuda()
    check(k, torch.from_numpy(s).cuda(), [length, length - 7], 1000, 4, 60)


def test_scores_that_are_not_numbers_count_as_the_least():
    # NaN and -inf are one value: of them the lower position is kept
    nan, inf = float("nan"), float("inf")
    s = torch.tensor([[[nan, -inf, nan, 1.0], [-inf, nan, -inf, nan], [nan, -3e38, -inf, nan], [-nan, -inf, inf, 0.0]]],
                     device="cuda")
    k = torch.arange(32, dtype=torch.float32, device="cuda").view(1, 4, 4, 2)
    assert gc.cache_evict(k, None, s, 2).positions.tolist() == [[[0, 3], [0, 1], [0, 1], [2, 3]]]
    assert gc.cache_evict(k, None, s, 1).positions.tolist() == [[[3], [0], [1], [2]]]
    check(k, s, [4], 3, 0, 0)
