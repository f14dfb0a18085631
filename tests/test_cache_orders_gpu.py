"""Eviction on the GPU with scores that are not numbers, and refusals of scores."""

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


def test_scores_that_are_not_numbers_count_as_the_least():
    # NaN and -inf are one value: of them the lower position is kept
    nan, inf = float("nan"), float("inf")
    s = torch.tensor([[[nan, -inf, nan, 1.0], [-inf, nan, -inf, nan], [nan, -3e38, -inf, nan], [-nan, -inf, inf, 0.0]]],
                     device="cuda")
    k = torch.arange(32, dtype=torch.float32, device="cuda").view(1, 4, 4, 2)
    assert gc.cache_evict(k, None, s, 2).positions.tolist() == [[[0, 3], [0, 1], [0, 1], [2, 3]]]
    assert gc.cache_evict(k, None, s, 1).positions.tolist() == [[[3], [0], [1], [2]]]
    check(k, s, [4], 3, 0, 0)


def test_scores_of_other_shapes_are_refused():
    w = torch.zeros(2, 6, 1, 20, device="cuda")
    for call in (lambda: gc.cache_score(w, None, heads=-1), lambda: gc.cache_score(w, None, heads=0),
                 lambda: gc.cache_score(w, torch.zeros(20, device="cuda")),
                 lambda: gc.cache_score(w, torch.zeros(2, 20, device="cuda")),
                 lambda: gc.cache_score(w, torch.zeros(2, 3, 20, device="cuda"), heads=2)):
        with pytest.raises(ValueError):
            call()
