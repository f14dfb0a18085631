"""Eviction on the GPU at sizes that take each of its selection kernels with
more CTAs than SMs, and with nearly all scores equal."""

import numpy as np
import pytest
import torch

from test_cache_orders_gpu import check

pytestmark = pytest.mark.gpu


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
