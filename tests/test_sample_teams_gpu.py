"""gc_sample by teams of 1 to 8 CTAs (a cluster per row) on each of its paths,
against the 64-bit form, and launched over and over: a CTA of a cluster must
not touch another's shared memory before that one runs.

Tolerances are check_sample's (test_rows_gpu.py)."""

import numpy as np
import pytest
import torch

from partition_pass_tile_gb300 import gc
from test_rows_gpu import check_sample, logits_of

pytestmark = pytest.mark.gpu

# One per path: greedy, unfiltered, min-p, a listed top-k, a top-k by
# histogram, top-p, both.
PATHS = [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.9, 0, 1.0, 0.05), (0.8, 20, 1.0, 0.0), (1.5, 3000, 1.0, 0.0),
         (1.1, 0, 0.95, 0.0), (0.9, 1500, 0.9, 0.01)]


def rows_of_team(team):
    """The most rows that get teams of this size where the vocabulary allows 8."""
    slots = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    return slots // team if team > 1 else slots // 2 + 1


@pytest.mark.parametrize("team", [8, 4, 2, 1])
@pytest.mark.parametrize("dtype,vocab", [("f32", 32771), ("bf16", 65540)])
def test_every_path_by_every_team(team, dtype, vocab):
    rng = np.random.default_rng(team)
    rows = rows_of_team(team)
    x, x64 = logits_of(rng, rows, vocab, dtype, "peaked", 1, 0)
    u = torch.from_numpy(rng.random((rows, vocab), dtype=np.float32)).clamp_(max=1 - 2.0 ** -24).cuda()
    check_sample(x, x64, u, [PATHS[r % len(PATHS)] for r in range(rows)], vocab)


@pytest.mark.parametrize("path", PATHS)
def test_many_launches_of_small_clusters(path):
    # Launches of few clusters follow one another without a pause, with
    # launches of other shapes between them, and every one finds the same.
    rng = np.random.default_rng(5)
    vocab = 33000
    x, x64 = logits_of(rng, 3, vocab, "f32", "peaked", 0, 0)
    u = torch.from_numpy(rng.random((3, vocab), dtype=np.float32)).cuda()
    t, k, p, q = path
    check_sample(x, x64, u, [path] * 3, vocab)
    want = gc.sample(x, u, temperature=t, top_k=k, top_p=p, min_p=q)
    got = []
    for i in range(200):
        got.append(gc.sample(x[i % 3:i % 3 + 1], u[i % 3:i % 3 + 1], temperature=t, top_k=k, top_p=p, min_p=q)[0])
        if i % 4 == 0:
            x.sum()
    assert torch.equal(torch.cat(got), want[0][torch.arange(200, device="cuda") % 3])
