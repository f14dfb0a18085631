"""The same call of gc_sample gives the same bits, log probabilities included,
in whatever order the tokens of a row got into a list."""

import numpy as np
import pytest
import torch

from partition_pass_tile_gb300 import gc
from test_rows_gpu import check_sample, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab,dtype,kind,t,k,p", [
    (48, 4000, "f32", "bulk", 1.0, 0, 0.9),      # short rows, all tokens listed
    (48, 4000, "bf16", "steps", 1.5, 0, 0.97),
    (160, 50000, "f32", "peaked", 0.5, 0, 0.95),  # long rows that end in the first pass's list
    (160, 100000, "bf16", "bulk", 0.6, 0, 0.9),
    (4, 100000, "f32", "bulk", 1.0, 0, 0.95),    # a cluster per row
    (4, 100000, "f32", "bulk", 1.0, 3000, 0.9),
    (320, 9000, "f32", "bulk", 1.2, 0, 0.9),     # a CTA per row, by histogram
])
def test_same_bits(rows, vocab, dtype, kind, t, k, p):
    rng = np.random.default_rng(vocab)
    x, x64 = logits_of(rng, rows, vocab, dtype, kind, 0, 0)
    u = torch.from_numpy(rng.random((rows, vocab), dtype=np.float32)).cuda()
    some = slice(0, min(rows, 24))
    check_sample(x[some], x64[some], u[some], [(t, k, p, 0.0)] * (some.stop - some.start), vocab)
    tokens, logprobs = gc.sample(x, u, temperature=t, top_k=k, top_p=p)
    for i in range(30):
        again = gc.sample(x, u, temperature=t, top_k=k, top_p=p)
        assert torch.equal(again[0], tokens)
        assert torch.equal(again[1], logprobs), i
