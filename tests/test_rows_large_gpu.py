"""The row operators' kernels for more items: dispatches above one launch's
pairs, the embedding gradient behind the sort by many CTAs, top-p by the pass
that lists and adds up, large vocabularies, and both sides of each boundary.

Checks and tolerances are test_rows_gpu.py's.  Where top-p ends is a comparison
of two sums of weights, and within their rounding it is open: each is off by at
most what a log probability's sum is (16 * 2^-22 for the weights, 2^-24 per
term of a thread's sum), twice that for both."""

import numpy as np
import pytest
import torch

import rows_ref as ref
from partition_pass_tile_gb300 import gc
from test_rows_gpu import check_sample, logits_of
from test_rows_gpu import test_embedding as check_embedding
from test_rows_gpu import test_exchange as check_exchange

pytestmark = pytest.mark.gpu


# tokens, topk, experts, align, width, dtype, ids, routing, pad, shift
@pytest.mark.parametrize("case", [
    (4096, 1, 8, 1, 2048, "bf16", "i64", "even", 0, 0),     # the last of one launch
    (4097, 1, 8, 1, 2048, "bf16", "i64", "even", 0, 0),     # the first of three
    (2100, 2, 9, 8, 1101, "bf16", "i32", "drop", 3, 1),     # element by element, twice around the row
    (1100, 4, 60, 128, 2056, "f16", "i64", "skew", 8, 8),   # 257 pieces: more than a CTA's threads
    (700, 6, 5, 16, 5000, "f32", "i32", "skew", 0, 0),      # more than four pieces to a thread
    (70, 64, 2048, 1, 24, "f32", "i64", "even", 0, 0),      # more choices than threads to a row
    (65, 64, 2048, 3, 264, "f16", "i32", "drop", 0, 2),
    (2100, 2, 9, 4, 40, "f32", "i64", "none", 0, 0),        # everything dropped
    (5000, 1, 1, 1, 516, "bf16", "i32", "one", 4, 4),
    (1031, 8, 333, 1, 96, "f32", "i64", "even", 1, 1),
], ids=str)
def test_dispatch_by_three_kernels(case):
    check_exchange(*case)


# n, vocab, width, dtype, out, ids, spread, pad, shift
@pytest.mark.parametrize("case", [
    (4096, 3000, 40, "f32", "f32", "i64", "zipf", 0, 0),        # the last that one CTA sorts
    (4096, 50, 256, "f32", "f32", "i32", "outside", 0, 0),      # and in bulk, long runs
    (4097, 3000, 2056, "bf16", "bf16", "i64", "zipf", 0, 0),    # several slices to a row, the last in part
    (6000, 500, 1028, "f32", "f32", "i32", "outside", 0, 0),
    (9000, 20000, 256, "f16", "f16", "i64", "zipf", 0, 0),      # several blocks to a CTA
    (9000, 3000, 264, "f16", "f32", "i32", "zipf", 8, 8),
    (5000, 7, 512, "bf16", "f32", "i64", "one", 0, 0),          # one run over many blocks
    (5000, 9000, 2048, "bf16", "f32", "i64", "outside", 0, 0),  # mostly absent rows
    (4500, 2000, 768, "bf16", "bf16", "i32", "all", 4, 0),      # rows on 8-byte boundaries: no bulk copies
    (600, 40, 20480, "bf16", "f32", "i64", "zipf", 0, 0),
], ids=str)
def test_embedding_gradient_by_bulk_copies(case):
    check_embedding(*case)


def drawn_of_cuts(x, u, t, top_p, min_p, slack):
    """(token, logprob, z of the token) for each cut that top-p has with sums of
    weights that are off by `slack`: nearly always one, and two or a few where a
    sum of the first tokens comes that near to top_p of all."""
    order, z, w = ref.kept_tokens(x, t, 0, 1.0, 0.0)
    if order.size == 0:
        return [(-1, -np.inf, 0.0)]
    upto = np.cumsum(w)
    first, last = (1 + np.searchsorted(upto[:-1], top_p * upto[-1] * (1 + s)) for s in (-slack, slack))
    score = z - np.log(-np.log(np.clip(u[order], ref.U_LO, ref.U_HI)))
    got = []
    for n in range(first, last + 1):
        n = n if min_p <= 0 else int((w[:n] >= min(min_p, 1.0)).sum())
        best = min(np.flatnonzero(score[:n] == score[:n].max()), key=lambda i: order[i])
        got.append((int(order[best]), float(z[best] - np.log(w[:n].sum())), float(z[best])))
    return got


@pytest.mark.parametrize("kind", ["bulk", "peaked", "flat", "steps", "masked", "lowest", "far", "broken"])
@pytest.mark.parametrize("dtype,vocab,pad,shift", [("f32", 50000, 0, 0), ("bf16", 100000, 0, 0),
                                                   ("f16", 100001, 5, 3), ("f32", 131073, 2, 1)])
def test_top_p_of_many_long_rows(dtype, vocab, pad, shift, kind):
    # A CTA to a row, which needs more rows than half the GPU's SMs hold: a
    # few rows are there many times, each time with other filters.
    params = [(t, 0, p, q) for t in (0.3, 0.5, 0.7, 1.0, 1.2, 5.0) for p, q in ((0.95, 0.0), (0.5, 0.0), (0.9, 0.05),
                                                                              (0.999, 0.0), (0.0, 0.0))]
    rng = np.random.default_rng(vocab + len(kind))
    some, some64 = logits_of(rng, 3, vocab, dtype, kind, pad, shift)
    u_some = rng.random((3, vocab), dtype=np.float32)
    rows = max(160, torch.cuda.get_device_properties(0).multi_processor_count + 8)
    at = np.arange(rows) % 3
    wide = torch.empty(rows, vocab + pad + shift, dtype=some.dtype, device="cuda")
    x = wide[:, shift:shift + vocab]
    x.copy_(some[torch.from_numpy(at).cuda()])
    u = torch.from_numpy(u_some).cuda()[torch.from_numpy(at).cuda()]
    each = [params[r // 3 % len(params)] for r in range(rows)]
    t, _, p, q = (torch.tensor(v, dtype=torch.float32, device="cuda") for v in zip(*each))
    tokens, logprobs = gc.sample(x, u, temperature=t, top_p=p, min_p=q)
    tokens, logprobs = tokens.cpu().numpy(), logprobs.double().cpu().numpy()
    f = lambda v: float(np.float32(v))  # noqa: E731
    wants = {}
    for r in range(rows):
        key = (at[r], each[r])
        if key not in wants:
            wants[key] = drawn_of_cuts(some64[at[r]], u_some[at[r]].astype(np.float64), f(each[r][0]), f(each[r][2]),
                                       f(each[r][3]), 2 * (2.0 ** -18 + (vocab / 1024 + 12) * 2.0 ** -24))
        assert any(tokens[r] == want and (logprobs[r] == lp if np.isinf(lp) else abs(logprobs[r] - lp) <=
                   2.0 ** -22 * (abs(z) + 16) + (vocab / 1024 + 12) * 2.0 ** -24 + 2.0 ** -23 * abs(lp))
                   for want, lp, z in wants[key]), (r, each[r], tokens[r], logprobs[r], wants[key])


@pytest.mark.parametrize("dtype,vocab,rows", [("bf16", 1000003, 6), ("f32", 4194304, 6), ("f16", 4194303, 3)])
def test_the_largest_vocabularies(dtype, vocab, rows):
    rng = np.random.default_rng(vocab)
    params = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (0.8, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.0, 0, 1.0, 0.0),
              (0.9, 2500, 0.95, 0.001)][:rows]
    x, x64 = logits_of(rng, rows, vocab, dtype, "peaked", 0, 0)
    u = torch.from_numpy(rng.random((rows, vocab), dtype=np.float32)).clamp_(max=1 - 2.0 ** -24).cuda()
    check_sample(x, x64, u, params, vocab)


@pytest.mark.parametrize("vocab", [4095, 4096, 4097])
@pytest.mark.parametrize("rows", [1, 400])
def test_rows_about_a_list(vocab, rows):
    rng = np.random.default_rng(vocab)
    x, x64 = logits_of(rng, rows, vocab, "f32", "bulk", 0, 0)
    u = torch.from_numpy(rng.random((rows, vocab), dtype=np.float32)).cuda()
    params = [(1.0, k, p, 0.0) for k in (0, 512, 513) for p in (0.9, 1.0)]
    check_sample(x, x64, u, [params[r % len(params)] for r in range(rows)], vocab)
