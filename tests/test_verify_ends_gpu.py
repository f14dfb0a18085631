"""Verification of drafted tokens where its arithmetic is at its ends: elements
outside a row's 16-byte pieces, logits far above those met first, random numbers
below 0, rows without a draft's probabilities.

Tolerances of a log probability, e = 2^-24, with z the distance of its logit
from the largest over T and Z the mean of z over the row's probabilities.  Terms
of z: log2(e) / T is off by 2.3 e, a weight's exponent by e z, the logarithm's
product and conversion by 2 e z: 8 e (z + Z) at most.  Constant ones of a row of
one chunk: 4 e for a weight's approximation; three joins of sums by different
maxima (single elements, lanes, warps), 6 e each; 18 additions; 4 e for the
logarithm and what is added to it: 44 e, taken as 64 e."""

import numpy as np
import pytest
import torch

import more_rows_ref as ref
from partition_pass_tile_gb300 import gc
from test_verify_gpu import DTYPES, check, rows_of, setup

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def log_p(x64, temperature):
    """-> log probabilities in 64 bits, z, the mean of z."""
    z = (x64.max(-1, keepdims=True) - x64) / float(np.float32(temperature))
    w = np.exp(-np.minimum(z, 800.0))
    total = w.sum(-1, keepdims=True)
    return -z - np.log(total), z, (w / total * np.minimum(z, 800.0)).sum(-1, keepdims=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("temperature,size", [(1.0, 10.0), (0.1, 10.0), (0.01, 10.0), (1e-3, 10.0), (1e-4, 10.0),
                                              (1.0, 4000.0), (0.1, 4000.0), (1e-4, 4000.0)])
def test_largest_logit_outside_the_pieces(dtype, temperature, size):
    # rows of odd length an odd distance apart start at every alignment; the largest logit is one of the first or last
    rng = np.random.default_rng(int(size) + round(1 / temperature))
    n, vocab = 48, 1003
    x = size * (0.5 + 0.1 * rng.standard_normal((n, 2, vocab)))
    at = rng.choice([0, 1, 2, 6, 500, vocab - 7, vocab - 3, vocab - 2, vocab - 1], (n, 2))
    np.put_along_axis(x, at[:, :, None], size * (1.2 + 0.3 * rng.random((n, 2, 1))), 2)
    xt, x64 = rows_of(x.astype(np.float32), dtype, 2)
    drafts = torch.from_numpy(at[:, :1].astype(np.int32)).cuda()
    uniform = torch.from_numpy(rng.random((n, vocab)).astype(np.float32)).cuda()
    tokens, accepted, logprobs = gc.sample_verify(xt, drafts, torch.zeros(n, 1, device="cuda"), uniform,
                                                  temperature=temperature)
    assert accepted.tolist() == [1] * n
    lp, z, mean = log_p(x64, temperature)
    tokens = tokens.cpu().numpy()[:, :, None].astype(np.int64)
    assert np.array_equal(tokens[:, 0, 0], at[:, 0])
    want, bound = np.take_along_axis(lp, tokens, 2), (64 + 8 * (np.take_along_axis(z, tokens, 2) + mean)) * E
    assert np.all(np.abs(logprobs.double().cpu().numpy()[:, :, None] - want) <= bound)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("temperature,size", [(1.0, 10.0), (0.01, 10.0), (1e-4, 10.0), (1.0, 4000.0)])
def test_a_certain_token_outside_the_pieces_is_accepted(dtype, temperature, size):
    # p = 1 is above every u q, u at most 1 - 2^-24
    rng = np.random.default_rng(int(size) + round(1 / temperature))
    n, vocab = 48, 77
    x = np.full((n, 2, vocab), -np.inf)
    at = rng.choice([0, 1, 2, 40, vocab - 3, vocab - 2, vocab - 1], (n, 2))
    np.put_along_axis(x, at[:, :, None], size * (1 + rng.random((n, 2, 1))), 2)
    xt, _ = rows_of(x.astype(np.float32), dtype, 2)
    drafts = torch.from_numpy(at[:, :1].astype(np.int32)).cuda()
    tokens, accepted, logprobs = gc.sample_verify(xt, drafts, torch.ones(n, 1, device="cuda"),
                                                  torch.rand(n, vocab, device="cuda"), temperature=temperature)
    assert accepted.tolist() == [1] * n and tokens.tolist() == at.tolist()
    # twice the weight's approximation, 4 e, at most
    assert bool((logprobs.abs() <= 8 * E).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_log_probability_is_above_zero(dtype):
    # one token outweighs all others: its log probability is 0 but for roundings, which must not show as p > 1
    rng = np.random.default_rng(8)
    n, vocab = 600, 2003
    x = 3 * rng.standard_normal((n, 1, vocab))
    x[np.arange(n), 0, rng.integers(0, vocab, n)] = 40 + 10 * rng.random(n)
    xt, _ = rows_of(x.astype(np.float32), dtype, 2)
    none = torch.empty(n, 0, dtype=torch.int32, device="cuda")
    for temperature in (1.3, 1.0, 0.7, 0.05):
        logprobs = gc.sample_verify(xt, none, none.float(), torch.rand(n, vocab, device="cuda"), temperature=temperature)[2]
        assert bool((logprobs <= 0).all())


@pytest.mark.parametrize("number", [-100.0, -float("inf"), -2.0 ** -30, float("nan")])
@pytest.mark.parametrize("dtype", DTYPES)
def test_random_numbers_below_zero_draw(dtype, number):
    # They count as 2^-25.  The token that has one weighs about 50 times each of the others, whose numbers are 0.5: its
    # ratio is 50 / 17.3, theirs 1 / 0.69, which is half of it.  With many sequences a thread has several pieces of a
    # row, and the token's is none of the first.
    for n, vocab in ((1, 1500), (3, 40001), (700, 9000)):
        x = torch.zeros(n, 1, vocab, dtype=DTYPES[dtype], device="cuda")
        uniform = torch.full((n, vocab), 0.5, device="cuda")
        rows = torch.arange(n, device="cuda")
        at = rows % 500 + vocab - 600
        x[rows, 0, at] = 3.9
        uniform[rows, at] = number
        none = torch.empty(n, 0, dtype=torch.int32, device="cuda")
        tokens, _, _ = gc.sample_verify(x, none, none.float(), uniform)
        assert torch.equal(tokens[:, 0].long(), at), (n, vocab)


@pytest.mark.parametrize("dtype", DTYPES)
def test_logits_far_above_the_first_of_a_thread(dtype):
    # Each thread's first piece of a row is low, some of the later ones are 25 to 40 above it, less than 2^60.
    # Beyond the constant terms above: exponents of up to 60 round by 22 e of the weight, in the sum, in p and twice in
    # the logarithm; one join of maxima as far apart, 42 e; up to three more joins, 6 e each, and 24 more additions:
    # 64 + 88 + 42 + 18 + 24, taken as 240 e.
    rng = np.random.default_rng(11)
    n, vocab = 40, 131072
    piece = 4 if dtype == "f32" else 8
    x = rng.standard_normal((n, 1, vocab)).astype(np.float32)
    number = np.arange(vocab) // (256 * piece)                  # of a thread's piece among its pieces
    later = (number % 2 == 1) & (rng.random((n, 1, vocab)) < 0.001)
    x[later] += rng.uniform(25, 40, int(later.sum())).astype(np.float32)
    xt, x64 = rows_of(x, dtype)
    none = torch.empty(n, 0, dtype=torch.int32, device="cuda")
    tokens, _, logprobs = gc.sample_verify(xt, none, none.float(), torch.rand(n, vocab, device="cuda"))
    lp, z, mean = log_p(x64, 1.0)
    tokens = tokens.cpu().numpy()[:, :, None].astype(np.int64)
    want, bound = np.take_along_axis(lp, tokens, 2), (240 + 8 * (np.take_along_axis(z, tokens, 2) + mean)) * E
    assert np.all(np.abs(logprobs.double().cpu().numpy()[:, :, None] - want) <= bound)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_draft_without_an_open_token_whose_token_is_closed(dtype):
    # u q < p is 0 < 0: rejected, and what is drawn from max(p - q, 0) is drawn from p
    rng = np.random.default_rng(4)
    for n, vocab in ((30, 301), (2, 20011), (800, 1003)):
        x = 2 * rng.standard_normal((n, 2, vocab)).astype(np.float32)
        ids = rng.integers(0, vocab, (n, 1))
        np.put_along_axis(x[:, :1], ids[:, :, None], -np.inf, 2)
        xt, x64 = rows_of(x, dtype, 3)
        d = torch.full((n, 1, vocab), -float("inf"), dtype=DTYPES[dtype], device="cuda")
        accept, uniform = rng.random((n, 1)).astype(np.float32), rng.random((n, vocab)).astype(np.float32)
        got = gc.sample_verify(xt, torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(accept).cuda(),
                               torch.from_numpy(uniform).cuda(), draft_logits=d)
        assert not got[1].any()
        compared = 0
        for b in range(n):
            want, a, lp, _ = ref.verify(x64[b], ids[b], accept[b], uniform[b], np.full((1, vocab), -np.inf), 1.0)
            # the first of the ratios is clear of the second by 2^-16 of it
            p, _ = ref.softmax(x64[b, 0])
            ratio = np.sort(p / -np.log(np.clip(uniform[b].astype(np.float64), ref.U_LO, ref.U_HI)))
            if ratio[-1] * (1 - 2.0 ** -16) > ratio[-2]:
                compared += 1
                assert a == 0 and got[0][b].tolist() == want.tolist()
        assert compared >= 0.9 * n


# sequences alone, at seeds for which the 64-bit form's decisions are clear
@pytest.mark.parametrize("seed,k,vocab,dtype,drafted", [
    (1, 0, 1, "f32", False), (2, 1, 1, "bf16", True), (1, 4, 4096, "f32", True), (3, 4, 4096, "f32", True),
    (7, 4, 4096, "f32", True), (3, 6, 30001, "bf16", True), (6, 6, 30001, "bf16", True), (4, 3, 999, "f16", False)])
def test_one_sequence(seed, k, vocab, dtype, drafted):
    (x, x64), (d, d64), ids, accept, uniform, _ = setup(seed, 1, k, vocab, dtype, drafted)
    drafts, acc, uni = (torch.from_numpy(a).cuda() for a in (ids.astype(np.int32), accept, uniform))
    got = gc.sample_verify(x, drafts, acc, uni, draft_logits=d)
    assert check(got, x64, d64, ids, accept, uniform, np.ones(1)) == 1


@pytest.mark.parametrize("dtype", DTYPES)
def test_weights_below_the_least_are_none(dtype):
    # exp(-80) is above 2^-126, exp(-100) below it: with q = 0 the first is accepted, the second is p = 0 and is not
    x = torch.zeros(2, 2, 50, dtype=DTYPES[dtype], device="cuda")
    x[0, 0, 20], x[1, 0, 20] = -80.0, -100.0
    d = torch.zeros(2, 1, 50, dtype=DTYPES[dtype], device="cuda")
    d[:, :, 20] = -float("inf")
    drafts = torch.full((2, 1), 20, dtype=torch.int32, device="cuda")
    tokens, accepted, logprobs = gc.sample_verify(x, drafts, torch.full((2, 1), 0.5, device="cuda"),
                                                  torch.rand(2, 50, device="cuda"), draft_logits=d)
    assert accepted.tolist() == [1, 0] and int(tokens[0, 0]) == 20 and int(tokens[1, 0]) not in (-1, 20)
    # 49 weights of 1: z and its product with ln 2 round by 3 e z, the rest as above
    assert abs(float(logprobs[0, 0]) + 80 + np.log(49.0)) <= (64 + 8 * 80) * E
