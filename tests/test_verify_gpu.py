"""Verification of drafted tokens on the GPU against a plain 64-bit form (more_rows_ref.py).

Tokens are whole numbers that hang on comparisons of rounded probabilities: p
and q are off by at most (4 + 5/4 |z|) 2^-22 of themselves, which for |z| <= 20
is below 2^-17, and their sums by less.  Where every comparison of the 64-bit
form is clear by 2^-16 the results have to be equal; the others, a few in 10^4
comparisons, are not compared.  Log probabilities: 2^-24 |lp| for the final
rounding, 3 |z| 2^-24 for z and 2^-18 for the logarithm of the sum."""

import numpy as np
import pytest
import torch

import more_rows_ref as ref
from partition_pass_tile_gb300 import gc

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rows_of(x, dtype, pad=0, shift=0):
    """[n, m, vocab] values as logits on the GPU (slices of wider rows) and what they hold."""
    n, m, vocab = x.shape
    wide = torch.zeros(n, m, vocab + pad + shift, dtype=DTYPES[dtype], device="cuda")
    wide[:, :, shift:shift + vocab] = torch.from_numpy(x).to(DTYPES[dtype]).cuda()
    got = wide[:, :, shift:shift + vocab]
    return got, got.double().cpu().numpy()


def setup(seed, n, k, vocab, dtype, drafted, pad=0, shift=0, forbidden=0.0, short=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, k + 1, vocab)).astype(np.float32) * 2
    x[rng.random(x.shape) < forbidden] = -np.inf
    d = np.where(rng.random((n, k, 1)) < 0.75, x[:, :k] + 0.3 * rng.standard_normal((n, k, vocab)),
                 2 * rng.standard_normal((n, k, vocab))).astype(np.float32)
    ids = np.zeros((n, k), np.int64)
    for b in range(n):
        for j in range(k):
            like = ref.clean(d[b, j] if rng.random() < 0.9 else rng.standard_normal(vocab))
            p, _ = ref.softmax(like)
            ids[b, j] = rng.choice(vocab, p=p / p.sum()) if p.sum() > 0 else 0
    if short:
        for b in range(n):
            if k and rng.random() < short:
                ids[b, rng.integers(k):] = rng.choice([-1, vocab, -2 ** 31, 2 ** 31 - 1])
    accept, uniform = rng.random((n, k)).astype(np.float32), rng.random((n, vocab)).astype(np.float32)
    t = rng.choice([0.0, 0.5, 1.0, 1.7], n).astype(np.float32)
    xt, x64 = rows_of(x, dtype, pad, shift)
    dt, d64 = rows_of(d, dtype, pad, 0) if drafted and k else (None, None)
    return (xt, x64), (dt, d64), ids, accept, uniform, t


def check(got, x64, d64, ids, accept, uniform, t):
    tokens, accepted, logprobs = (a.cpu().numpy() for a in got)
    n, k = ids.shape
    compared = 0
    for b in range(n):
        want, a, lp, sure = ref.verify(x64[b], ids[b], None if accept is None else accept[b],
                                       None if uniform is None else uniform[b], None if d64 is None else d64[b],
                                       float(t[b]))
        if not sure:
            continue
        compared += 1
        assert tokens[b].tolist() == want.tolist() and accepted[b] == a, b
        dead = ~np.isfinite(lp)
        assert np.array_equal(dead, ~np.isfinite(logprobs[b])) and np.all(logprobs[b][dead] == -np.inf)
        # |z| is at most |lp| + the logarithm of the vocabulary
        bound = (4 * np.abs(lp[~dead]) + 3 * np.log(x64.shape[2])) * 2.0 ** -24 + 2.0 ** -18
        assert np.all(np.abs(logprobs[b][~dead] - lp[~dead]) <= bound)
    return compared


# sequences, drafts, vocab, dtype, drafted, pad, shift, forbidden, short
VERIFY = [
    (1, 0, 1, "f32", False, 0, 0, 0.0, 0.0),
    (1, 1, 1, "bf16", True, 0, 0, 0.0, 0.0),
    (1, 4, 4096, "f32", True, 0, 0, 0.0, 0.0),
    (2, 3, 5, "f16", True, 3, 1, 0.2, 0.3),
    (5, 0, 1000, "bf16", False, 0, 0, 0.0, 0.0),
    (7, 2, 31, "bf16", False, 1, 0, 0.0, 0.5),
    (16, 5, 2049, "f32", True, 0, 0, 0.5, 0.2),
    (9, 7, 10007, "bf16", True, 5, 3, 0.0, 0.3),
    (9, 7, 10007, "f16", False, 0, 0, 0.0, 0.3),
    (3, 64, 300, "bf16", True, 0, 0, 0.0, 0.0),
    (200, 3, 513, "bf16", True, 0, 0, 0.1, 0.2),
    (3, 2, 131072, "bf16", True, 0, 0, 0.0, 0.0),
    (2, 1, 200001, "f32", False, 0, 0, 0.0, 0.0),
    (700, 2, 64, "f32", True, 0, 0, 0.0, 0.1),
    (400, 3, 3001, "f16", False, 1, 0, 0.1, 0.3),
    # five times as many chunks as CTAs at a time: positions are decided on the way
    (1200, 3, 301, "f16", False, 1, 0, 0.1, 0.3),
    (950, 2, 500, "bf16", True, 0, 0, 0.0, 0.2),
    (520, 4, 300, "f32", True, 3, 1, 0.3, 0.4),
    (1300, 0, 40, "bf16", False, 0, 0, 0.0, 0.0),
]


@pytest.mark.parametrize("n,k,vocab,dtype,drafted,pad,shift,forbidden,short", VERIFY)
def test_verify(n, k, vocab, dtype, drafted, pad, shift, forbidden, short):
    (x, x64), (d, d64), ids, accept, uniform, t = setup(n * 1000 + vocab, n, k, vocab, dtype, drafted, pad, shift,
                                                        forbidden, short)
    drafts = torch.from_numpy(ids.astype(np.int32)).cuda()
    acc, uni, temp = (torch.from_numpy(a).cuda() for a in (accept, uniform, t))
    got = gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp)
    assert check(got, x64, d64, ids, accept, uniform, t) >= 0.95 * n - 1
    again = gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    greedy = gc.sample_verify(x, drafts)
    assert check(greedy, x64, d64, ids, None, None, np.zeros(n)) == n
    one = gc.sample_verify(x, drafts, acc, uni, draft_logits=d)
    check(one, x64, d64, ids, accept, uniform, np.ones(n))


def test_rows_that_are_skipped():
    # many more chunks than the GPU holds at a time, two to a row: rows behind a rejection are not read, and what they
    # hold does not matter
    (x, x64), (d, d64), ids, accept, uniform, t = setup(77, 280, 4, 33000, "bf16", True, short=0.2)
    t[:] = np.where(t > 0, t, 1.0)
    drafts, acc, uni, temp = (torch.from_numpy(a).cuda() for a in (ids.astype(np.int32), accept, uniform, t))
    got = gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp)
    assert check(got, x64, d64, ids, accept, uniform, t) >= 250
    for b, a in enumerate(got[1].tolist()):
        x[b, a + 1:] = float("nan")
        d[b, a + 1:] = float("inf")
    again = gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drafted", [True, False])
def test_forbidden_and_infinite_logits(dtype, drafted):
    inf, nan = float("inf"), float("nan")
    v = 300
    x = torch.zeros(6, 2, v, dtype=DTYPES[dtype], device="cuda")
    x[0] = -inf                       # nothing can be drawn
    x[1] = nan
    x[2, :, 7] = inf                  # certain
    x[3] = -inf
    x[3, :, 11] = -3e4                # the only one left
    x[4, 0, ::2] = nan                # half forbidden
    x[5, 1] = -inf                    # the place past the draft
    x[5, 0, 3] = inf
    d = torch.zeros(6, 1, v, dtype=DTYPES[dtype], device="cuda") if drafted else None
    if drafted:
        d[4] = -inf                   # a draft that says nothing: q is 0
        d[2, 0, 9] = nan
    drafts = torch.tensor([[5], [5], [7], [11], [9], [3]], dtype=torch.int32, device="cuda")
    accept = torch.full((6, 1), 0.5, device="cuda")
    uniform = torch.rand(6, v, device="cuda")
    for t in (1.0, 0.0):
        tokens, accepted, logprobs = gc.sample_verify(x, drafts, accept, uniform, draft_logits=d, temperature=t)
        assert tokens[:2].tolist() == [[-1, -1]] * 2 and accepted[:2].tolist() == [0, 0]
        assert bool((logprobs[:2] == -inf).all())
        assert tokens[2].tolist() == [7, 7] and accepted[2] == 1 and logprobs[2].tolist() == [0.0, 0.0]
        assert tokens[3].tolist() == [11, 11] and accepted[3] == 1
        assert tokens[5].tolist() == [3, -1] and accepted[5] == 1 and logprobs[5].tolist() == [0.0, -inf]
    tokens, accepted, _ = gc.sample_verify(x, drafts, accept, uniform, draft_logits=d, temperature=1.0)
    assert int(tokens[4, 0]) % 2 == 1
    assert int(accepted[4]) == (1 if drafted else 0)


def test_random_numbers_at_their_ends():
    # u counts as [2^-25, 1 - 2^-24], NaN as 2^-25
    x = torch.zeros(4, 2, 2, device="cuda")
    x[:, 0, 1] = -4.0
    drafts = torch.ones(4, 1, dtype=torch.int32, device="cuda")
    accept = torch.tensor([[0.0], [1.0], [float("nan")], [-3.0]], device="cuda")
    uniform = torch.tensor([[0.0, 1.0], [1.0, 0.0], [float("nan"), 0.5], [0.5, 0.5]], device="cuda")
    tokens, accepted, _ = gc.sample_verify(x, drafts, accept, uniform)
    assert accepted.tolist() == [1, 0, 1, 1]
    assert tokens.tolist() == [[1, 1], [0, -1], [1, 1], [1, 0]]


def test_the_first_token_is_distributed_as_the_target():
    # 2^18 sequences of one draft each: a share p is off by more than
    # 5 sqrt(p (1 - p) / n) with a chance of 6e-7
    n, v = 1 << 18, 6
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.tensor([2.0, 1.0, 0.0, -1.0, 0.5, 1.5], device="cuda")
    d = torch.tensor([0.0, 1.0, 2.0, 0.0, -2.0, 1.0], device="cuda")
    p = torch.softmax(x.double(), 0).cpu().numpy()
    logits = x.expand(n, 2, v).contiguous()
    drafts = torch.multinomial(torch.softmax(d, 0), n, replacement=True, generator=g).int().unsqueeze(1)
    accept, uniform = torch.rand(n, 1, generator=g, device="cuda"), torch.rand(n, v, generator=g, device="cuda")
    for draft in (d.expand(n, 1, v).contiguous(), None):
        tokens, accepted, _ = gc.sample_verify(logits, drafts, accept, uniform, draft_logits=draft)
        for place, rows in ((0, torch.ones(n, dtype=torch.bool, device="cuda")), (1, accepted == 1)):
            got = torch.bincount(tokens[rows, place].long(), minlength=v).double().cpu().numpy()
            m = got.sum()
            assert np.all(np.abs(got / m - p) <= 5 * np.sqrt(p * (1 - p) / m)), (place, got / m, p)


def test_differences_that_round_to_nothing_still_draw():
    # a draft that differs by less than a rounding, and a number that rejects wherever that can be: always a token
    n = 4096
    x = torch.zeros(n, 2, 3, device="cuda")
    d = torch.zeros(n, 1, 3, device="cuda")
    d[:, 0, 0] = torch.arange(n, device="cuda") * 2.0 ** -31
    drafts = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    tokens, accepted, _ = gc.sample_verify(x, drafts, torch.ones(n, 1, device="cuda"), torch.rand(n, 3, device="cuda"),
                                           draft_logits=d)
    assert bool(((tokens[:, 0] >= 0) & (tokens[:, 0] < 3)).all())
    assert bool((tokens[accepted == 1, 1] >= 0).all()) and bool((tokens[accepted == 0, 1] == -1).all())


def test_offsets_past_32_bits():
    (x, x64), (d, d64), ids, accept, uniform, t = setup(3, 3, 2, 64, "bf16", True)
    big = torch.empty(9 << 29, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((3, 3, 64), (3 << 29, 1 << 29, 1))
    far.copy_(x)
    drafts, acc, uni, temp = (torch.from_numpy(a).cuda() for a in (ids.astype(np.int32), accept, uniform, t))
    for draft in (d, None):
        want = gc.sample_verify(x, drafts, acc, uni, draft_logits=draft, temperature=temp)
        got = gc.sample_verify(far, drafts, acc, uni, draft_logits=draft, temperature=temp)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("temperature", [1e-45, 1e-30, 1e30, float("inf"), float("nan"), -1.0])
@pytest.mark.parametrize("dtype", DTYPES)
def test_temperatures_at_their_ends(dtype, temperature):
    # next to 0 the largest logit is all there is, at infinity every open token weighs the same
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (3 * torch.randn(50, 2, 777, generator=g, device="cuda")).to(DTYPES[dtype])
    top = x.float().argmax(2)
    drafts = top[:, :1].int()
    drafts[25:] = (drafts[25:] + 1) % 777
    accept, uniform = torch.full((50, 1), 0.5, device="cuda"), torch.rand(50, 777, generator=g, device="cuda")
    tokens, accepted, logprobs = gc.sample_verify(x, drafts, accept, uniform, temperature=temperature)
    if temperature > 1:
        assert not accepted.any() and bool(((tokens[:, 0] >= 0) & (tokens[:, 0] != drafts[:, 0])).all())
        # off by |z| of at most 1e-28, the sum's 777 additions and its logarithm
        assert bool(((logprobs[:, 0] + np.log(777)).abs() <= 800 * 2.0 ** -24).all())
        return
    first = (x.float() == x.float().amax(2, keepdim=True)).float().argmax(2)
    unique = (x.float() == x.float().amax(2, keepdim=True)).sum(2) == 1
    sure = unique.all(1)
    assert sure.sum() > 20
    assert bool((accepted[:25][sure[:25]] == 1).all()) and bool((accepted[25:][sure[25:]] == 0).all())
    assert torch.equal(tokens[:25][sure[:25]], first[:25][sure[:25]].int())
    assert torch.equal(tokens[25:, 0][sure[25:]], first[25:, 0][sure[25:]].int())
    assert bool((logprobs[:, 0][sure] == 0).all())


def test_logits_of_any_size():
    # values whose difference, or product with log2(e) / T, leaves float32
    for big in (3e38, 1e30, 1e25):
        x = torch.full((4, 2, 100), -big, device="cuda")
        x[0, :, 3] = big                      # one far above the rest
        x[1, :, 3], x[1, :, 4] = big, big     # two
        x[2, :, 50:] = big                    # half
        drafts = torch.tensor([[3], [4], [60], [0]], dtype=torch.int32, device="cuda")
        accept, uniform = torch.full((4, 1), 0.001, device="cuda"), torch.rand(4, 100, device="cuda")
        for t in (1.0, 1e-3, 1e3):
            tokens, accepted, lp = gc.sample_verify(x, drafts, accept, uniform, draft_logits=torch.zeros(4, 1, 100, device="cuda"), temperature=t)
            assert accepted.tolist() == [1, 1, 1, 1]
            assert tokens[0].tolist() == [3, 3] and int(tokens[1, 1]) in (3, 4) and int(tokens[2, 1]) >= 50
            want = torch.log(torch.tensor([1.0, 0.5, 1 / 50, 1 / 100], device="cuda"))
            assert bool(((lp[:, 0] - want).abs() <= 2.0 ** -18).all())
            r = gc.expert_route(x[:, 0], 3)
            assert r.ids[0, 0] == 3 and r.ids[1].tolist()[:2] == [3, 4] and r.ids[2].tolist() == [50, 51, 52]
            assert torch.equal(r.ids[3], torch.arange(3, dtype=torch.int32, device="cuda"))
            assert bool(((r.weights.sum(1) - 1).abs() <= 8 * 2.0 ** -24).all())


def test_nothing_to_verify():
    tokens, accepted, logprobs = gc.sample_verify(torch.empty(0, 3, 8, device="cuda"),
                                                  torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert tokens.shape == (0, 3) and accepted.shape == (0,) and logprobs.shape == (0, 3)


def test_without_drafts_it_is_sampling():
    # the same draw as an unfiltered gc.sample's, but for the roundings of two scores
    x, u = 2 * torch.randn(64, 1, 5000, device="cuda"), torch.rand(64, 5000, device="cuda")
    none = torch.empty(64, 0, dtype=torch.int32, device="cuda")
    tokens, accepted, logprobs = gc.sample_verify(x, none, none.float(), u, temperature=0.8)
    want, lp = gc.sample(x[:, 0], u, temperature=0.8)
    assert not accepted.any() and (tokens[:, 0] == want).sum() >= 63
    same = tokens[:, 0] == want
    assert bool(((logprobs[:, 0] - lp).abs()[same] <= 2.0 ** -17).all())


def test_streams_graphs_and_given_outputs():
    (x, x64), (d, d64), ids, accept, uniform, t = setup(5, 40, 4, 30000, "bf16", True)
    drafts, acc, uni, temp = (torch.from_numpy(a).cuda() for a in (ids.astype(np.int32), accept, uniform, t))
    want = gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out = (torch.empty(40, 5, dtype=torch.int32, device="cuda"), torch.empty(40, dtype=torch.int32, device="cuda"),
           torch.empty(40, 5, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp, tokens=out[0], accepted=out[1],
                         logprobs=out[2])
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = gc.sample_verify(x, drafts, acc, uni, draft_logits=d, temperature=temp)
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        uni.copy_(torch.rand_like(uni))
        acc.copy_(torch.rand_like(acc))


def test_refusals():
    x, d = torch.randn(2, 3, 50, device="cuda"), torch.randn(2, 2, 50, device="cuda")
    ids, acc, u = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.rand(2, 2, device="cuda"), torch.rand(2, 50, device="cuda")
    for call in (lambda: gc.sample_verify(x[0], ids), lambda: gc.sample_verify(x, ids[:, :1]),
                 lambda: gc.sample_verify(x, ids, acc), lambda: gc.sample_verify(x, ids, acc, u[:, :49]),
                 lambda: gc.sample_verify(x, ids, acc, u, draft_logits=d[:, :1]),
                 lambda: gc.sample_verify(x, ids, acc, u, draft_logits=d.bfloat16()),
                 lambda: gc.sample_verify(x, ids, acc, u, temperature=torch.ones(3, device="cuda")),
                 lambda: gc.sample_verify(torch.randn(2, 6, 50, device="cuda")[:, :3], ids),
                 lambda: gc.sample_verify(x.transpose(1, 2), ids)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        gc.sample_verify(x, ids.long(), acc, u)
    with pytest.raises(gc.GcError):
        gc.sample_verify(torch.randn(1, 66, 8, device="cuda"), torch.zeros(1, 65, dtype=torch.int32, device="cuda"))
