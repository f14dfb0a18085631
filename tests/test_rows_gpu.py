"""The row operators on the GPU against plain 64-bit forms (rows_ref.py).

Tolerances, from the arithmetic: a sum of n float32 products, each rounded
once per addition, is off by at most n * 2^-24 * (sum of the magnitudes),
plus one rounding to the output's type; copies, plans and tokens are equal."""

import numpy as np
import pytest
import torch

import rows_ref as ref
from partition_pass_tile_gb300 import gc

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IDS = {"i32": torch.int32, "i64": torch.int64}


def rows_of(rng, n, width, dtype, pad=0, shift=0):
    """Rows on the GPU (a slice of wider ones, `shift` elements in) and the values they hold."""
    wide = torch.from_numpy(rng.standard_normal((n, width + pad + shift)).astype(np.float32)).to(DTYPES[dtype])
    x = wide.cuda()[:, shift:shift + width]
    return x, wide[:, shift:shift + width].double().numpy()


def off(got, want, size, terms, dtype):
    """Largest error over its bound."""
    got = got.double().cpu().numpy()
    bound = (terms + 1) * 2.0 ** -24 * size * (1 + 2 * ref.UNIT[dtype]) + ref.UNIT[dtype] * np.abs(want) + ref.TINY[dtype]
    assert got.shape == want.shape
    return float(np.max(np.abs(got - want) / bound, initial=0.0))


def routing(rng, tokens, topk, experts, how, ids):
    n = tokens * topk
    if how == "one":
        e = np.full(n, experts - 1)
    elif how == "none":
        e = rng.choice([-1, experts, -7, experts + 3], n)
    elif how == "drop":
        e = rng.integers(-2, experts + 2, n)
    else:
        e = np.minimum(rng.geometric(0.2, n) - 1, experts - 1) if how == "skew" else rng.integers(0, experts, n)
    e = e.reshape(tokens, topk)
    return torch.from_numpy(e.astype(np.int64 if ids == "i64" else np.int32)).cuda(), e


# tokens, topk, experts, align, width, dtype, ids, routing, pad, shift
EXCHANGE = [
    (1, 1, 1, 1, 1, "f32", "i32", "even", 0, 0),
    (1, 4, 64, 1, 256, "bf16", "i64", "even", 0, 0),
    (1, 8, 8, 128, 64, "f16", "i64", "one", 0, 0),
    (3, 2, 5, 7, 33, "bf16", "i32", "drop", 3, 1),
    (16, 4, 64, 1, 2048, "bf16", "i64", "even", 0, 0),
    (31, 1, 2, 16, 514, "f16", "i32", "skew", 2, 0),
    (32, 64, 2048, 1, 24, "f32", "i64", "even", 0, 0),
    (100, 3, 7, 16, 1001, "f16", "i32", "drop", 5, 2),
    (129, 8, 60, 128, 520, "bf16", "i64", "skew", 8, 8),
    (257, 2, 3, 1, 12, "f32", "i64", "none", 0, 0),
    (512, 2, 513, 8, 68, "f32", "i32", "drop", 0, 4),
    (513, 2, 16, 64, 129, "bf16", "i64", "even", 0, 0),
    (700, 10, 333, 1, 96, "f16", "i64", "even", 0, 0),
    (1025, 1, 1, 1, 40, "bf16", "i32", "one", 0, 0),
    (2500, 6, 128, 16, 72, "bf16", "i64", "skew", 0, 0),
    (40000, 5, 256, 32, 8, "bf16", "i32", "drop", 0, 0),
    (4, 3, 9, 2, 20000, "bf16", "i32", "even", 0, 0),
]


@pytest.mark.parametrize("tokens,topk,experts,align,width,dtype,ids,how,pad,shift", EXCHANGE)
def test_exchange(tokens, topk, experts, align, width, dtype, ids, how, pad, shift):
    rng = np.random.default_rng(tokens * 131 + topk)
    x, x64 = rows_of(rng, tokens, width, dtype, pad, shift)
    e, e_host = routing(rng, tokens, topk, experts, how, ids)
    cap = ref.capacity(tokens, topk, experts, align)
    assert gc.expert_rows(tokens, topk, experts, align) == cap
    offsets, counts, slots, pairs = ref.plan(e_host, experts, align, cap)
    out, plan = gc.expert_dispatch(x, e, experts, align=align)
    for got, want in zip(plan, (offsets, counts, slots, pairs)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(out.double().cpu().numpy(), ref.dispatch(x64, pairs, topk))
    only, again = gc.expert_dispatch(None, e, experts, align=align)
    assert only is None and all(torch.equal(a, b) for a, b in zip(plan, again))

    y, y64 = rows_of(rng, cap, width, dtype, pad, shift)
    g, g64 = rows_of(rng, tokens, width, dtype, pad, shift)
    w64 = rng.random((tokens, topk)).astype(np.float32)
    w = torch.from_numpy(w64).cuda()
    for weights, host in ((w, w64), (None, None)):
        want, size = ref.combine(y64, slots, host)
        got = gc.expert_combine(y, plan.slots, weights)
        assert off(got, want, size, topk, dtype) <= 1
    assert torch.equal(gc.expert_dispatch_grad(y, plan.slots), got)
    for weights, host in ((None, None), (w, w64)):
        dy, dw, size = ref.combine_grad(g64, y64, slots, pairs, host)
        got_y, got_w = gc.expert_combine_grad(g, y, plan.slots, plan.pairs, weights)
        assert off(got_y, dy, np.abs(dy), 0, dtype) <= 1
        assert off(got_w, dw, size, width, "f32") <= 1
    alone, none = gc.expert_combine_grad(g, None, plan.slots, plan.pairs, w)
    assert none is None and torch.equal(alone, got_y)


def test_exchange_rows_beyond_the_need_and_strided_outputs():
    # 5 rows more than any routing needs, and outputs that are slices of wider rows, whose rest stays.
    rng = np.random.default_rng(5)
    x, x64 = rows_of(rng, 50, 24, "bf16")
    e, e_host = routing(rng, 50, 3, 6, "drop", "i32")
    rows = gc.expert_rows(50, 3, 6, 4) + 5
    plan = gc.ExpertPlan(*(torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (7, 6, 150, rows)))
    wide = torch.full((rows, 40), 9.0, dtype=torch.bfloat16, device="cuda")
    gc.expert_dispatch(x, e, 6, align=4, out=wide[:, 8:32], plan=plan)
    _, _, slots, pairs = ref.plan(e_host, 6, 4, rows)
    assert np.array_equal(plan.pairs.cpu().numpy(), pairs)
    assert np.array_equal(wide[:, 8:32].double().cpu().numpy(), ref.dispatch(x64, pairs, 3))
    assert bool((wide[:, :8] == 9).all()) and bool((wide[:, 32:] == 9).all())
    back = torch.full((50, 30), 9.0, dtype=torch.bfloat16, device="cuda")
    gc.expert_combine(wide[:, 8:32], plan.slots.view(50, 3), None, out=back[:, 3:27])
    want, size = ref.combine(ref.dispatch(x64, pairs, 3), slots, None)
    assert off(back[:, 3:27], want, size, 3, "bf16") <= 1
    assert bool((back[:, :3] == 9).all()) and bool((back[:, 27:] == 9).all())


def test_exchange_without_tokens():
    x = torch.empty(0, 16, device="cuda")
    ids = torch.empty(0, 2, dtype=torch.int64, device="cuda")
    out, plan = gc.expert_dispatch(x, ids, 4, align=8)
    assert out.shape == (0, 16) and not plan.offsets.any() and not plan.counts.any()
    assert gc.expert_combine(out, plan.slots).shape == (0, 16)
    rows = gc.ExpertPlan(*(torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in (5, 4, 0, 3)))
    out, _ = gc.expert_dispatch(x, ids, 4, align=8, out=torch.ones(3, 16, device="cuda"), plan=rows)
    assert not out.any() and bool((rows.pairs == -1).all()) and not rows.offsets.any()


def test_indices_out_of_range_select_nothing():
    # A plan that does not fit the arrays is never followed out of them.
    y = torch.randn(6, 32, device="cuda")
    slots = torch.tensor([[0, 6], [2 ** 31 - 1, -5]], dtype=torch.int32, device="cuda")
    out = gc.expert_combine(y, slots)
    assert torch.equal(out[0], y[0]) and not out[1].any()
    pairs = torch.tensor([0, 4, -9, 2 ** 31 - 1, -1, -1], dtype=torch.int32, device="cuda")
    dy, dw = gc.expert_combine_grad(torch.ones(2, 32, device="cuda"), y, slots, pairs)
    assert bool((dy[0] == 1).all()) and not dy[1:].any()
    assert not dw[1].any() and dw[0, 1] == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_rows_do_not_leak(dtype):
    # Infinities and NaN in rows that no pair points to stay out of every sum.
    y = torch.full((8, 48), float("nan"), dtype=DTYPES[dtype], device="cuda")
    y[3] = 1.0
    slots = torch.tensor([[3, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    pairs = torch.tensor([-1, -1, -1, 0, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    out = gc.expert_combine(y, slots, torch.tensor([[0.5, float("nan")], [float("inf"), 1.0]], device="cuda"))
    assert bool((out[0] == 0.5).all()) and not out[1].any()
    dy, dw = gc.expert_combine_grad(torch.ones(2, 48, dtype=DTYPES[dtype], device="cuda"), y, slots, pairs)
    assert bool((dy[3] == 1).all()) and not dy[:3].any() and not dy[4:].any()
    assert dw.tolist() == [[48.0, 0.0], [0.0, 0.0]]


def test_exchange_gradients_against_differences():
    # combine is linear in y and in the weights, and dispatch in x: a central
    # difference with step h is exact but for the rounding of the two results,
    # 2^-24 * 2 * 3 terms * magnitudes, over 2 h.
    rng = np.random.default_rng(11)
    tokens, topk, width, experts = 40, 3, 65, 5
    e, _ = routing(rng, tokens, topk, experts, "drop", "i64")
    x, _ = rows_of(rng, tokens, width, "f32")
    g, g64 = rows_of(rng, tokens, width, "f32")
    w = torch.rand(tokens, topk, device="cuda")
    rows, plan = gc.expert_dispatch(x, e, experts, align=4)
    y, _ = rows_of(rng, rows.shape[0], width, "f32")
    dy, dw = gc.expert_combine_grad(g, y, plan.slots, plan.pairs, w)
    by, bw, bx = torch.randn_like(y), torch.randn_like(w), torch.randn_like(x)
    h = 0.25

    def loss(fn, a, b):
        return ((fn(a).double() - fn(b).double()) * g.double()).sum().item() / (2 * h)

    scale = g.double().abs().sum().item() * 64 * 2.0 ** -24 / h
    num = loss(lambda v: gc.expert_combine(v, plan.slots, w), y + h * by, y - h * by)
    assert abs(num - (dy.double() * by.double()).sum().item()) <= scale
    num = loss(lambda v: gc.expert_combine(y, plan.slots, v), w + h * bw, w - h * bw)
    assert abs(num - (dw.double() * bw.double()).sum().item()) <= scale
    gr, _ = rows_of(rng, rows.shape[0], width, "f32")
    hi, lo = (gc.expert_dispatch(x + k * bx, e, experts, align=4)[0] for k in (h, -h))
    num = ((hi.double() - lo.double()) * gr.double()).sum().item() / (2 * h)
    got = (gc.expert_dispatch_grad(gr, plan.slots).double() * bx.double()).sum().item()
    assert abs(num - got) <= gr.double().abs().sum().item() * 64 * 2.0 ** -24 / h


# n, vocab, width, dtype, out, ids, spread, pad, shift
EMBED = [
    (1, 1, 1, "f32", "f32", "i32", "all", 0, 0),
    (1, 300000, 64, "bf16", "f32", "i64", "all", 0, 0),
    (7, 3, 33, "f16", "f16", "i64", "outside", 1, 1),
    (300, 1, 129, "bf16", "bf16", "i32", "all", 0, 0),
    (1023, 511, 96, "f32", "f32", "i64", "zipf", 0, 0),
    (1025, 512, 31, "bf16", "f32", "i32", "outside", 5, 0),
    (5000, 70000, 24, "f16", "f32", "i64", "zipf", 8, 8),
    (5000, 262143, 8, "bf16", "bf16", "i32", "zipf", 0, 0),
    (5000, 300001, 12, "f32", "f32", "i64", "all", 0, 4),
    (3000, 10, 520, "bf16", "f32", "i64", "one", 0, 0),
    (9000, 50, 2050, "bf16", "f32", "i32", "zipf", 0, 0),
    (66000, 1000, 16, "f16", "f16", "i32", "zipf", 0, 0),
]


def token_ids(rng, n, vocab, spread, ids):
    if spread == "one":
        v = np.full(n, vocab // 2)
        v[::97] = -1
    elif spread == "zipf":
        v = np.minimum(np.exp(rng.random(n) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
    elif spread == "outside":
        v = rng.integers(-vocab, 2 * vocab, n)
    else:
        v = rng.integers(0, vocab, n)
    return torch.from_numpy(v.astype(np.int64 if ids == "i64" else np.int32)).cuda(), v


@pytest.mark.parametrize("n,vocab,width,dtype,odt,ids,spread,pad,shift", EMBED)
def test_embedding(n, vocab, width, dtype, odt, ids, spread, pad, shift):
    rng = np.random.default_rng(n + vocab)
    table, t64 = rows_of(rng, vocab, width, dtype, pad, shift)
    v, v_host = token_ids(rng, n, vocab, spread, ids)
    for scale in (1.0, 22.627417):
        want = ref.embedding(t64, v_host, scale)
        got = gc.embedding(table, v, scale=scale)
        assert off(got, want, np.abs(want), 0 if scale == 1.0 else 1, dtype) <= (0 if scale == 1.0 else 1)
    assert torch.equal(gc.embedding(table, v.view(1, n), scale=scale)[0], got)

    g, g64 = rows_of(rng, n, width, dtype, pad, shift)
    want, size, count = ref.embedding_grad(g64, v_host, vocab, scale)
    got = gc.embedding_grad(g, v, vocab, scale=scale, out_dtype=DTYPES[odt])
    assert off(got, want, size, count[:, None], odt) <= 1
    assert torch.equal(got, gc.embedding_grad(g, v, vocab, scale=scale, out_dtype=DTYPES[odt]))
    # added to what is there, absent tokens' rows left as they are
    there, there64 = rows_of(rng, vocab, width, odt)
    sums, keep = there.clone(), torch.from_numpy(count == 0).cuda()
    gc.embedding_grad(g, v, vocab, scale=scale, out=sums, accumulate=True)
    assert off(sums, want + there64, size + np.abs(there64), count[:, None] + 1, odt) <= 1
    assert torch.equal(sums[keep], there[keep])


def test_embedding_nothing():
    table = torch.randn(5, 8, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert gc.embedding(table, none).shape == (0, 8)
    out = torch.ones(5, 8, device="cuda")
    gc.embedding_grad(torch.empty(0, 8, device="cuda"), none, 5, out=out, accumulate=True)
    assert bool((out == 1).all())
    gc.embedding_grad(torch.empty(0, 8, device="cuda"), none, 5, out=out)
    assert not out.any()


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(3)
    table, _ = rows_of(rng, 30, 40, "f32")
    v, _ = token_ids(rng, 200, 30, "outside", "i64")
    g, _ = rows_of(rng, 200, 40, "f32")
    d, h = torch.randn_like(table), 0.25
    up, down = (gc.embedding(table + k * d, v, scale=3.0).double() for k in (h, -h))
    num = ((up - down) * g.double()).sum().item() / (2 * h)
    got = (gc.embedding_grad(g, v, 30, scale=3.0).double() * d.double()).sum().item()
    assert abs(num - got) <= g.double().abs().sum().item() * 64 * 2.0 ** -24 * 3 / h


def test_embedding_grad_strided_output_keeps_its_surroundings():
    rng = np.random.default_rng(8)
    g, g64 = rows_of(rng, 90, 20, "bf16")
    v, host = token_ids(rng, 90, 12, "zipf", "i32")
    wide = torch.full((12, 27), 5.0, device="cuda")
    gc.embedding_grad(g, v, 12, out=wide[:, 3:23])
    want, size, count = ref.embedding_grad(g64, host, 12, 1.0)
    assert off(wide[:, 3:23], want, size, count[:, None], "f32") <= 1
    assert bool((wide[:, :3] == 5).all()) and bool((wide[:, 23:] == 5).all())


PARAMS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (0.8, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.9, 40, 0.95, 0.01),
          (0.0, 5, 0.5, 0.5), (1.3, 1, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (0.5, 0, 1.0, 1.0), (2.0, 3, 0.6, 0.0),
          (1.0, 300, 0.99, 0.0), (0.01, 0, 0.3, 0.0), (1.0, -4, 1.5, -1.0), (50.0, 0, 0.97, 0.0),
          (float("nan"), 0, 1.0, 0.0), (1.0, 2 ** 31 - 1, 1.0, 2.0)]


def check_sample(x, x64, u, params, vocab):
    """Tokens equal; log probabilities within the rounding of z, of the weights and of their sum."""
    t, k, p, q = zip(*params)
    col = lambda v, d: torch.tensor(v, dtype=d, device="cuda")  # noqa: E731
    tokens, logprobs = gc.sample(x, u, temperature=col(t, torch.float32), top_k=col(k, torch.int32),
                                 top_p=col(p, torch.float32), min_p=col(q, torch.float32))
    tokens, logprobs, u64 = tokens.cpu().numpy(), logprobs.double().cpu().numpy(), u.double().cpu().numpy()
    f = lambda v: float(np.float32(v))  # noqa: E731
    for r in range(x64.shape[0]):
        want, lp, z = ref.sample(x64[r], u64[r], f(t[r]), k[r], f(p[r]), f(q[r]))
        assert tokens[r] == want, (r, params[r])
        if np.isinf(lp):
            assert logprobs[r] == lp
        else:
            tol = 2.0 ** -22 * (abs(z) + 16) + (vocab / 1024 + 12) * 2.0 ** -24 + 2.0 ** -23 * abs(lp)
            assert abs(logprobs[r] - lp) <= tol, (r, params[r], logprobs[r], lp)


def logits_of(rng, rows, vocab, dtype, kind, pad, shift):
    x = rng.standard_normal((rows, vocab + pad + shift)).astype(np.float32) * 2.5
    if kind == "peaked":
        for r in range(rows):
            x[r, rng.integers(0, x.shape[1], 20)] += 12 * rng.random(20)
    elif kind == "flat":
        x[:] = 1.5
    elif kind == "steps":
        x = np.round(x)
    elif kind == "masked":
        x[rng.random(x.shape) < 0.9] = -np.inf
    elif kind == "lowest":
        x[rng.random(x.shape) < 0.9] = torch.finfo(DTYPES[dtype]).min
    elif kind == "far":
        x *= 40
    elif kind == "broken":
        # NaN and -inf among the logits, and in every third row some infinities
        x[rng.random(x.shape) < 0.2] = np.nan
        x[rng.random(x.shape) < 0.1] = -np.inf
        for r in range(0, rows, 3):
            x[r, rng.integers(0, x.shape[1], 3)] = np.inf
    wide = torch.from_numpy(x).to(DTYPES[dtype])
    return wide.cuda()[:, shift:shift + vocab], wide[:, shift:shift + vocab].double().numpy()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["bulk", "peaked", "flat", "steps", "masked", "lowest", "far", "broken"])
@pytest.mark.parametrize("vocab,pad,shift", [(1, 0, 0), (2, 3, 1), (33, 0, 0), (1000, 1, 1), (4096, 0, 8),
                                             (5003, 5, 2), (40001, 0, 0)])
def test_sample(vocab, pad, shift, kind, dtype):
    rng = np.random.default_rng(vocab * 7 + len(kind))
    x, x64 = logits_of(rng, len(PARAMS), vocab, dtype, kind, pad, shift)
    u = torch.from_numpy(rng.random((len(PARAMS), vocab + pad)).astype(np.float32)).clamp_(max=1 - 2.0 ** -24).cuda()
    check_sample(x, x64, u[:, :vocab], PARAMS, vocab)


@pytest.mark.parametrize("kind", ["bulk", "flat", "lowest", "far", "broken"])
@pytest.mark.parametrize("vocab,dtype", [(64, "f32"), (65, "bf16"), (1024, "f16"), (1025, "f32"), (4095, "f32"),
                                         (4097, "bf16")])
def test_sample_many_short_rows(vocab, dtype, kind):
    rng = np.random.default_rng(vocab + len(kind))
    params = [(t, k, p, q) for t in (0.02, 1.0, 5.0) for k in (0, 64, 257, 513) for p in (1.0, 0.9, 0.4)
              for q in (0.0, 0.02)] * 3
    x, x64 = logits_of(rng, len(params), vocab, dtype, kind, 3, 0)
    u = torch.from_numpy(rng.random((len(params), vocab)).astype(np.float32)).clamp_(max=1 - 2.0 ** -24).cuda()
    check_sample(x, x64, u, params, vocab)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 262147), ("f32", 131072), ("f16", 200001)])
def test_sample_large_vocabulary(dtype, vocab):
    rng = np.random.default_rng(vocab)
    for kind in ("peaked", "bulk"):
        x, x64 = logits_of(rng, len(PARAMS), vocab, dtype, kind, 0, 0)
        u = torch.rand(len(PARAMS), vocab, device="cuda")
        check_sample(x, x64, u, PARAMS, vocab)


@pytest.mark.parametrize("rows", [1, 2, 5, 150, 700])
def test_sample_batches(rows):
    rng = np.random.default_rng(rows)
    x, x64 = logits_of(rng, rows, 9000, "bf16", "peaked", 0, 0)
    u = torch.rand(rows, 9000, device="cuda")
    check_sample(x, x64, u, [PARAMS[r % len(PARAMS)] for r in range(rows)], 9000)


def test_sample_special_values():
    inf, nan, low = float("inf"), float("nan"), -3.4028234663852886e38
    x = torch.tensor([[-inf] * 6, [nan] * 6, [-inf, nan, 1.0, -inf, nan, -inf], [0.0, inf, 5.0, inf, nan, -inf],
                      [low] * 6, [-0.0, 0.0, -0.0, -1.0, -1.0, -2.0], [low, 3.4028234663852886e38, low, 0, 0, 0]],
                     device="cuda")
    u = torch.full((7, 6), 0.5, device="cuda")
    tokens, logprobs = gc.sample(x, u)
    assert tokens.tolist() == [-1, -1, 2, 1, 0, 0, 1]
    want = [-inf, -inf, 0.0, np.log(0.5), np.log(1 / 6), -np.log(3 + 2 * np.exp(-1) + np.exp(-2)), 0.0]
    got = logprobs.double().cpu().numpy()
    assert np.array_equal(np.isinf(got), np.isinf(want))
    fine = np.isfinite(want)
    assert np.max(np.abs(got[fine] - np.array(want)[fine])) <= 2.0 ** -19
    # equal values: the lowest index is first, -0 and +0 are equal
    assert gc.sample(x)[0].tolist() == [-1, -1, 2, 1, 0, 0, 1]
    assert gc.sample(x[5:6].expand(1, 6), u[:1], top_k=1)[0].item() == 0
    # the random numbers' ends and NaN
    v = torch.tensor([[0.0, 1.0, nan, 2.0, -1.0, 0.5]], device="cuda")
    assert gc.sample(torch.zeros(1, 6, device="cuda"), v)[0].item() == 1
    assert gc.sample(torch.zeros(1, 6, device="cuda"), torch.full((1, 6), nan, device="cuda"))[0].item() == 0


def test_sample_frequencies():
    # 60000 draws of 6 tokens, top-p cutting the last two: each frequency within 5 standard deviations.
    p = np.array([0.4, 0.25, 0.15, 0.12, 0.05, 0.03])
    n = 60000
    x = torch.from_numpy(np.log(p)).float().cuda().expand(n, 6).contiguous()
    gen = torch.Generator(device="cuda").manual_seed(9)
    tokens, logprobs = gc.sample(x, torch.rand(n, 6, generator=gen, device="cuda"), top_p=0.9)
    kept = np.array([0.4, 0.25, 0.15, 0.12, 0, 0]) / 0.92
    seen = np.bincount(tokens.cpu().numpy(), minlength=6) / n
    assert np.all(np.abs(seen - kept) <= 5 * np.sqrt(kept * (1 - kept) / n))
    assert np.allclose(logprobs.cpu().numpy(), np.log(kept[tokens.cpu().numpy()]), atol=1e-5)


def test_row_operators_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(4)
    x, _ = rows_of(rng, 300, 128, "bf16")
    table, _ = rows_of(rng, 500, 128, "bf16")
    logits, _ = rows_of(rng, 4, 500, "f32")
    u = torch.rand(4, 500, device="cuda")
    e, _ = routing(rng, 300, 2, 9, "drop", "i64")
    ids = torch.randint(500, (300,), device="cuda")
    w = torch.rand(300, 2, device="cuda")

    def step(stream=None):
        h = gc.embedding(table, ids, scale=2.0, stream=stream)
        rows, plan = gc.expert_dispatch(x, e, 9, align=8, stream=stream)
        out = gc.expert_combine(rows, plan.slots, w, stream=stream)
        dy, dw = gc.expert_combine_grad(x, rows, plan.slots, plan.pairs, w, stream=stream)
        dx = gc.expert_dispatch_grad(dy, plan.slots, stream=stream)
        dt = gc.embedding_grad(x, ids, 500, out_dtype=torch.float32, stream=stream)
        tok, lp = gc.sample(logits, u, temperature=0.9, top_k=20, top_p=0.9, stream=stream)
        return [h, rows, *plan, out, dy, dw, dx, dt, tok, lp]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    got = step(side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.mul_(0.5), ids.copy_(ids.flip(0)), e.copy_(e.flip(0)), logits.add_(torch.randn_like(logits))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_offsets_beyond_32_bits():
    # Rows whose element offsets pass 2^32: the last of a large table, its
    # gradient, and logits whose rows lie 2^31 - 16 elements apart.
    vocab, width = 1_100_000, 4096
    table = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, vocab - 2, vocab, vocab - 1], device="cuda")
    table[ids[:3]] = torch.arange(3, device="cuda", dtype=torch.bfloat16).unsqueeze(1) + 1
    out = gc.embedding(table, ids)
    assert out[:, 0].tolist() == [1.0, 2.0, 3.0, 0.0, 1.0] and bool((out == out[:, :1]).all())
    g = torch.ones(5, width, dtype=torch.bfloat16, device="cuda")
    table.fill_(7.0)
    gc.embedding_grad(g, ids, vocab, out=table)
    assert table[ids[:3], 5].tolist() == [2.0, 1.0, 1.0] and not table[1:vocab - 2].any()
    del table
    stride, vocab = 2 ** 31 - 16, 5001
    wide = torch.full((2 * stride + vocab,), -9.0, dtype=torch.bfloat16, device="cuda")
    x = wide.as_strided((3, vocab), (stride, 1))
    x[2, 4321] = 30.0
    u = torch.rand(3, vocab, device="cuda")
    assert gc.sample(x)[0].tolist() == [0, 0, 4321]
    assert gc.sample(x, u, top_p=0.9)[0][2].item() == 4321
    y = wide.as_strided((3, 64), (stride, 1))
    slots = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    assert bool((gc.expert_combine(y, slots)[0] == -18.0).all())


def test_example_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "language_model_step.py")
    spec = importlib.util.spec_from_file_location("language_model_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Model(vocab=300, width=64, experts=5, topk=2, align=8)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(300, (90,), generator=g, device="cuda")
    targets = (ids * 7 + 3) % 300
    # the gradient along itself against a central difference: the loss is
    # smooth but for the choice of experts, which a step of 1e-3 leaves alone;
    # float32 sums of the loss leave about 1e-6 / 1e-3 of noise
    loss, d_logits, saved = model.loss(ids, targets)
    grads = model.backward(d_logits, saved)
    for name, grad in grads.items():
        d = grad / grad.norm()
        ends = []
        for h in (1e-3, -1e-3):
            model.params[name] += h * d
            ends.append(model.loss(ids, targets)[0].double().item())
            model.params[name] -= h * d
        assert abs((ends[0] - ends[1]) / 2e-3 - grad.norm().item()) <= 0.02 * grad.norm().item() + 2e-3, name
    first = loss.item()
    for _ in range(60):
        last = model.train_step(ids, targets).item()
    assert last < 0.5 * first
    tokens, logprobs = model.sample(ids, g)
    assert tokens.shape == (90,) and bool((logprobs <= 0).all())
