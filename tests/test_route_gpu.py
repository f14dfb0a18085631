"""Routing and its gradient on the GPU against plain 64-bit forms (more_rows_ref.py).

Tolerances, from the arithmetic, with |z| the distance of a logit from its
token's largest and e = 2^-24: a probability is 2^y / sum of 2^y, y = z log2(e).
y takes two roundings of its own and one of the constant, so 2^y is off by
3 |z| e of itself, and 4 e more by the approximation of 2^y (2^-22); the sum by
the mean of that over its terms, with at most 64 + 5 additions of e; the
quotient by 3 e.  Weights over their sum: the same once more with at most 64
additions.  Elements below 2^-126 may be 0.  Sums over tokens and experts: one 2^-24 for each addition on
a term's way, of terms that are not negative."""

import numpy as np
import pytest
import torch

import more_rows_ref as ref
from partition_pass_tile_gb300 import gc
from rows_ref import TINY, UNIT

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def logits_of(rng, tokens, experts, dtype, forbidden=0.0, pad=0, shift=0, scale=2.0):
    """Logits on the GPU (a slice of wider rows, `shift` elements in) and the values they hold."""
    x = (scale * rng.standard_normal((tokens, experts + pad + shift))).astype(np.float32)
    x[rng.random(x.shape) < forbidden] = -np.inf
    wide = torch.from_numpy(x).to(DTYPES[dtype])
    return wide.cuda()[:, shift:shift + experts], wide[:, shift:shift + experts].double().numpy()


def relative(p, z):
    """Of each probability: how far off it may be."""
    return (3 * z + 4 + (p * (3 * z + 4)).sum(-1, keepdims=True) + 72) * E


def terms(tokens, experts):
    """Additions of float32 on the way of a token to a sum over tokens: its thread's, its CTA's and the CTAs'."""
    if experts > 32:
        groups, most = (16, 304) if experts <= 256 else (8, 304) if experts <= 512 else (8, 152)
    else:
        groups, most = 256 // (1 if experts <= 8 else 2 if experts <= 16 else 4), 456
    # one CTA alone takes up to twice its tokens
    groups = groups if -(-tokens // groups) > 2 else max(1, groups // 2)
    grid = min(-(-tokens // groups), most)
    return -(-tokens // (grid * groups)) + 64


def check_route(r, x64, topk, normalize, mask):
    ids, weights, counts, load, loss, p, z = ref.route(x64, topk, normalize, mask)
    tokens, experts = x64.shape
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    rel = relative(p, z)
    at = np.maximum(ids, 0)
    own = np.take_along_axis(rel, at, 1) + (rel.max(1, keepdims=True) + 72 * E if normalize else 0.0)
    got = r.weights.double().cpu().numpy()
    assert np.all(np.abs(got - weights) <= own * weights + 2.0 ** -126)
    n = max(counts[experts], 1)
    off = (p * rel).sum(0) / n + (terms(tokens, experts) + 1) * E * load + 2.0 ** -126
    assert np.all(np.abs(r.load.double().cpu().numpy() - load) <= off)
    share = counts[:experts] / max(counts[:experts].sum(), 1)
    # its sum over the experts: at most 64 additions of one thread, 10 of its CTA, 8 of the CTAs', and three products
    assert abs(float(r.loss) - loss) <= experts * float(share @ off) + 85 * E * loss
    return ids, counts


# tokens, experts, topk, dtype, normalize, masked, forbidden, pad, shift
ROUTE = [
    (1, 1, 1, "f32", True, 0.0, 0.0, 0, 0),
    (1, 64, 4, "bf16", False, 0.0, 0.0, 0, 0),
    (3, 2, 2, "f16", True, 0.0, 0.5, 3, 1),
    (24, 64, 4, "f32", True, 0.0, 0.0, 0, 0),
    (33, 7, 3, "bf16", False, 0.4, 0.3, 1, 2),
    (100, 8, 8, "bf16", True, 0.0, 0.2, 0, 0),
    (255, 9, 1, "f32", False, 0.1, 0.0, 0, 0),
    (257, 16, 2, "f16", True, 0.0, 0.0, 8, 8),
    (1000, 60, 6, "f16", False, 0.2, 0.1, 5, 0),
    (513, 128, 64, "bf16", True, 0.0, 0.0, 0, 0),
    (700, 256, 8, "f32", True, 0.0, 0.0, 0, 0),
    (300, 257, 5, "bf16", False, 0.1, 0.2, 0, 0),
    (130, 512, 10, "f32", True, 0.0, 0.0, 0, 4),
    (90, 1000, 33, "f16", False, 0.0, 0.0, 0, 0),
    (70, 2048, 64, "bf16", True, 0.1, 0.9, 0, 0),
    (40, 2047, 64, "f32", False, 0.0, 0.0, 0, 0),
    (20000, 4, 2, "bf16", True, 0.1, 0.0, 0, 0),
    (2001, 33, 12, "f32", True, 0.0, 0.0, 0, 0),
    (500, 64, 13, "bf16", False, 0.1, 0.0, 0, 0),
    (1777, 65, 6, "f16", True, 0.0, 0.4, 0, 0),
    (3001, 128, 8, "bf16", True, 0.0, 0.0, 0, 0),
    (600, 129, 2, "f32", False, 0.3, 0.9, 3, 1),
    (800, 256, 12, "bf16", True, 0.0, 0.99, 0, 0),
    (300, 200, 16, "f32", True, 0.0, 0.0, 0, 0),
    (20000, 256, 8, "f32", True, 0.05, 0.0, 0, 0),
    (15000, 100, 4, "bf16", False, 0.0, 0.1, 0, 0),
    (12000, 300, 3, "f16", True, 0.0, 0.0, 0, 0),
    (9000, 32, 4, "f32", False, 0.0, 0.0, 0, 0),
]


@pytest.mark.parametrize("tokens,experts,topk,dtype,normalize,masked,forbidden,pad,shift", ROUTE)
def test_route_and_gradient(tokens, experts, topk, dtype, normalize, masked, forbidden, pad, shift):
    rng = np.random.default_rng(tokens * 31 + experts)
    x, x64 = logits_of(rng, tokens, experts, dtype, forbidden, pad, shift)
    mask = rng.random(tokens) >= masked if masked else None
    m = None if mask is None else torch.from_numpy(mask).cuda()
    r = gc.expert_route(x, topk, normalize=normalize, mask=m)
    ids, counts = check_route(r, x64, topk, normalize, mask)
    alone = gc.expert_route(x, topk, normalize=normalize, mask=m, balance=False)
    assert torch.equal(alone.ids, r.ids) and torch.equal(alone.weights, r.weights)
    assert alone.counts is None and alone.load is None and alone.loss is None

    g, dl = rng.standard_normal((tokens, topk)).astype(np.float32), np.float32(0.3)
    masked64 = ref.clean(x64) if mask is None else np.where(mask[:, None], ref.clean(x64), -np.inf)
    p, z = ref.softmax(masked64)
    rel = relative(p, z)
    rel = rel + rel.max(1, keepdims=True) + (2 * topk + 160) * E  # the sums <p, a>, <w, g>, their differences
    for dw, loss in ((g, None), (None, dl), (g, dl)):
        want, size = ref.route_grad(x64, ids, counts, dw, loss, normalize)
        got = gc.expert_route_grad(x, r.ids, r.counts, dweights=None if dw is None else torch.from_numpy(dw).cuda(),
                                   dloss=None if loss is None else torch.full((1,), float(loss), device="cuda"),
                                   normalize=normalize)
        assert got.dtype == x.dtype
        bound = rel * size * (1 + 2 * UNIT[dtype]) + UNIT[dtype] * np.abs(want) + TINY[dtype] + 2.0 ** -120
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)
    assert not gc.expert_route_grad(x, r.ids, normalize=normalize).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_and_forbidden_logits(dtype):
    # equal values go by index; NaN and -inf close an expert, +inf counts as the largest finite value
    inf, nan = float("inf"), float("nan")
    rows = [[1.0] * 9, [-inf] * 9, [nan] * 9, [-inf, 2, nan, 2, -inf, 2, nan, -inf, -inf], [inf, 1, inf, 0, 0, 0, 0, 0, 0],
            [0.0, -0.0, 0.0, -0.0, -1, -1, -1, -1, -1], [-inf, -inf, -inf, -inf, -inf, -inf, -inf, -inf, -3e4]]
    x = torch.tensor(rows, device="cuda").to(DTYPES[dtype])
    r = gc.expert_route(x, 4)
    assert r.ids.tolist() == [[0, 1, 2, 3], [-1] * 4, [-1] * 4, [1, 3, 5, -1], [0, 2, 1, 3], [0, 1, 2, 3], [8, -1, -1, -1]]
    want = [[0.25] * 4, [0] * 4, [0] * 4, [1 / 3] * 3 + [0], [0.5, 0.5, 0, 0], [0.25] * 4, [1, 0, 0, 0]]
    assert np.all(np.abs(r.weights.cpu().numpy() - np.array(want)) <= 8 * E)
    assert r.counts.tolist() == [3, 4, 3, 4, 0, 1, 0, 0, 1, 5]
    check_route(r, x.double().cpu().numpy(), 4, True, None)
    dx = gc.expert_route_grad(x, r.ids, r.counts, dweights=torch.ones_like(r.weights),
                              dloss=torch.ones(1, device="cuda"))
    assert bool(torch.isfinite(dx).all()) and not dx[1:3].any()


def test_masked_tokens_do_not_leak():
    x = torch.full((40, 16), float("nan"), device="cuda")
    x[::3] = torch.randn(14, 16, device="cuda")
    x[1::3] = float("inf")
    mask = torch.zeros(40, dtype=torch.bool, device="cuda")
    mask[::3] = True
    r = gc.expert_route(x, 3, mask=mask)
    check_route(r, x.double().cpu().numpy(), 3, True, mask.cpu().numpy())
    dw = torch.full((40, 3), float("nan"), device="cuda")
    dw[::3] = 1.0
    dx = gc.expert_route_grad(x, r.ids, r.counts, dweights=dw, dloss=torch.ones(1, device="cuda"))
    assert bool(torch.isfinite(dx).all()) and not dx[1::3].any() and not dx[2::3].any() and dx[::3].any()


def test_no_tokens():
    r = gc.expert_route(torch.empty(0, 8, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and not r.counts.any() and not r.load.any() and not r.loss.any()
    r = gc.expert_route(torch.randn(5000, 8, device="cuda"), 2, mask=torch.zeros(5000, dtype=torch.bool, device="cuda"))
    assert bool((r.ids == -1).all()) and not r.weights.any() and not r.counts.any()
    assert not r.load.any() and not r.loss.any()
    assert gc.expert_route_grad(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 8)


@pytest.mark.parametrize("normalize", [True, False])
def test_ids_outside_or_twice(normalize):
    # ids that are no expert have no part, one that occurs twice has both, whatever expert_route would have chosen
    rng = np.random.default_rng(8)
    x, x64 = logits_of(rng, 6, 20, "f32")
    ids = np.array([[3, 3, 3], [0, -1, 25], [-1, 2, 3], [19, 2 ** 31 - 1, 19], [5, 4, 5], [20, 1, 1]], np.int32)
    g = rng.standard_normal(ids.shape).astype(np.float32)
    counts = np.arange(21).astype(np.int32)
    want, size = ref.route_grad(x64, ids, counts, g, 0.5, normalize)
    got = gc.expert_route_grad(x, torch.from_numpy(ids).cuda(), torch.from_numpy(counts).cuda(),
                               dweights=torch.from_numpy(g).cuda(), dloss=torch.full((1,), 0.5, device="cuda"),
                               normalize=normalize).double().cpu().numpy()
    p, z = ref.softmax(x64)
    rel = relative(p, z)
    assert np.all(np.abs(got - want) <= (rel + rel.max(1, keepdims=True) + 180 * E) * size + E * np.abs(want))


def test_gradient_against_differences():
    # a central difference of step h is off by h^2 times a third derivative,
    # which for products of softmaxes is below 8 * the sum of |gradients|, and by
    # the roundings of two values, 2^-22 * magnitudes * |z| / h
    rng = np.random.default_rng(4)
    x, _ = logits_of(rng, 50, 12, "f32", scale=1.0)
    g = torch.from_numpy(rng.standard_normal((50, 3)).astype(np.float32)).cuda()
    by = torch.from_numpy(rng.standard_normal((50, 12)).astype(np.float32)).cuda()
    h = 2.0 ** -8
    for normalize in (True, False):
        r = gc.expert_route(x, 3, normalize=normalize)
        # the choices have to stay the same: move only tokens whose order is clear
        s = x.sort(1).values
        clear = ((s[:, 1:] - s[:, :-1]).amin(1) > 4 * h * by.abs().amax(1)).unsqueeze(1)
        step = torch.where(clear, by, 0.0)
        dx = gc.expert_route_grad(x, r.ids, r.counts, dweights=g, dloss=torch.full((1,), 5.0, device="cuda"),
                                  normalize=normalize)

        def value(y):
            q = gc.expert_route(y, 3, normalize=normalize)
            assert torch.equal(q.ids, r.ids)
            return (q.weights.double() * g.double()).sum().item() + 5.0 * q.loss.double().item()
        num = (value(x + h * step) - value(x - h * step)) / (2 * h)
        size = g.abs().sum().item() + 5.0 * 12
        assert clear.sum() > 5
        assert abs(num - (dx.double() * step.double()).sum().item()) <= size * (8 * h * h * by.abs().amax().item() ** 3 + 2.0 ** -22 * 8 / h)


def test_strided_gradient_and_given_outputs():
    rng = np.random.default_rng(6)
    x, x64 = logits_of(rng, 77, 30, "bf16", pad=10, shift=2)
    out = gc.Routing(torch.empty(77, 2, dtype=torch.int32, device="cuda"), torch.empty(77, 2, device="cuda"),
                     torch.empty(31, dtype=torch.int32, device="cuda"), torch.empty(30, device="cuda"),
                     torch.empty(1, device="cuda"))
    r = gc.expert_route(x, 2, out=out)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(r, out))
    check_route(r, x64, 2, True, None)
    wide = torch.full((77, 50), 9.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.randn(77, 2, device="cuda")
    got = gc.expert_route_grad(x, r.ids, r.counts, dweights=dw, out=wide[:, 7:37])
    assert torch.equal(got, gc.expert_route_grad(x.contiguous(), r.ids, r.counts, dweights=dw))
    assert bool((wide[:, :7] == 9).all()) and bool((wide[:, 37:] == 9).all())


def test_repeats_streams_and_graphs():
    x = torch.randn(30000, 96, device="cuda")
    first = gc.expert_route(x, 6)
    g = torch.randn(30000, 6, device="cuda")
    dl = torch.ones(1, device="cuda")
    dx = gc.expert_route_grad(x, first.ids, first.counts, dweights=g, dloss=dl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = gc.expert_route(x, 6)
    third = gc.expert_route(x, 6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, again, third))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = gc.expert_route(x, 6)
        d = gc.expert_route_grad(x, r.ids, r.counts, dweights=g, dloss=dl)
    for scale in (1.0, 0.5):
        x.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        want = gc.expert_route(x, 6)
        assert all(torch.equal(a, b) for a, b in zip(r, want))
        assert torch.equal(d, gc.expert_route_grad(x, want.ids, want.counts, dweights=g, dloss=dl))
    assert torch.equal(dx, dx)


def test_offsets_past_32_bits():
    big = torch.empty(20 << 28, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((20, 40), (1 << 28, 1))
    x = torch.randn(20, 40, device="cuda").bfloat16()
    far.copy_(x)
    near, there = gc.expert_route(x, 3), gc.expert_route(far, 3)
    assert all(torch.equal(a, b) for a, b in zip(near, there))
    dw, dl = torch.randn(20, 3, device="cuda"), torch.ones(1, device="cuda")
    want = gc.expert_route_grad(x, near.ids, near.counts, dweights=dw, dloss=dl)
    assert torch.equal(want, gc.expert_route_grad(far, near.ids, near.counts, dweights=dw, dloss=dl))
    gc.expert_route_grad(x, near.ids, near.counts, dweights=dw, dloss=dl, out=far)
    assert torch.equal(want, far.contiguous())


def test_refusals():
    x = torch.randn(4, 8, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for call in (lambda: gc.expert_route(x, 0), lambda: gc.expert_route(x, 9), lambda: gc.expert_route(x[0], 1),
                 lambda: gc.expert_route(x, 2, mask=torch.ones(3, dtype=torch.bool, device="cuda")),
                 lambda: gc.expert_route(x.t(), 2), lambda: gc.expert_route_grad(x, ids[:3]),
                 lambda: gc.expert_route_grad(x, ids, counts=torch.zeros(8, dtype=torch.int32, device="cuda")),
                 lambda: gc.expert_route_grad(x, ids, out=torch.empty(4, 7, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gc.expert_route(x.double(), 2), lambda: gc.expert_route_grad(x, ids.long()),
                 lambda: gc.expert_route(x, 2, mask=torch.ones(4, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gc.expert_route_grad(x, ids, dloss=torch.ones(1, device="cuda")),
                 lambda: gc.expert_route_grad(x, ids, out=x),
                 lambda: gc.expert_route(torch.randn(4, 128, device="cuda"), 65)):
        with pytest.raises(gc.GcError):
            call()
