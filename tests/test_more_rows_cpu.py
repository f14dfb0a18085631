"""Argument checks, sizes and reference forms of routing, verification and the cache, without a GPU."""

import ctypes

import numpy as np
import pytest
import torch

import more_rows_ref as ref
from partition_pass_tile_gb300 import build as gc_build
from partition_pass_tile_gb300 import gc

E = {v: k for k, v in gc.STATUS.items()}
BAD, SMALL, MIS = E["GC_ERR_INVALID_VALUE"], E["GC_ERR_WORKSPACE_TOO_SMALL"], E["GC_ERR_MISALIGNED"]
# Fake device addresses 256 MiB apart: every call below is refused before the device.
A, B, C, D, F, G, H, I, J, WS = (0x10000000 * k for k in range(1, 11))


@pytest.fixture(scope="module")
def lib():
    gc_build.build()
    return gc.load()


def test_workspace_sizes(lib):
    assert gc.expert_route_workspace_bytes(1, 64) >= 256
    assert gc.expert_route_workspace_bytes(10 ** 6, 64) >= gc.expert_route_workspace_bytes(10 ** 3, 64)
    for bad in ((2 ** 31, 4), (4, 0), (4, 2049)):
        assert gc.expert_route_workspace_bytes(*bad) == 0, bad
    assert gc.sample_verify_workspace_bytes(4, 3, 1000) >= 8 * 4 * 7
    assert gc.sample_verify_workspace_bytes(0, 0, 1) > 0
    for bad in ((2 ** 31, 1, 5), (4, 65, 5), (4, 1, 0), (4, 1, (1 << 22) + 1), (2 ** 31 - 1, 64, 1 << 22)):
        assert gc.sample_verify_workspace_bytes(*bad) == 0, bad
    assert gc.cache_evict_workspace_bytes(2, 3, 100) >= 4 * 600
    for bad in ((2 ** 31, 1, 5), (2 ** 20, 2 ** 20, 5), (1, 1, 0), (1, 1, 2 ** 24 + 1), (2 ** 16, 2 ** 10, 2 ** 10)):
        assert gc.cache_evict_workspace_bytes(*bad) == 0, bad


def test_route_refusals(lib):
    ok = dict(x=A, xs=64, tokens=100, experts=64, dt=gc.ROW_BF16, k=4, norm=1, mask=B, ids=C, w=D, counts=F, load=G,
              loss=H, ws=WS, wsb=1 << 20)

    def call(**kw):
        return lib.gc_expert_route(*dict(ok, **kw).values(), None)
    for kw in (dict(x=None), dict(xs=63), dict(tokens=2 ** 31), dict(experts=0, xs=4), dict(experts=2049, xs=4096),
               dict(dt=3), dict(k=0), dict(k=65), dict(experts=3, k=4), dict(ids=None), dict(w=None), dict(ws=None),
               dict(counts=None), dict(counts=None, load=None), dict(counts=None, loss=None), dict(ids=A + 64),
               dict(w=C), dict(load=F + 8), dict(loss=G), dict(mask=WS + 512), dict(counts=D + 16)):
        assert call(**kw) == BAD, kw
    for kw in (dict(x=A + 1), dict(ids=C + 2), dict(w=D + 1), dict(counts=F + 2), dict(load=G + 1), dict(loss=H + 3),
               dict(ws=WS + 64)):
        assert call(**kw) == MIS, kw
    assert call(wsb=16) == SMALL


def test_route_grad_refusals(lib):
    ok = dict(x=A, xs=64, tokens=100, experts=64, dt=gc.ROW_F32, k=4, norm=0, ids=B, counts=C, dw=D, dl=F, dx=G, ds=64)

    def call(**kw):
        return lib.gc_expert_route_grad(*dict(ok, **kw).values(), None)
    for kw in (dict(x=None), dict(xs=63), dict(ds=63), dict(tokens=2 ** 31), dict(experts=0), dict(dt=-1), dict(k=0),
               dict(k=65), dict(ids=None), dict(counts=None), dict(dx=None), dict(dx=A), dict(dx=B + 128), dict(dx=D),
               dict(dx=F)):
        assert call(**kw) == BAD, kw
    for kw in (dict(x=A + 2), dict(ids=B + 2), dict(counts=C + 1), dict(dw=D + 2), dict(dl=F + 2), dict(dx=G + 2)):
        assert call(**kw) == MIS, kw


def test_verify_refusals(lib):
    ok = dict(x=A, xs=1000, d=B, ds=1000, n=4, k=3, vocab=1000, dt=gc.ROW_F16, ids=C, acc=D, u=F, us=1000, t=G,
              tokens=H, accepted=I, lp=J, ws=WS, wsb=1 << 20)

    def call(**kw):
        return lib.gc_sample_verify(*dict(ok, **kw).values(), None)
    for kw in (dict(x=None), dict(xs=999), dict(ds=999), dict(us=999), dict(n=2 ** 31), dict(k=65), dict(vocab=0),
               dict(vocab=(1 << 22) + 1, xs=1 << 23, ds=1 << 23, us=1 << 23), dict(dt=5), dict(ids=None),
               dict(acc=None), dict(tokens=None), dict(accepted=None), dict(ws=None), dict(tokens=A + 400),
               dict(accepted=H), dict(lp=H + 4), dict(lp=F), dict(ids=WS + 256)):
        assert call(**kw) == BAD, kw
    for kw in (dict(x=A + 1), dict(d=B + 1), dict(ids=C + 2), dict(acc=D + 1), dict(u=F + 2), dict(t=G + 1),
               dict(tokens=H + 2), dict(accepted=I + 1), dict(lp=J + 2), dict(ws=WS + 32)):
        assert call(**kw) == MIS, kw
    assert call(wsb=64) == SMALL


def test_score_refusals(lib):
    ok = dict(w=A, bs=8 * 6 * 500, hs=6 * 500, qs=500, dt=gc.ROW_BF16, batch=2, heads=2, group=4, queries=6, length=500,
              s=B, ss=500, decay=1.0, lengths=C, counted=D, out=F, os=500)

    def call(**kw):
        return lib.gc_cache_score(*dict(ok, **kw).values(), None)
    for kw in (dict(w=None), dict(dt=3), dict(batch=2 ** 31), dict(heads=2 ** 31), dict(group=0), dict(group=2 ** 31),
               dict(batch=2 ** 16, heads=2 ** 16), dict(queries=2 ** 31), dict(length=2 ** 24 + 1, ss=2 ** 25, os=2 ** 25),
               dict(bs=2 ** 62), dict(hs=2 ** 60), dict(qs=2 ** 60), dict(ss=499), dict(os=499), dict(out=None),
               dict(out=A + 64), dict(out=B + 400), dict(out=B, os=504), dict(out=C)):
        assert call(**kw) == BAD, kw
    for kw in (dict(w=A + 1), dict(s=B + 2), dict(lengths=C + 2), dict(counted=D + 1), dict(out=F + 2)):
        assert call(**kw) == MIS, kw


def test_evict_refusals(lib):
    def cache(p, rows, width=64, row=None, head=None, batch=None):
        row = width if row is None else row
        head = rows * row if head is None else head
        return gc.CacheRows(p, 3 * head if batch is None else batch, head, row, width)
    ok = dict(k=cache(A, 500), v=cache(B, 500, 32), dt=gc.ROW_BF16, s=C, ss=500, p=D, ps=500, lengths=F, batch=2,
              heads=3, length=500, budget=100, sinks=4, recent=20, kk=cache(G, 100), kv=cache(H, 100, 32), ks=I,
              kp=I + 4096, kl=I + 16384, ws=WS, wsb=1 << 20)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.gc_cache_evict(*(ctypes.byref(v) if isinstance(v, gc.CacheRows) else v for v in a.values()), None)
    for kw in (dict(k=None), dict(kk=None), dict(v=None), dict(kv=None), dict(dt=3), dict(s=None), dict(ss=499),
               dict(ps=499), dict(batch=2 ** 31), dict(length=2 ** 24 + 1, ss=2 ** 25, ps=2 ** 25), dict(budget=0),
               dict(sinks=101), dict(sinks=90, recent=11), dict(ks=None), dict(kp=None), dict(kl=None), dict(ws=None),
               dict(k=cache(None, 500)), dict(v=cache(None, 500, 32)), dict(kk=cache(None, 100)),
               dict(k=cache(A, 500, 0)), dict(k=cache(A, 500, 60)), dict(kv=cache(H, 100, 30)),
               dict(k=cache(A, 500, 64, row=2 ** 31)), dict(k=cache(A, 500, 64, head=2 ** 48)),
               # kept rows that lie on one another
               dict(kk=cache(G, 100, 64, row=32)), dict(kk=cache(G, 100, 64, head=64)),
               dict(kk=cache(G, 100, 64, batch=6400)), dict(kk=cache(G, 100, 64, row=0)),
               # outputs on inputs and on one another
               dict(kk=cache(A + 4096, 100)), dict(kk=cache(H, 100)), dict(kp=I), dict(kl=F), dict(ks=C)):
        assert call(**kw) == BAD, kw
    for kw in (dict(k=cache(A + 1, 500)), dict(v=cache(B + 1, 500, 32)), dict(s=C + 2), dict(p=D + 1),
               dict(lengths=F + 2), dict(kk=cache(G + 1, 100)), dict(ks=I + 2), dict(kp=I + 4097), dict(kl=I + 16386),
               dict(ws=WS + 8)):
        assert call(**kw) == MIS, kw
    assert call(wsb=256) == SMALL


def test_binding_refusals(lib):
    x = torch.zeros(4, 8)
    for call in (lambda: gc.expert_route(x, 2), lambda: gc.expert_route_grad(x, torch.zeros(4, 2, dtype=torch.int32)),
                 lambda: gc.sample_verify(torch.zeros(2, 3, 8), torch.zeros(2, 2, dtype=torch.int32)),
                 lambda: gc.cache_score(torch.zeros(2, 4, 3, 8), torch.zeros(2, 2, 8)),
                 lambda: gc.cache_evict(torch.zeros(2, 2, 8, 4), None, torch.zeros(2, 2, 8), 4)):
        with pytest.raises(ValueError):  # not on a GPU
            call()


def test_reference_routing_by_hand():
    x = np.log(np.array([[0.1, 0.4, 0.4, 0.1], [0.7, 0.1, 0.1, 0.1], [0.25, 0.25, 0.25, 0.25]]))
    ids, w, counts, load, loss, _, _ = ref.route(x, 2, False, np.array([True, True, False]))
    assert ids.tolist() == [[1, 2], [0, 1], [-1, -1]]
    assert np.allclose(w, [[0.4, 0.4], [0.7, 0.1], [0, 0]])
    assert counts.tolist() == [1, 2, 1, 0, 2]
    assert np.allclose(load, [0.4, 0.25, 0.25, 0.1])
    assert np.isclose(loss, 4 * (0.4 + 2 * 0.25 + 0.25) / 4)
    # even use: 1
    assert np.isclose(ref.route(np.zeros((4, 1)), 1, True, None)[4], 1.0)


@pytest.mark.parametrize("normalize", [True, False])
def test_reference_route_gradient_against_differences(normalize):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((7, 5))
    x[2, 3] = -np.inf
    mask = np.array([True] * 6 + [False])
    ids, _, counts, _, _, _, _ = ref.route(x, 3, normalize, mask)
    g, dl = rng.standard_normal(ids.shape), 0.7
    dx, _ = ref.route_grad(x, ids, counts, g, dl, normalize)

    def value(y):
        got, w, c, _, loss, _, _ = ref.route(y, 3, normalize, mask)
        assert np.array_equal(got, ids)  # the choices stay
        return float((w * g).sum() + dl * loss)
    by, h = np.where(np.isinf(x), 0.0, rng.standard_normal(x.shape)), 1e-5
    assert abs((value(x + h * by) - value(x - h * by)) / (2 * h) - float((dx * by).sum())) < 1e-8
    assert not dx[6].any() and dx[2, 3] == 0.0


def test_reference_verification_draws_the_target():
    # whatever the draft, the first token is distributed as the target: 20000
    # draws of 4 tokens, a share p off by more than 5 sqrt(p (1 - p) / 20000)
    # has a chance of 6e-7
    rng = np.random.default_rng(0)
    x, d = np.log(np.array([0.5, 0.3, 0.15, 0.05])), np.log(np.array([0.1, 0.2, 0.3, 0.4]))
    n = 20000
    for draft in (d, None):
        first = np.zeros(4)
        for _ in range(n):
            token = rng.choice(4, p=np.exp(d))
            u, v = rng.random(1), rng.random(4)
            t, a, _, _ = ref.verify(np.stack([x, x]), [token], u, v, None if draft is None else draft[None], 1.0)
            first[t[0]] += 1
        p = np.exp(x)
        assert np.all(np.abs(first / n - p) <= 5 * np.sqrt(p * (1 - p) / n))


def test_reference_eviction_by_hand():
    s = np.array([0, 9, 1, 5, 5, 5, 2, 0], np.float32)
    assert ref.kept(s, 8, 5, 1, 1).tolist() == [0, 1, 3, 4, 7]
    assert ref.kept(s, 5, 5, 1, 1).tolist() == [0, 1, 2, 3, 4]
    assert ref.kept(np.full(8, np.nan, np.float32), 8, 3, 0, 1).tolist() == [0, 1, 7]
    assert ref.kept(s, 8, 2, 1, 1).tolist() == [0, 7]
