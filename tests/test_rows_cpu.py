"""The row operators' argument checks, sizes and reference forms, without a GPU."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import rows_ref as ref
from partition_pass_tile_gb300 import build as gc_build
from partition_pass_tile_gb300 import gc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = {v: k for k, v in gc.STATUS.items()}
BAD, UNSUP, SMALL, MIS = (E["GC_ERR_INVALID_VALUE"], E["GC_ERR_UNSUPPORTED"], E["GC_ERR_WORKSPACE_TOO_SMALL"],
                          E["GC_ERR_MISALIGNED"])
# Fake device addresses 256 MiB apart: every call below is refused before the device.
A, B, C, D, F, G, H, WS = (0x10000000 * k for k in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    gc_build.build()
    return gc.load()


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "gc.h")).read()
    for name in ("GC_ROW_F32", "GC_ROW_BF16", "GC_ROW_F16", "GC_ID_I32", "GC_ID_I64"):
        value = int(re.search(rf"{name} = (\d+)", text).group(1))
        assert getattr(gc, name[3:]) == value


def test_expert_sizes(lib):
    assert gc.expert_rows(16, 4, 64) == 64
    assert gc.expert_rows(16, 4, 64, 16) == 64 + 64 * 15
    assert gc.expert_rows(2, 1, 64, 16) == 2 + 2 * 15
    assert gc.expert_rows(0, 4, 64, 16) == 0
    for bad in ((1 << 30, 4, 8, 1), (4, 0, 8, 1), (4, 65, 8, 1), (4, 2, 0, 1), (4, 2, 2049, 1), (4, 2, 8, 0),
                (4, 2, 8, 65537), (2 ** 31 - 1, 1, 2048, 2)):
        assert gc.expert_rows(*bad) == 0, bad
    for e in (1, 64, 2048):
        sizes = [gc.expert_workspace_bytes(t, 2, e) for t in (0, 1, 1000, 10 ** 6, 10 ** 9)]
        assert sizes[-1] >= sizes[0] > 0
    assert gc.expert_workspace_bytes(1, 1, 2049) == 0
    assert gc.embedding_grad_workspace_bytes(1000, 500, 64) >= 16 * 1000 + 8 * 500
    for bad in ((2 ** 31, 5, 5), (5, 2 ** 31 - 1, 5), (5, 5, 0), (5, 5, 2 ** 24 + 1)):
        assert gc.embedding_grad_workspace_bytes(*bad) == 0, bad


def test_dispatch_refusals(lib):
    ok = dict(ids=A, it=gc.ID_I64, tokens=100, topk=2, experts=8, align=4, x=B, xs=64, width=64, dt=gc.ROW_BF16, out=C,
              os=64, rows=300, off=D, cnt=F, slots=G, pairs=H, ws=WS, wsb=1 << 20)

    def call(**kw):
        return lib.gc_expert_dispatch(*dict(ok, **kw).values(), None)
    for kw in (dict(it=2), dict(topk=0), dict(topk=65), dict(tokens=2 ** 31), dict(experts=0), dict(experts=2049),
               dict(align=0), dict(align=1 << 17), dict(rows=223), dict(rows=2 ** 31), dict(dt=3), dict(dt=-1),
               dict(width=0), dict(xs=63), dict(os=63), dict(width=1 << 25, xs=1 << 25, os=1 << 25), dict(x=None),
               dict(out=None), dict(ids=None), dict(off=None), dict(cnt=None), dict(slots=None), dict(pairs=None),
               dict(ws=None), dict(out=B + 64), dict(slots=A + 8), dict(pairs=C + 128), dict(off=F + 4),
               dict(x=WS + 4096), dict(os=2 ** 31)):
        assert call(**kw) == BAD, kw
    for kw in (dict(ids=A + 4), dict(x=B + 1), dict(out=C + 1), dict(off=D + 2), dict(cnt=F + 1), dict(slots=G + 2),
               dict(pairs=H + 3), dict(ws=WS + 16)):
        assert call(**kw) == MIS, kw
    assert call(wsb=8) == SMALL


def test_combine_refusals(lib):
    ok = dict(y=A, ys=64, rows=300, slots=B, w=C, tokens=100, topk=2, width=64, dt=gc.ROW_F16, out=D, os=64)

    def call(**kw):
        return lib.gc_expert_combine(*dict(ok, **kw).values(), None)
    for kw in (dict(y=None), dict(ys=63), dict(rows=2 ** 31), dict(slots=None), dict(topk=0), dict(topk=65),
               dict(width=0), dict(dt=9), dict(out=None), dict(os=1), dict(out=A), dict(out=B), dict(out=C)):
        assert call(**kw) == BAD, kw
    for kw in (dict(y=A + 1), dict(slots=B + 2), dict(w=C + 2), dict(out=D + 1)):
        assert call(**kw) == MIS, kw


def test_combine_grad_refusals(lib):
    ok = dict(g=A, gs=64, y=B, ys=64, rows=300, slots=C, pairs=D, w=F, tokens=100, topk=2, width=64, dt=gc.ROW_F32,
              dy=G, ds=64, dw=H)

    def call(**kw):
        return lib.gc_expert_combine_grad(*dict(ok, **kw).values(), None)
    for kw in (dict(g=None), dict(y=None), dict(slots=None), dict(pairs=None), dict(dy=None), dict(gs=5), dict(ys=5),
               dict(ds=5), dict(dt=4), dict(topk=100), dict(width=0), dict(dy=A), dict(dw=B), dict(dy=B + 256),
               dict(dw=G)):
        assert call(**kw) == BAD, kw
    for kw in (dict(g=A + 2), dict(y=B + 2), dict(slots=C + 1), dict(pairs=D + 1), dict(w=F + 1), dict(dy=G + 2),
               dict(dw=H + 2)):
        assert call(**kw) == MIS, kw


def test_embedding_refusals(lib):
    ok = dict(table=A, ts=64, vocab=1000, width=64, dt=gc.ROW_BF16, ids=B, it=gc.ID_I32, n=100, scale=1.0, out=C, os=64)

    def call(**kw):
        return lib.gc_embedding(*dict(ok, **kw).values(), None)
    for kw in (dict(table=None), dict(ts=63), dict(vocab=2 ** 31), dict(width=0), dict(dt=7), dict(ids=None),
               dict(it=5), dict(n=2 ** 31), dict(out=None), dict(os=63), dict(out=A + 128), dict(out=B)):
        assert call(**kw) == BAD, kw
    for kw in (dict(table=A + 1), dict(ids=B + 2), dict(out=C + 1), dict(it=gc.ID_I64, ids=B + 4)):
        assert call(**kw) == MIS, kw


def test_embedding_grad_refusals(lib):
    ok = dict(g=A, gs=64, gd=gc.ROW_BF16, ids=B, it=gc.ID_I32, n=100, vocab=1000, width=64, scale=1.0, out=C, os=64,
              od=gc.ROW_F32, acc=0, ws=WS, wsb=1 << 24)

    def call(**kw):
        return lib.gc_embedding_grad(*dict(ok, **kw).values(), None)
    for kw in (dict(g=None), dict(gs=63), dict(gd=3), dict(ids=None), dict(it=2), dict(n=2 ** 31), dict(vocab=2 ** 31 - 1),
               dict(width=0), dict(out=None), dict(os=63), dict(od=3), dict(ws=None), dict(out=A), dict(out=B),
               dict(out=WS + 256)):
        assert call(**kw) == BAD, kw
    assert call(od=gc.ROW_F16) == UNSUP
    assert call(gd=gc.ROW_F32, od=gc.ROW_BF16) == UNSUP
    for kw in (dict(g=A + 1), dict(ids=B + 2), dict(out=C + 2), dict(ws=WS + 8)):
        assert call(**kw) == MIS, kw
    assert call(wsb=1000) == SMALL


def test_sample_refusals(lib):
    ok = dict(x=A, xs=1000, rows=4, vocab=1000, dt=gc.ROW_F32, u=B, us=1000, t=C, k=C + 64, p=C + 128, q=C + 192,
              tokens=D, lp=F)

    def call(**kw):
        return lib.gc_sample(*dict(ok, **kw).values(), None)
    for kw in (dict(x=None), dict(xs=999), dict(rows=2 ** 31), dict(vocab=0), dict(vocab=(1 << 22) + 1, xs=1 << 23, us=1 << 23),
               dict(dt=3), dict(us=999), dict(tokens=None), dict(tokens=A + 400), dict(lp=D + 4), dict(lp=B)):
        assert call(**kw) == BAD, kw
    for kw in (dict(x=A + 2), dict(u=B + 1), dict(t=C + 2), dict(k=C + 65), dict(p=C + 130), dict(q=C + 193),
               dict(tokens=D + 1), dict(lp=F + 2)):
        assert call(**kw) == MIS, kw


def test_binding_refusals(lib):
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
    for call in (lambda: gc.expert_dispatch(x, ids, 4), lambda: gc.expert_combine(x, ids.int()),
                 lambda: gc.embedding(x, ids), lambda: gc.embedding_grad(x, ids[:, 0], 5), lambda: gc.sample(x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        gc.row_dtype_code(torch.float64)
    with pytest.raises(ValueError):
        gc.expert_dispatch(x, ids[0], 4)
    with pytest.raises(ValueError):
        gc.embedding_grad(x, ids[:, 0], 5, accumulate=True)
    for experts, align in ((0, 1), (2049, 1), (-3, 1), (4, 0), (4, 1 << 17)):
        with pytest.raises(gc.GcError):
            gc.expert_dispatch(x, ids, experts, align=align)


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 4, (6, 2))
    rows = ref.capacity(6, 2, 4, 2)
    _, _, slots, pairs = ref.plan(ids, 4, 2, rows)
    y, g, w = rng.standard_normal((rows, 5)), rng.standard_normal((6, 5)), rng.random((6, 2))
    dy, dw, _ = ref.combine_grad(g, y, slots, pairs, w)
    by, bw, h = rng.standard_normal(y.shape), rng.standard_normal(w.shape), 1e-3
    num = ((ref.combine(y + h * by, slots, w)[0] - ref.combine(y - h * by, slots, w)[0]) * g).sum() / (2 * h)
    assert abs(num - (dy * by).sum()) < 1e-9
    num = ((ref.combine(y, slots, w + h * bw)[0] - ref.combine(y, slots, w - h * bw)[0]) * g).sum() / (2 * h)
    assert abs(num - (dw * bw).sum()) < 1e-9
    # sorted by expert, stably, and back
    assert all(ids.reshape(-1)[p] == e for e, p in ((ids.reshape(-1)[q], q) for q in pairs[pairs >= 0]))
    x = rng.standard_normal((6, 5))
    back, _ = ref.combine(ref.dispatch(x, pairs, 2), slots, None)
    assert np.allclose(back, x * (ids >= 0).sum(1)[:, None])
    v = rng.integers(-1, 7, 20)
    t, bt, gt = rng.standard_normal((7, 3)), rng.standard_normal((7, 3)), rng.standard_normal((20, 3))
    num = ((ref.embedding(t + h * bt, v, 2.0) - ref.embedding(t - h * bt, v, 2.0)) * gt).sum() / (2 * h)
    assert abs(num - (ref.embedding_grad(gt, v, 7, 2.0)[0] * bt).sum()) < 1e-9


def test_reference_sampling_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    assert ref.kept_tokens(x, 1.0, 3, 1.0, 0.0)[0].tolist() == [1, 2, 3]
    assert ref.kept_tokens(x, 1.0, 0, 0.5, 0.0)[0].tolist() == [1, 2]
    assert ref.kept_tokens(x, 1.0, 0, 0.3, 0.0)[0].tolist() == [1]
    assert ref.kept_tokens(x, 1.0, 0, 1.0, 0.4)[0].tolist() == [1, 2, 3]
    assert ref.sample(x, np.full(5, 0.5), 0.0, 0, 1.0, 0.0)[0] == 1
    assert ref.sample(np.full(4, -np.inf), np.full(4, 0.5), 1.0, 0, 1.0, 0.0)[0] == -1
