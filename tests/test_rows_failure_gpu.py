"""The embedding gradient whose bulk copies do not arrive in time: the wait
gives up, the host can read that, and no row that lacks a summand looks right.
The planted failure is a wait for bytes that nobody copies (gc_testing.h)."""

import numpy as np
import pytest
import torch

import rows_ref as ref
from partition_pass_tile_gb300 import gc
from test_rows_gpu import off, rows_of, token_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,odt,width", [("f32", "f32", 256), ("bf16", "f32", 264), ("bf16", "bf16", 512),
                                             ("f16", "f16", 2312)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_missing_copies_are_reported_and_make_nan(dtype, odt, width, accumulate):
    rng = np.random.default_rng(width)
    n, vocab = 300, 700
    g, g64 = rows_of(rng, n, width, dtype)
    ids, host = token_ids(rng, n, vocab, "zipf", "i64")  # runs within blocks and across them
    out, there64 = rows_of(rng, vocab, width, odt)
    there = out.clone()
    ws = torch.empty(gc.embedding_grad_workspace_bytes(n, vocab, width), dtype=torch.uint8, device="cuda")
    assert gc.testing_embedding_grad_stalled(g, ids, out, ws, timeout_ns=2_000_000, accumulate=accumulate) == 0
    torch.cuda.synchronize()  # the kernels finished: nothing hung
    assert gc.query_device_status(ws) == 6  # GC_ERR_TIMEOUT
    assert gc.query_device_status(ws) == 0  # read and cleared
    present = torch.zeros(vocab, dtype=torch.bool)
    present[torch.from_numpy(host)] = True
    present = present.cuda()
    assert bool(out[present].isnan().all())
    assert torch.equal(out[~present], there[~present] if accumulate else torch.zeros_like(out[~present]))
    # the same workspace and context: a normal call is right again
    out.copy_(there)
    gc.embedding_grad(g, ids, vocab, out=out, accumulate=accumulate, ws=ws)
    assert gc.query_device_status(ws) == 0
    want, size, count = ref.embedding_grad(g64, host, vocab, 1.0)
    if accumulate:
        want, size, count = want + there64, size + np.abs(there64), count + 1
    assert off(out, want, size, count[:, None], odt) <= 1


def test_rows_that_are_not_copied_in_bulk_do_not_wait():
    rng = np.random.default_rng(2)
    g, g64 = rows_of(rng, 100, 33, "f32")
    ids, host = token_ids(rng, 100, 50, "all", "i32")
    out = torch.empty(50, 33, device="cuda")
    ws = torch.empty(gc.embedding_grad_workspace_bytes(100, 50, 33), dtype=torch.uint8, device="cuda")
    assert gc.testing_embedding_grad_stalled(g, ids, out, ws, timeout_ns=2_000_000) == 0
    assert gc.query_device_status(ws) == 0
    want, size, count = ref.embedding_grad(g64, host, 50, 1.0)
    assert off(out, want, size, count[:, None], "f32") <= 1


@pytest.mark.parametrize("n,vocab", [(5, 0), (0, 0), (0, 7), (5, 7), (5000, 7)])
def test_the_status_of_a_call_on_an_uninitialised_workspace(n, vocab):
    # a workspace needs no initialisation, whatever the call has to do
    ws = torch.full((gc.embedding_grad_workspace_bytes(n, vocab, 64),), 255, dtype=torch.uint8, device="cuda")
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    for accumulate in (False, True):
        ws.fill_(255)
        out = torch.zeros(vocab, 64, device="cuda")
        gc.embedding_grad(torch.ones(n, 64, device="cuda"), ids, vocab, out=out, accumulate=accumulate, ws=ws)
        assert gc.query_device_status(ws) == 0
        assert not out[1:].any() and (vocab == 0 or bool((out[0] == n).all()))
