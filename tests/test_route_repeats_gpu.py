"""The gradient of routing repeats to the last bit, on any stream and whatever runs beside it."""

import pytest
import torch

from partition_pass_tile_gb300 import gc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,topk", [(30000, 96, 6), (5000, 16, 2), (3000, 600, 20), (4, 64, 4)])
def test_gradient_repeats(tokens, experts, topk):
    g = torch.Generator(device="cuda").manual_seed(experts)
    x = torch.randn(tokens, experts, generator=g, device="cuda")
    dw, dl = torch.randn(tokens, topk, generator=g, device="cuda"), torch.ones(1, device="cuda")
    r = gc.expert_route(x, topk)
    want = gc.expert_route_grad(x, r.ids, r.counts, dweights=dw, dloss=dl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        beside = gc.expert_route(x, topk)
        again = gc.expert_route_grad(x, r.ids, r.counts, dweights=dw, dloss=dl, stream=side)
        side.synchronize()
        assert torch.equal(want, again)
        assert all(torch.equal(a, b) for a, b in zip(r, beside))
        assert torch.equal(want, gc.expert_route_grad(x, r.ids, r.counts, dweights=dw, dloss=dl))
