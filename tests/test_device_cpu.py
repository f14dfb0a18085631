"""Tensors on a device that is not the current one are refused before anything
is launched (on stand-ins for CUDA tensors, without a GPU)."""

import pytest
import torch

from partition_pass_tile_gb300 import gc


class OnDevice:
    """What the binding asks of a tensor on cuda:`index`."""

    def __init__(self, t, index):
        self.t, self.index = t, index
        self.device, self.is_cuda = torch.device("cuda", index), True
        self.dtype, self.shape = t.dtype, t.shape

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x10000000

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(gc, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(gc, "_handle", lambda stream, device: 0)
    monkeypatch.setattr(gc, "_stream", lambda stream: 0)

    class Library:
        """Every entry point notes that it was called."""

        def __init__(self):
            self.calls = []

        def __getattr__(self, name):
            return lambda *a: self.calls.append(name) or 0

    lib = Library()
    monkeypatch.setattr(gc, "load", lambda path=None: lib)
    return lib


def rows(index, n=4, width=8):
    return OnDevice(torch.zeros(n, width), index)


def flat(index, n, dtype=torch.int32, shape=None):
    return OnDevice(torch.zeros(shape or (n,), dtype=dtype), index)


CALLS = {
    "combine": lambda a, b: gc.expert_combine(rows(a, 9), flat(b, 8, shape=(4, 2)), None, out=rows(a)),
    "combine's weights": lambda a, b: gc.expert_combine(rows(a, 9), flat(a, 8, shape=(4, 2)),
                                                        flat(b, 8, torch.float32), out=rows(a)),
    "combine's out": lambda a, b: gc.expert_combine(rows(a, 9), flat(a, 8, shape=(4, 2)), None, out=rows(b)),
    "combine_grad": lambda a, b: gc.expert_combine_grad(rows(a), rows(b, 9), flat(a, 8, shape=(4, 2)), flat(a, 9),
                                                        dy=rows(a, 9), dweights=flat(a, 8, torch.float32, (4, 2))),
    "embedding": lambda a, b: gc.embedding(rows(a, 30), flat(b, 4), out=rows(a)),
    "embedding_grad": lambda a, b: gc.embedding_grad(rows(a), flat(b, 4), 30, out=rows(a, 30), ws=flat(a, 4096, torch.uint8)),
    "sample": lambda a, b: gc.sample(rows(a), rows(b), tokens=flat(a, 4), logprobs=flat(a, 4, torch.float32)),
    "scan": lambda a, b: gc.exclusive_scan(flat(a, 16), out=flat(b, 16), total=flat(a, 1), ws=flat(a, 4096, torch.uint8)),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_elsewhere_are_refused(name, current):
    CALLS[name](0, 0)
    reached = len(current.calls)
    assert reached > 0
    for a, b in ((1, 1), (0, 1), (1, 0)):
        current.calls.clear()
        with pytest.raises(ValueError):
            CALLS[name](a, b)
        assert all(c.endswith("_bytes") for c in current.calls)
