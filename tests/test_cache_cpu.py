"""Refusals of eviction that need no GPU."""

import ctypes

import pytest

from partition_pass_tile_gb300 import build as gc_build
from partition_pass_tile_gb300 import gc

BAD = {v: k for k, v in gc.STATUS.items()}["GC_ERR_INVALID_VALUE"]
# Fake device addresses 256 MiB apart: the calls are refused before the device.
A, B, C, D, F, G = (0x10000000 * k for k in range(1, 7))


@pytest.mark.parametrize("batch", [0, 1, 3])
def test_a_cache_without_heads_is_refused(batch):
    # it has lengths that the call could not write
    gc_build.build()
    lib = gc.load()
    assert gc.cache_evict_workspace_bytes(batch, 0, 10) == 0
    keys, kept = gc.CacheRows(A, 0, 0, 8, 8), gc.CacheRows(B, 0, 0, 8, 8)
    assert lib.gc_cache_evict(ctypes.byref(keys), None, gc.ROW_BF16, C, 100, None, 0, None, batch, 0, 100, 10, 0, 0,
                              ctypes.byref(kept), None, D, D + 4096, F, G, 1 << 20, None) == BAD
