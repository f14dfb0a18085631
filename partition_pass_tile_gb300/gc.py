"""Python binding of libgc (include/gc.h): argument marshalling only.

Every function here turns torch tensors into device pointers, sizes and enum
codes, calls the C entry point of the same name, and raises ``GcError`` on a
non-zero status.  No step of the computation runs in Python: the predicate,
the scan and the scatter all run in libgc's CUDA kernels.  PyTorch supplies
device memory and streams.

The library is loaded on first use from this package's directory; if it has
not been built (``__graft_entry__.build()`` or ``python -m
partition_pass_tile_gb300.build``) the first call raises.
"""

from __future__ import annotations

import ctypes
from functools import lru_cache
from pathlib import Path
from typing import NamedTuple

import torch

LIB_PATH = Path(__file__).resolve().parent / "libgc.so"

# enum values of include/gc.h
I32, U32, F32 = 0, 1, 2
NONZERO, ODD, EVEN = 0, 1, 2
OP_EXCLUSIVE_SCAN, OP_SELECT_IF, OP_PARTITION, OP_SPLIT_RADIX, OP_SELECT_IF_ATOMIC = range(5)
OP_INCLUSIVE_SCAN = 5
OP_RADIX_SORT = 6
OP_REDUCE = 7
OP_COUNT_IF = 8
LT, LE, GT, GE, EQ, NE, MASK_EQ, MASK_NE = range(8)
ROW_F32, ROW_BF16, ROW_F16 = 0, 1, 2
ID_I32, ID_I64 = 0, 1
CMP_NAMES = {"<": LT, "<=": LE, ">": GT, ">=": GE, "==": EQ, "!=": NE,
             "mask==": MASK_EQ, "mask!=": MASK_NE}


class Predicate(ctypes.Structure):
    """gc_predicate: x OP operand in the dtype's order, or (bits & mask) OP operand."""
    _fields_ = [("cmp", ctypes.c_int), ("operand", ctypes.c_uint32), ("mask", ctypes.c_uint32)]
STATUS = {0: "GC_OK", 1: "GC_ERR_INVALID_VALUE", 2: "GC_ERR_UNSUPPORTED",
          3: "GC_ERR_WORKSPACE_TOO_SMALL", 4: "GC_ERR_MISALIGNED", 5: "GC_ERR_CUDA",
          6: "GC_ERR_TIMEOUT", 7: "GC_ERR_DEVICE_CHECK"}
PRED_NAMES = {"nonzero": NONZERO, "odd": ODD, "even": EVEN}

_lib = None


class GcError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


def load(path: str | Path | None = None) -> ctypes.CDLL:
    """Load libgc.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path is not None else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build the CUDA library first "
                           "(python -m partition_pass_tile_gb300.build)")
    lib = ctypes.CDLL(str(p))
    V, Z, I, U64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64
    S, U32T, F = ctypes.c_int, ctypes.c_uint32, ctypes.c_float
    sig = {
        "gc_status_string": ([S], ctypes.c_char_p),
        "gc_version": ([], ctypes.c_char_p),
        "gc_workspace_bytes": ([I, Z, I], Z),
        "gc_tile_elements": ([I], Z),
        "gc_workspace_init": ([V, Z, V], S),
        "gc_exclusive_scan": ([V, V, V, Z, I, V, Z, V], S),
        "gc_select_if": ([V, V, V, Z, I, I, V, Z, V], S),
        "gc_partition": ([V, V, V, Z, I, I, V, Z, V], S),
        "gc_split_radix": ([V, V, V, V, Z, I, I, V, Z, V], S),
        "gc_select_if_atomic": ([V, V, V, Z, I, I, V, Z, V], S),
        "gc_select_if_atomic_tile": ([V, V, V, Z, I, I, V, Z, V], S),
        "gc_query_device_status": ([V, V], S),
        "gc_testing_select_if_skip_tile0": ([V, V, V, Z, I, I, V, Z, U64, V], S),
        "gc_testing_exclusive_scan_stalled_barrier": ([V, V, V, Z, I, V, Z, U64, V], S),
        "gc_inclusive_scan": ([V, V, V, Z, I, V, Z, V], S),
        "gc_select_if_pred": ([V, V, V, Z, I, ctypes.POINTER(Predicate), V, Z, V], S),
        "gc_partition_pred": ([V, V, V, Z, I, ctypes.POINTER(Predicate), V, Z, V], S),
        "gc_radix_sort": ([V, V, V, V, Z, I, V, Z, V], S),
        "gc_reduce": ([V, V, Z, I, V, Z, V], S),
        "gc_count_if": ([V, V, Z, I, I, V, Z, V], S),
        "gc_shard_offsets": ([I, I, V, ctypes.POINTER(U64), Z, Z, V, V], S),
        "gc_exclusive_scan_carry": ([V, V, V, Z, I, V, V, Z, V], S),
        "gc_select_if_at": ([V, V, Z, V, V, Z, I, I, V, Z, V], S),
        "gc_partition_at": ([V, V, Z, V, V, Z, I, I, V, Z, V], S),
        "gc_expert_rows": ([Z, Z, U32T, U32T], Z),
        "gc_expert_workspace_bytes": ([Z, Z, U32T], Z),
        "gc_expert_dispatch": ([V, I, Z, Z, U32T, U32T, V, Z, Z, I, V, Z, Z, V, V, V, V, V, Z, V], S),
        "gc_expert_combine": ([V, Z, Z, V, V, Z, Z, Z, I, V, Z, V], S),
        "gc_expert_combine_grad": ([V, Z, V, Z, Z, V, V, V, Z, Z, Z, I, V, Z, V, V], S),
        "gc_embedding": ([V, Z, Z, Z, I, V, I, Z, F, V, Z, V], S),
        "gc_embedding_grad_workspace_bytes": ([Z, Z, Z], Z),
        "gc_embedding_grad": ([V, Z, I, V, I, Z, Z, Z, F, V, Z, I, I, V, Z, V], S),
        "gc_testing_embedding_grad_stalled": ([V, Z, I, V, I, Z, Z, Z, F, V, Z, I, I, V, Z, U64, V], S),
        "gc_sample": ([V, Z, Z, Z, I, V, Z, V, V, V, V, V, V, V], S),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    if path is None:
        _lib = lib
    return lib


def _check(status: int, what: str) -> None:
    if status != 0:
        raise GcError(status, what)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.int32:
        return I32
    if t.dtype == torch.uint32:
        return U32
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"libgc handles int32, uint32 and float32 tensors, not {t.dtype}")


def pred_code(pred) -> int:
    return PRED_NAMES[pred] if isinstance(pred, str) else int(pred)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_device(t: torch.Tensor) -> None:
    """libgc launches on the current device, so every tensor has to be there."""
    at = t.get_device()
    if at < 0:
        raise ValueError("libgc takes CUDA tensors (device pointers)")
    if at != _current_device():
        raise ValueError(f"libgc runs on the current device, cuda:{_current_device()}, and a tensor is on cuda:{at}")


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    _on_device(t)
    if not t.is_contiguous():
        raise ValueError("libgc takes contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def tile_elements(op: int) -> int:
    return int(load().gc_tile_elements(op))


def workspace_bytes(op: int, n: int, dtype: int = I32) -> int:
    return int(load().gc_workspace_bytes(op, n, dtype))


def workspace(op: int, n: int, dtype: int = I32, device=None) -> torch.Tensor:
    """A zero-filled workspace for (op, n, dtype) on `device` (torch-allocated)."""
    nbytes = max(workspace_bytes(op, n, dtype), 512)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def _ws(ws, op, n, dtype, device):
    return ws if ws is not None else workspace(op, n, dtype, device)


def exclusive_scan(x: torch.Tensor, out: torch.Tensor | None = None,
                   total: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   stream=None, with_total: bool = True):
    """-> (out, total); total is a 1-element device tensor of x's dtype (or None)."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if total is None and with_total:
        total = torch.empty(1, dtype=x.dtype, device=x.device)
    ws = _ws(ws, OP_EXCLUSIVE_SCAN, n, dt, x.device)
    _check(load().gc_exclusive_scan(_ptr(x), _ptr(out), _ptr(total), n, dt, _ptr(ws),
                                    ws.numel(), _stream(stream)), "gc_exclusive_scan")
    return out, total


def inclusive_scan(x: torch.Tensor, out: torch.Tensor | None = None,
                   total: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   stream=None, with_total: bool = True):
    """-> (out, total) with out[i] = x[0] + ... + x[i]."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if total is None and with_total:
        total = torch.empty(1, dtype=x.dtype, device=x.device)
    ws = _ws(ws, OP_INCLUSIVE_SCAN, n, dt, x.device)
    _check(load().gc_inclusive_scan(_ptr(x), _ptr(out), _ptr(total), n, dt, _ptr(ws),
                                    ws.numel(), _stream(stream)), "gc_inclusive_scan")
    return out, total


def predicate(x: torch.Tensor, cmp, operand=0, mask: int = 0) -> Predicate:
    """A gc_predicate for tensor x: cmp in "<", "<=", ">", ">=", "==", "!=" (operand
    a number of x's dtype) or "mask==", "mask!=" (operand, mask: raw 32-bit patterns)."""
    c = CMP_NAMES[cmp] if isinstance(cmp, str) else int(cmp)
    if c >= MASK_EQ:
        bits = int(operand) & 0xFFFFFFFF
    else:
        np_dtype = {torch.int32: "<i4", torch.uint32: "<u4", torch.float32: "<f4"}[x.dtype]
        import numpy as np
        bits = int(np.array([operand], dtype=np_dtype).view(np.uint32)[0])
    return Predicate(c, bits, int(mask) & 0xFFFFFFFF)


def select_if_pred(x: torch.Tensor, pred: Predicate, out: torch.Tensor | None = None,
                   count: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """Stable select-if with a parameterised predicate -> (out, count)."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if count is None:
        count = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_SELECT_IF, n, dt, x.device)
    _check(load().gc_select_if_pred(_ptr(x), _ptr(out), _ptr(count), n, dt, ctypes.byref(pred),
                                    _ptr(ws), ws.numel(), _stream(stream)), "gc_select_if_pred")
    return out, count


def partition_pred(x: torch.Tensor, pred: Predicate, out: torch.Tensor | None = None,
                   count_true: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   stream=None):
    """Stable partition with a parameterised predicate -> (out, count_true)."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if count_true is None:
        count_true = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_PARTITION, n, dt, x.device)
    _check(load().gc_partition_pred(_ptr(x), _ptr(out), _ptr(count_true), n, dt,
                                    ctypes.byref(pred), _ptr(ws), ws.numel(), _stream(stream)),
           "gc_partition_pred")
    return out, count_true


def select_if(x: torch.Tensor, pred, out: torch.Tensor | None = None,
              count: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """-> (out, count): out has x's size, its first count[0] elements are the survivors."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if count is None:
        count = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_SELECT_IF, n, dt, x.device)
    _check(load().gc_select_if(_ptr(x), _ptr(out), _ptr(count), n, dt, pred_code(pred),
                               _ptr(ws), ws.numel(), _stream(stream)), "gc_select_if")
    return out, count


def select_if_atomic(x: torch.Tensor, pred, out: torch.Tensor | None = None,
                     count: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None, per_tile: bool = False):
    """The atomic-counter comparison path -> (out, count): the survivors in an
    order the atomics decide.  One atomic per survivor (gc_select_if_atomic),
    or per tile with per_tile=True (gc_select_if_atomic_tile)."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if count is None:
        count = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_SELECT_IF_ATOMIC, n, dt, x.device)
    name = "gc_select_if_atomic_tile" if per_tile else "gc_select_if_atomic"
    _check(getattr(load(), name)(_ptr(x), _ptr(out), _ptr(count), n, dt, pred_code(pred),
                                 _ptr(ws), ws.numel(), _stream(stream)), name)
    return out, count


def partition(x: torch.Tensor, pred, out: torch.Tensor | None = None,
              count_true: torch.Tensor | None = None, ws: torch.Tensor | None = None,
              stream=None):
    """-> (out, count_true)."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if count_true is None:
        count_true = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_PARTITION, n, dt, x.device)
    _check(load().gc_partition(_ptr(x), _ptr(out), _ptr(count_true), n, dt, pred_code(pred),
                               _ptr(ws), ws.numel(), _stream(stream)), "gc_partition")
    return out, count_true


def split_radix(keys: torch.Tensor, vals: torch.Tensor | None = None, begin_bit: int = 0,
                end_bit: int = 32, keys_out: torch.Tensor | None = None,
                vals_out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                stream=None):
    """-> (keys_out, vals_out).  Keys and payloads are 32-bit (uint32 or int32 bits)."""
    n = keys.numel()
    for t in (keys, vals):
        if t is not None and t.element_size() != 4:
            raise TypeError("split_radix takes 32-bit keys and payloads")
    if keys_out is None:
        keys_out = torch.empty_like(keys)
    if vals is not None and vals_out is None:
        vals_out = torch.empty_like(vals)
    ws = _ws(ws, OP_SPLIT_RADIX, n, U32, keys.device)
    _check(load().gc_split_radix(_ptr(keys), _ptr(vals), _ptr(keys_out), _ptr(vals_out), n,
                                 begin_bit, end_bit, _ptr(ws), ws.numel(), _stream(stream)),
           "gc_split_radix")
    return keys_out, vals_out


def radix_sort(keys: torch.Tensor, vals: torch.Tensor | None = None,
               keys_out: torch.Tensor | None = None, vals_out: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, stream=None):
    """-> (keys_out, vals_out): stable ascending sort in keys' dtype order (float32:
    IEEE 754 totalOrder), 32-bit payloads carried."""
    n = keys.numel()
    dt = dtype_code(keys)
    if vals is not None and vals.element_size() != 4:
        raise TypeError("radix_sort carries 32-bit payloads")
    if keys_out is None:
        keys_out = torch.empty_like(keys)
    if vals is not None and vals_out is None:
        vals_out = torch.empty_like(vals)
    ws = _ws(ws, OP_RADIX_SORT, n, dt, keys.device)
    _check(load().gc_radix_sort(_ptr(keys), _ptr(vals), _ptr(keys_out), _ptr(vals_out), n, dt,
                                _ptr(ws), ws.numel(), _stream(stream)), "gc_radix_sort")
    return keys_out, vals_out


def query_device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronous: the workspace's device-side error code (0 = none), then cleared."""
    return int(load().gc_query_device_status(_ptr(ws), _stream(stream)))


def testing_select_if_skip_tile0(x: torch.Tensor, pred, out, count, ws, timeout_ns: int,
                                 stream=None) -> int:
    """Test hook (include/gc_testing.h): returns the launch status."""
    return int(load().gc_testing_select_if_skip_tile0(
        _ptr(x), _ptr(out), _ptr(count), x.numel(), dtype_code(x), pred_code(pred), _ptr(ws),
        ws.numel(), timeout_ns, _stream(stream)))


def testing_force_fallback(on: bool) -> None:
    """Test hook (include/gc_testing.h): one-tile-per-CTA kernels while on."""
    f = load().gc_testing_force_fallback
    f.argtypes = [ctypes.c_int]
    f.restype = None
    f(1 if on else 0)


def testing_exclusive_scan_stalled_barrier(x: torch.Tensor, out, total, ws, timeout_ns: int,
                                           stream=None) -> int:
    """Test hook (include/gc_testing.h): returns the launch status."""
    return int(load().gc_testing_exclusive_scan_stalled_barrier(
        _ptr(x), _ptr(out), _ptr(total), x.numel(), dtype_code(x), _ptr(ws), ws.numel(),
        timeout_ns, _stream(stream)))


NOALLOC_MAX_ELEMENTS = 1 << 28


def select_if_noalloc_status(stream=None) -> int:
    """Synchronous: the no-workspace entry point's device-side error code
    (0 = none) on the current device, then cleared."""
    f = load().gc_select_if_noalloc_status
    f.argtypes = [ctypes.c_void_p]
    f.restype = ctypes.c_int
    return int(f(_stream(stream)))


def testing_select_if_noalloc_stalled_barrier(x: torch.Tensor, pred, out, count, timeout_ns: int,
                                              stream=None) -> int:
    """Test hook (include/gc_testing.h): returns the launch status."""
    f = load().gc_testing_select_if_noalloc_stalled_barrier
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                  ctypes.c_int, ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p]
    f.restype = ctypes.c_int
    return int(f(_ptr(x), _ptr(out), _ptr(count), x.numel(), dtype_code(x), pred_code(pred),
                 timeout_ns, _stream(stream)))


def select_if_noalloc(x: torch.Tensor, pred, out: torch.Tensor | None = None,
                      count: torch.Tensor | None = None, stream=None):
    """gc_select_if_noalloc: select-if with the library's own fixed scratch
    (no workspace argument, no allocation by the library).  -> (out, count)."""
    lib = load()
    f = lib.gc_select_if_noalloc
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                  ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    f.restype = ctypes.c_int
    if out is None:
        out = torch.empty_like(x)
    if count is None:
        count = torch.empty(1, dtype=torch.uint32, device=x.device)
    _check(f(_ptr(x), _ptr(out), _ptr(count), x.numel(), dtype_code(x), pred_code(pred),
             _stream(stream)), "gc_select_if_noalloc")
    return out, count


# ---------------------------------------------------------------- shards

def reduce(x: torch.Tensor, total: torch.Tensor | None = None, ws: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """gc_reduce: a 1-element device tensor of x's dtype holding sum(x)."""
    n = x.numel()
    dt = dtype_code(x)
    if total is None:
        total = torch.empty(1, dtype=x.dtype, device=x.device)
    ws = _ws(ws, OP_REDUCE, n, dt, x.device)
    _check(load().gc_reduce(_ptr(x), _ptr(total), n, dt, _ptr(ws), ws.numel(), _stream(stream)),
           "gc_reduce")
    return total


def count_if(x: torch.Tensor, pred, count: torch.Tensor | None = None,
             ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gc_count_if: a 1-element uint32 device tensor, how many elements pred keeps."""
    n = x.numel()
    dt = dtype_code(x)
    if count is None:
        count = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_COUNT_IF, n, dt, x.device)
    _check(load().gc_count_if(_ptr(x), _ptr(count), n, dt, pred_code(pred), _ptr(ws), ws.numel(),
                              _stream(stream)), "gc_count_if")
    return count


def shard_offsets(op: int, totals: torch.Tensor, rank: int, sizes=None, dtype: int | None = None,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gc_shard_offsets for shard `rank` of totals.numel() shards.  Returns one
    element of totals' dtype (scan), one 64-bit offset (select-if) or two
    (partition: kept before, first rejected position; `sizes` = the shards'
    element counts, host integers) as an int64 tensor."""
    parts = totals.numel()
    dt = dtype_code(totals) if dtype is None else dtype
    if out is None:
        if op == OP_EXCLUSIVE_SCAN:
            out = torch.empty(1, dtype=totals.dtype, device=totals.device)
        else:
            # uint64 on the device; int64 here (the offsets stay below 2^63)
            out = torch.empty(2 if op == OP_PARTITION else 1, dtype=torch.int64,
                              device=totals.device)
    h = None
    if sizes is not None:
        h = (ctypes.c_uint64 * parts)(*[int(v) for v in sizes])
    _check(load().gc_shard_offsets(op, dt, _ptr(totals), h, parts, rank, _ptr(out),
                                   _stream(stream)), "gc_shard_offsets")
    return out


def exclusive_scan_carry(x: torch.Tensor, carry: torch.Tensor, out: torch.Tensor | None = None,
                         total: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                         stream=None, with_total: bool = True):
    """-> (out, total): out[i] = carry + x[0] + ... + x[i-1], total = carry + sum(x)."""
    n = x.numel()
    dt = dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if total is None and with_total:
        total = torch.empty(1, dtype=x.dtype, device=x.device)
    ws = _ws(ws, OP_EXCLUSIVE_SCAN, n, dt, x.device)
    _check(load().gc_exclusive_scan_carry(_ptr(x), _ptr(out), _ptr(total), n, dt, _ptr(carry),
                                          _ptr(ws), ws.numel(), _stream(stream)),
           "gc_exclusive_scan_carry")
    return out, total


def select_if_at(x: torch.Tensor, pred, out: torch.Tensor, base: torch.Tensor,
                 count: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """Survivors of x to out[base + rank] (out: the whole output; base: a
    1-element uint64 device tensor) -> (out, count of this call)."""
    n = x.numel()
    dt = dtype_code(x)
    if count is None:
        count = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_SELECT_IF, n, dt, x.device)
    _check(load().gc_select_if_at(_ptr(x), _ptr(out), out.numel(), _ptr(base), _ptr(count), n, dt,
                                  pred_code(pred), _ptr(ws), ws.numel(), _stream(stream)),
           "gc_select_if_at")
    return out, count


def partition_at(x: torch.Tensor, pred, out: torch.Tensor, offsets: torch.Tensor,
                 count_true: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                 stream=None):
    """One shard of a partition into the whole output (offsets: the two uint64
    of shard_offsets) -> (out, this shard's kept count)."""
    n = x.numel()
    dt = dtype_code(x)
    if count_true is None:
        count_true = torch.empty(1, dtype=torch.uint32, device=x.device)
    ws = _ws(ws, OP_PARTITION, n, dt, x.device)
    _check(load().gc_partition_at(_ptr(x), _ptr(out), out.numel(), _ptr(offsets), _ptr(count_true),
                                  n, dt, pred_code(pred), _ptr(ws), ws.numel(), _stream(stream)),
           "gc_partition_at")
    return out, count_true


# ---------------------------------------------------------------- rows
#
# Autograd does not see these calls: their results have no grad_fn, whatever
# requires a gradient among the arguments.  Each gradient is a call of its own.

ROW_DTYPES = {torch.float32: ROW_F32, torch.bfloat16: ROW_BF16, torch.float16: ROW_F16}


class ExpertPlan(NamedTuple):
    """Where gc_expert_dispatch put the pairs (token, choice); int32 tensors."""
    offsets: torch.Tensor  # [experts + 1] first row of each expert's block
    counts: torch.Tensor   # [experts] rows of the block that hold a pair
    slots: torch.Tensor    # [tokens, topk] row of each pair, -1 if dropped
    pairs: torch.Tensor    # [rows] pair of each row, -1 if none


def row_dtype_code(dtype: torch.dtype) -> int:
    code = ROW_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"libgc handles rows of float32, bfloat16 and float16, not {dtype}")
    return code


def _rows(t: torch.Tensor) -> tuple[int, int]:
    """(pointer, row stride) of a 2-D tensor whose rows are contiguous."""
    _on_device(t)
    stride, shape = t.stride(), t.shape
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError("libgc takes 2-D row arrays whose rows are contiguous")
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1]


# The current stream's handle without the stream object that
# torch.cuda.current_stream() makes (0.1 against 2.8 us a call).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, device: torch.device) -> int:
    if stream is None and _current_raw_stream is not None:
        return _current_raw_stream(device.index)
    return _stream(stream)


def _ids(t: torch.Tensor) -> int:
    if t.dtype == torch.int64:
        return ID_I64
    if t.dtype == torch.int32:
        return ID_I32
    raise TypeError(f"libgc takes int32 or int64 ids, not {t.dtype}")


def _typed(t: torch.Tensor | None, dtype: torch.dtype, n: int, what: str) -> int | None:
    """Pointer of a contiguous tensor of n elements of dtype (None stays None)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{what} is a {dtype} tensor, not {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} elements, not {n}")
    return _ptr(t)


def _new(shape, dtype: torch.dtype, device, stream, value=None) -> torch.Tensor:
    """A tensor whose memory belongs to the stream that the call runs on."""
    if stream is None:
        if value is None:
            return torch.empty(shape, dtype=dtype, device=device)
        return torch.full(shape, value, dtype=dtype, device=device)
    s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        return _new(shape, dtype, device, None, value)


def _like(t: torch.Tensor | None, shape, dtype: torch.dtype, device, stream, what: str) -> torch.Tensor:
    """The caller's output, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{what} is a {dtype} tensor of shape {tuple(shape)}")
    return t


def _scratch(ws: torch.Tensor | None, nbytes: int, device, stream) -> torch.Tensor:
    return ws if ws is not None else _new(max(nbytes, 256), torch.uint8, device, stream)


# gc_expert_workspace_bytes of a dispatch whose workspace is checked and not touched.
EXPERT_WORKSPACE_UNUSED = 256


@lru_cache(maxsize=None)
def _untouched(device: torch.device) -> torch.Tensor:
    """What such calls on a device pass as their workspace."""
    return torch.empty(EXPERT_WORKSPACE_UNUSED, dtype=torch.uint8, device=device)


@lru_cache(maxsize=1024)
def expert_rows(tokens: int, topk: int, experts: int, align: int = 1) -> int:
    """gc_expert_rows: rows that hold any routing (0 for arguments out of range)."""
    return int(load().gc_expert_rows(tokens, topk, experts, align))


@lru_cache(maxsize=1024)
def expert_workspace_bytes(tokens: int, topk: int, experts: int) -> int:
    return int(load().gc_expert_workspace_bytes(tokens, topk, experts))


def expert_dispatch(x: torch.Tensor | None, ids: torch.Tensor, experts: int, align: int = 1,
                    out: torch.Tensor | None = None, plan: ExpertPlan | None = None,
                    ws: torch.Tensor | None = None, stream=None):
    """Tokens' rows sorted by expert -> (rows, plan).

    x: [tokens, width] rows; ids: [tokens, topk] int32 or int64, ids outside
    [0, experts) are dropped.  rows: [expert_rows(...), width], each expert's
    block starting at a multiple of `align`; rows without a pair are zeros.
    x None makes the plan alone (rows None).  The gradient with respect to x is
    expert_dispatch_grad; autograd does not see the call.
    """
    shape = ids.shape
    if len(shape) != 2:
        raise ValueError("ids is [tokens, topk]")
    tokens, topk = shape
    dev = ids.device
    need = expert_workspace_bytes(tokens, topk, experts)
    if plan is None:
        rows = expert_rows(tokens, topk, experts, align)
        if need == 0 or (rows == 0 and tokens > 0):
            raise GcError(1, "gc_expert_dispatch")  # arguments out of range
        # four tensors: each costs the host less than a view of a common one
        plan = ExpertPlan(_new(experts + 1, torch.int32, dev, stream), _new(experts, torch.int32, dev, stream),
                          _new(shape, torch.int32, dev, stream), _new(rows, torch.int32, dev, stream))
        where = (plan.offsets.data_ptr(), plan.counts.data_ptr(), plan.slots.data_ptr(), plan.pairs.data_ptr())
    else:
        rows = plan.pairs.numel()
        where = (_typed(plan.offsets, torch.int32, experts + 1, "plan.offsets"),
                 _typed(plan.counts, torch.int32, experts, "plan.counts"),
                 _typed(plan.slots, torch.int32, tokens * topk, "plan.slots"),
                 _typed(plan.pairs, torch.int32, rows, "plan.pairs"))
    if ws is None:
        ws = _untouched(dev) if need == EXPERT_WORKSPACE_UNUSED else _scratch(None, need, dev, stream)
    xp, xs, op, os, width, dt = None, 0, None, 0, 0, ROW_F32
    if x is not None:
        xp, xs = _rows(x)
        n, width = x.shape
        if n != tokens:
            raise ValueError(f"x has {n} rows, ids has {tokens} tokens")
        dt = row_dtype_code(x.dtype)
        out = _like(out, (rows, width), x.dtype, dev, stream, "out")
        op, os = _rows(out)
    _check(load().gc_expert_dispatch(
        _ptr(ids), _ids(ids), tokens, topk, experts, align, xp, xs, width, dt, op, os, rows, *where, _ptr(ws),
        ws.numel(), _handle(stream, dev)), "gc_expert_dispatch")
    return out, plan


def expert_combine(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[slots[t, j]] (weights None: all 1; slot -1: nothing).

    The gradients are expert_combine_grad's; autograd does not see the call.
    """
    if slots.dim() != 2:
        raise ValueError("slots is [tokens, topk]")
    tokens, topk = slots.shape
    yp, ys = _rows(y)
    rows, width = y.shape
    out = _like(out, (tokens, width), y.dtype, y.device, stream, "out")
    op, os = _rows(out)
    _check(load().gc_expert_combine(
        yp, ys, rows, _typed(slots, torch.int32, tokens * topk, "slots"),
        _typed(weights, torch.float32, tokens * topk, "weights"), tokens, topk, width,
        row_dtype_code(y.dtype), op, os, _handle(stream, y.device)), "gc_expert_combine")
    return out


def expert_dispatch_grad(d_rows: torch.Tensor, slots: torch.Tensor, out: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Gradient of expert_dispatch with respect to x: the sum of the gradients of each token's rows."""
    return expert_combine(d_rows, slots, None, out=out, stream=stream)


def expert_combine_grad(g: torch.Tensor, y: torch.Tensor | None, slots: torch.Tensor, pairs: torch.Tensor,
                        weights: torch.Tensor | None = None, dy: torch.Tensor | None = None,
                        dweights: torch.Tensor | None = None, stream=None):
    """Gradient of expert_combine -> (dy, dweights).

    g: [tokens, width], the gradient of its output.  y None: only dy is
    computed and dweights is None.
    """
    if slots.dim() != 2:
        raise ValueError("slots is [tokens, topk]")
    tokens, topk = slots.shape
    rows = pairs.numel()
    gp, gs = _rows(g)
    if g.size(0) != tokens:
        raise ValueError(f"g has {g.size(0)} rows, slots has {tokens} tokens")
    width = g.size(1)
    dy = _like(dy, (rows, width), g.dtype, g.device, stream, "dy")
    dp, ds = _rows(dy)
    yp, ys, wp = None, 0, None
    if y is not None:
        if tuple(y.shape) != (rows, width) or y.dtype != g.dtype:
            raise ValueError(f"y is a {g.dtype} tensor of shape {(rows, width)}")
        yp, ys = _rows(y)
        dweights = _like(dweights, (tokens, topk), torch.float32, g.device, stream, "dweights")
        wp = _ptr(dweights)
    _check(load().gc_expert_combine_grad(
        gp, gs, yp, ys, rows, _typed(slots, torch.int32, tokens * topk, "slots"),
        _typed(pairs, torch.int32, rows, "pairs"), _typed(weights, torch.float32, tokens * topk, "weights"),
        tokens, topk, width, row_dtype_code(g.dtype), dp, ds, wp, _handle(stream, g.device)), "gc_expert_combine_grad")
    return dy, dweights if y is not None else None


def embedding(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """scale * table[ids], zeros for ids outside the table -> ids.shape + (width,).

    The gradient is embedding_grad; autograd does not see the call.
    """
    n = ids.numel()
    tp, ts = _rows(table)
    vocab, width = table.shape
    out = _like(out, (*ids.shape, width), table.dtype, table.device, stream, "out")
    op, os = _rows(out if out.dim() == 2 else out.view(n, width))
    _check(load().gc_embedding(tp, ts, vocab, width, row_dtype_code(table.dtype), _ptr(ids), _ids(ids), n,
                               scale, op, os, _handle(stream, table.device)), "gc_embedding")
    return out


def embedding_grad_workspace_bytes(n: int, vocab: int, width: int) -> int:
    return int(load().gc_embedding_grad_workspace_bytes(n, vocab, width))


def embedding_grad(g: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                   out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                   accumulate: bool = False, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of embedding with respect to its table -> [vocab, width].

    g: the gradient of embedding's output, ids.shape + (width,).  out_dtype:
    g's type (the default) or float32.  accumulate adds to `out`, leaving the
    rows of absent tokens alone.  Rows whose staged copies did not arrive in
    time are NaN; query_device_status of the caller's `ws` says so too.
    """
    n, width = ids.numel(), g.size(-1)
    if accumulate and out is None:
        raise ValueError("accumulate adds to the caller's out")
    if g.numel() != n * width:
        raise ValueError(f"g has {g.numel()} elements for {n} ids of width {width}")
    gp, gs = _rows(g if g.dim() == 2 else g.view(n, width))
    dt = out_dtype or (out.dtype if out is not None else g.dtype)
    out = _like(out, (vocab, width), dt, g.device, stream, "out")
    op, os = _rows(out)
    lib = load()
    ws = _scratch(ws, lib.gc_embedding_grad_workspace_bytes(n, vocab, width), g.device, stream)
    _check(lib.gc_embedding_grad(gp, gs, row_dtype_code(g.dtype), _ptr(ids), _ids(ids), n, vocab, width, scale,
                                 op, os, row_dtype_code(dt), int(accumulate), _ptr(ws), ws.numel(),
                                 _handle(stream, g.device)), "gc_embedding_grad")
    return out


def testing_embedding_grad_stalled(g: torch.Tensor, ids: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                                   timeout_ns: int, accumulate: bool = False, stream=None) -> int:
    """Test hook (include/gc_testing.h): returns the launch status."""
    gp, gs = _rows(g)
    op, os = _rows(out)
    return int(load().gc_testing_embedding_grad_stalled(
        gp, gs, row_dtype_code(g.dtype), _ptr(ids), _ids(ids), ids.numel(), out.size(0), out.size(1), 1.0, op, os,
        row_dtype_code(out.dtype), int(accumulate), _ptr(ws), ws.numel(), timeout_ns, _handle(stream, g.device)))


def _per_row(v, dtype: torch.dtype, rows: int, device, stream) -> torch.Tensor | None:
    return v if v is None or isinstance(v, torch.Tensor) else _new((rows,), dtype, device, stream, v)


def sample(logits: torch.Tensor, uniform: torch.Tensor | None = None, temperature=None, top_k=None, top_p=None,
           min_p=None, tokens: torch.Tensor | None = None, logprobs: torch.Tensor | None = None, stream=None):
    """One token per row of logits -> (tokens int32, logprobs float32).

    uniform: float32 random numbers of [0, 1), logits' shape; None takes the
    largest logit of every row.  temperature, top_k (int32), top_p, min_p: a
    number or one value per row; None leaves the filter out.
    """
    lp, ls = _rows(logits)
    rows, vocab = logits.shape
    up, us = None, 0
    if uniform is not None:
        if uniform.dtype != torch.float32 or tuple(uniform.shape) != (rows, vocab):
            raise ValueError("uniform is a float32 tensor of logits' shape")
        up, us = _rows(uniform)
    dev = logits.device
    temperature = _per_row(temperature, torch.float32, rows, dev, stream)
    top_k = _per_row(top_k, torch.int32, rows, dev, stream)
    top_p = _per_row(top_p, torch.float32, rows, dev, stream)
    min_p = _per_row(min_p, torch.float32, rows, dev, stream)
    tokens = _like(tokens, (rows,), torch.int32, dev, stream, "tokens")
    logprobs = _like(logprobs, (rows,), torch.float32, dev, stream, "logprobs")
    _check(load().gc_sample(lp, ls, rows, vocab, row_dtype_code(logits.dtype), up, us,
                            _typed(temperature, torch.float32, rows, "temperature"),
                            _typed(top_k, torch.int32, rows, "top_k"),
                            _typed(top_p, torch.float32, rows, "top_p"),
                            _typed(min_p, torch.float32, rows, "min_p"), _ptr(tokens), _ptr(logprobs),
                            _handle(stream, dev)), "gc_sample")
    return tokens, logprobs
