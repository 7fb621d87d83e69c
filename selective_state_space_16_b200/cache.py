"""ctypes binding of the state cache (include/ssm_cache.h): argument marshalling only."""
from __future__ import annotations

import ctypes
import struct

import torch

from .binding import _check
from .gated import _buffer, _call, _dense, _lib

SSM_CACHE_NEW = -1  # as a parent: the page of a new sequence, all zeros
MAX_POOLS = 8
_POOL = struct.Struct("@Pqqqi4x")  # ssm_cache_pool_t
_I32 = (torch.int32,)


def declare(lib: ctypes.CDLL) -> None:
    """Declare the argument and result types of this header's entry points."""
    vp, ci, sz, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_char_p
    lib.ssm_cache_workspace_size.argtypes = [ci, ci]
    lib.ssm_cache_workspace_size.restype = sz
    lib.ssm_cache_copy.argtypes = [st, ci, ci, vp, vp, ci, vp, sz, vp]
    lib.ssm_cache_copy.restype = ci
    lib.ssm_cache_fork.argtypes = [st, ci, ci, vp, vp, vp, ci, vp, sz, vp]
    lib.ssm_cache_fork.restype = ci
    lib.ssm_cache_free.argtypes = [st, ci, ci, vp, vp, ci, ci, vp]
    lib.ssm_cache_free.restype = ci
    lib.ssm_cache_compact.argtypes = [st, ci, ci, vp, vp, ci, vp, vp, vp, sz, vp]
    lib.ssm_cache_compact.restype = ci


class CachePools:
    """The pools of a cache: tensors (layers, slots, ...) of any types, whose pages (the part behind the first
    two dimensions) are dense.  They are described to the library once, here, and kept alive by this object."""

    def __init__(self, tensors):
        tensors = list(tensors)
        if not 1 <= len(tensors) <= MAX_POOLS:
            raise ValueError(f"{len(tensors)} pools (1 to {MAX_POOLS})")
        packed = []
        for k, t in enumerate(tensors):
            if t.dim() < 2 or not t.is_cuda:
                raise ValueError(f"pool {k}: expected a CUDA tensor (layers, slots, ...)")
            if t.shape[1] != tensors[0].shape[1] or t.device != tensors[0].device:
                raise ValueError(f"pool {k}: {t.shape[1]} slots on {t.device} (pool 0: {tensors[0].shape[1]} on {tensors[0].device})")
            dense = 1
            for size, stride in zip(reversed(t.shape[2:]), reversed(t.stride()[2:])):
                if size > 1 and stride != dense:
                    raise ValueError(f"pool {k}: a page is not dense")
                dense *= size
            e = t.element_size()
            packed.append(_POOL.pack(t.data_ptr(), dense * e, t.stride(1) * e, t.stride(0) * e, t.shape[0]))
        self.tensors, self.n_slots, self.device = tensors, tensors[0].shape[1], tensors[0].device
        self.index = tensors[0].get_device()
        self.packed, self.n_pools = b"".join(packed), len(tensors)


def _list(t, name, pools):
    if t is None or t.dim() != 1:
        raise ValueError(f"{name}: expected a list of slots (int32, one dimension)")
    return _dense(t, name, t.shape, _I32, pools.index)


def ssm_cache_workspace_size(n_slots: int, n: int) -> int:
    return int(_lib().ssm_cache_workspace_size(n_slots, n))


def new_cache_workspace(pools, n=0, device=None):
    """Allocate (with torch) a workspace for calls on these pools with lists of up to n entries."""
    return torch.empty(ssm_cache_workspace_size(pools.n_slots, n), dtype=torch.uint8, device=device or pools.device)


def ssm_cache_copy(pools, src, dst, workspace, stream=None, check=True):
    """Copy page src[j] to page dst[j], as if one after another.  src, dst: (n) int32."""
    a, b = _list(src, "src", pools), _list(dst, "dst", pools)
    if src.shape != dst.shape:
        raise ValueError(f"{src.numel()} sources, {dst.numel()} destinations")
    code = _call(pools.index, stream, _lib().ssm_cache_copy, pools.packed, pools.n_pools, pools.n_slots, a, b, src.numel(),
                 *_buffer(workspace, "workspace", pools.index))
    if check:
        _check(code, "ssm_cache_copy")
    return code


def ssm_cache_fork(pools, used, parents, children, workspace, stream=None, check=True):
    """Fork sequences into free slots.  used: (slots) int32 in/out; parents: (n) int32 (SSM_CACHE_NEW: a page of
    zeros); children: (n) int32 output, -1 where there was no such parent or no slot left."""
    a, b = _list(parents, "parents", pools), _list(children, "children", pools)
    if parents.shape != children.shape:
        raise ValueError(f"{parents.numel()} parents, {children.numel()} children")
    code = _call(pools.index, stream, _lib().ssm_cache_fork, pools.packed, pools.n_pools, pools.n_slots,
                 _dense(used, "used", (pools.n_slots,), _I32, pools.index), a, b, parents.numel(),
                 *_buffer(workspace, "workspace", pools.index))
    if check:
        _check(code, "ssm_cache_fork")
    return code


def ssm_cache_free(pools, used, slots, zero_pages=False, stream=None, check=True):
    """Free the listed slots (used = 0), with zero_pages also clearing their pages."""
    a = _list(slots, "slots", pools)
    code = _call(pools.index, stream, _lib().ssm_cache_free, pools.packed, pools.n_pools, pools.n_slots,
                 _dense(used, "used", (pools.n_slots,), _I32, pools.index), a, slots.numel(), int(bool(zero_pages)))
    if check:
        _check(code, "ssm_cache_free")
    return code


def ssm_cache_compact(pools, used, table, remap, count, workspace, stream=None, check=True):
    """Move the used pages to the front.  used: (slots) int32 in/out; table: (n) int32 slots that follow their pages,
    or None; remap: (slots) int32 output or None; count: (1) int32 output or None."""
    code = _call(pools.index, stream, _lib().ssm_cache_compact, pools.packed, pools.n_pools, pools.n_slots,
                 _dense(used, "used", (pools.n_slots,), _I32, pools.index), 0 if table is None else _list(table, "table", pools),
                 0 if table is None else table.numel(), _dense(remap, "remap", (pools.n_slots,), _I32, pools.index),
                 _dense(count, "count", (1,), _I32, pools.index), *_buffer(workspace, "workspace", pools.index))
    if check:
        _check(code, "ssm_cache_compact")
    return code
