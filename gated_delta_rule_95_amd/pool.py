"""Torch front of the state pools' entry points (C ABI: include/pool.h).

    pool_alloc(pools, used, n) -> slots         (free slots taken, zeroed)
    pool_fork(pools, used, src) -> dst          (free slots taken for copies)
    pool_free(used, slots)
    pool_compact(pools, used, table=None) -> remap
    pool_copy(from_pools, src, to_pools, dst)

pools: a tensor [n_slots, ...], or a list of them with the same n_slots (the
states of each layer, of any shapes and dtypes): request state j is slot j of
every pool.  used: bool [n_slots] on the device, which slots are taken, read
and updated by the calls.  Marshalling only: the work runs in the library's
kernels on the device of the slot numbers and its current stream.
"""
from __future__ import annotations

import array
import math
from typing import Optional, Sequence, Union

import torch

from . import _lib
from .gdr import _need, _ptr
from .glr import _int32, _run

__all__ = ["pool_alloc", "pool_fork", "pool_free", "pool_compact", "pool_copy",
           "pool_compact_workspace_bytes"]

Pools = Union[torch.Tensor, Sequence[torch.Tensor]]


def _device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} is on {t.device}: the kernels run on a GPU, there is no CPU fallback")
    return t.device


def _rows(pools: Pools, name: str, n_slots: Optional[int], dev):
    """The pools as an array of (address, bytes a row) and their count of slots."""
    if isinstance(pools, torch.Tensor):
        pools = (pools,)
    words = []
    for p in pools:
        if not isinstance(p, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor or a list of them")
        shape = p.shape
        if not shape:
            raise ValueError(f"{name} must be [n_slots, ...]")
        if n_slots is None:
            n_slots = shape[0]
            _int32((n_slots, "n_slots"))
        if shape[0] != n_slots or p.device != dev or not p.is_contiguous():
            _need(p, name, p.dtype, (n_slots,) + shape[1:], dev)
        row = math.prod(shape[1:]) * p.element_size()
        if row == 0:
            raise ValueError(f"{name} must have rows of one element at least")
        words += (p.data_ptr(), row)
    return array.array("Q", words), len(words) // 2, 0 if n_slots is None else n_slots


def _used(used):
    if isinstance(used, torch.Tensor) and used.dtype is torch.bool and used.is_cuda and used.dim() == 1 \
            and used.is_contiguous() and not used.shape[0] >> 31:
        return used.device, used.shape[0]
    dev = _device(used, "used")
    if used.dim() != 1:
        raise ValueError("used must be [n_slots]")
    _int32((used.shape[0], "n_slots"))
    _need(used, "used", torch.bool, used.shape, dev)
    return dev, used.shape[0]


def _numbers(t, name, dev):
    if isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == dev and t.dim() == 1 and t.is_contiguous() \
            and not t.shape[0] >> 31:
        return t.shape[0]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 1:
        raise ValueError(f"{name} must have one dimension")
    _int32((t.shape[0], f"the length of {name}"))
    _need(t, name, torch.int32, t.shape, dev)
    return t.shape[0]


def pool_alloc(pools: Pools, used: torch.Tensor, n: int) -> torch.Tensor:
    """Takes n free slots, lowest numbers first, writes zeros to their rows and
    marks them in used.  Returns their numbers, int32 [n] on the device; -1
    where no free slot is left."""
    dev, n_slots = _used(used)
    rows, k, _ = _rows(pools, "pools", n_slots, dev)
    if n < 0:
        raise ValueError("n must be >= 0")
    _int32((n, "n"))
    slots = torch.empty(n, dtype=torch.int32, device=dev)
    _run(dev, _lib.load().pool_alloc, rows.buffer_info()[0], k, _ptr(used), n_slots, n, _ptr(slots))
    return slots


def pool_fork(pools: Pools, used: torch.Tensor, src: torch.Tensor) -> torch.Tensor:
    """Takes a free slot for a copy of each slot src[i] (int32 [n] on the device,
    the same one any number of times).  Returns the copies' slots, int32 [n]:
    the lowest free ones, in order; -1 where src[i] is no used slot or no free
    slot is left."""
    dev, n_slots = _used(used)
    n = _numbers(src, "src", dev)
    rows, k, _ = _rows(pools, "pools", n_slots, dev)
    dst = torch.empty_like(src)
    _run(dev, _lib.load().pool_fork, rows.buffer_info()[0], k, _ptr(used), n_slots, _ptr(src), n, _ptr(dst))
    return dst


def pool_free(used: torch.Tensor, slots: torch.Tensor) -> None:
    """Marks the slots (int32 [n] on the device) as free; numbers outside the
    pool and free slots are ignored."""
    dev, n_slots = _used(used)
    n = _numbers(slots, "slots", dev)
    _run(dev, _lib.load().pool_free, _ptr(used), n_slots, _ptr(slots), n)


def pool_compact_workspace_bytes(n_slots: int) -> int:
    """Bytes of workspace pool_compact needs for this count of slots (0 for one that it refuses)."""
    return 0 if n_slots >> 31 else int(_lib.load().pool_compact_workspace_bytes(n_slots))


def pool_compact(pools: Pools, used: torch.Tensor, table: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Moves the used slots to the front: with m of them, those at m and behind
    go, in order, into the free ones below m.  used is updated, and the entries
    of table (int32 on the device, any shape) that are slot numbers are
    rewritten (-1 where one named a free slot).  Returns int32 [n_slots]: each
    used slot's new number, -1 for a free one."""
    dev, n_slots = _used(used)
    rows, k, _ = _rows(pools, "pools", n_slots, dev)
    if table is not None:
        _need(table, "table", torch.int32, getattr(table, "shape", None), dev)
    if workspace is None:
        workspace = torch.empty(pool_compact_workspace_bytes(n_slots), dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), dev)
    remap = torch.empty(n_slots, dtype=torch.int32, device=dev)
    _run(dev, _lib.load().pool_compact, rows.buffer_info()[0], k, _ptr(used), n_slots, _ptr(table),
         0 if table is None else table.numel(), _ptr(remap), _ptr(workspace), workspace.numel())
    return remap


def pool_copy(from_pools: Pools, src: torch.Tensor, to_pools: Pools, dst: torch.Tensor) -> None:
    """Copies slot src[i] of each of from_pools to slot dst[i] of its counterpart
    in to_pools (int32 [n] on the device): the same pools, or others of the same
    rows with another number of slots.  Pairs with a number outside the pools
    are left out; a slot must not be two pairs' destination, nor one's
    destination and another's source in the same pools."""
    dev = _device(src, "src")
    n = _numbers(src, "src", dev)
    if _numbers(dst, "dst", dev) != n:
        raise ValueError("dst must be as long as src")
    a, k, from_slots = _rows(from_pools, "from_pools", None, dev)
    b, m, to_slots = _rows(to_pools, "to_pools", None, dev)
    if k != m:
        raise ValueError("to_pools must be as many as from_pools")
    _run(dev, _lib.load().pool_copy, a.buffer_info()[0], b.buffer_info()[0], k, from_slots, to_slots, _ptr(src), _ptr(dst), n)
