"""Pools of states that serving steps read (gdn_step, glr_step): slots copied, forked, freed and
compacted on the device (include/pool.h): argument marshalling only.

A pool is a contiguous tensor [slots, ...] of any dtype; a call takes one pool or several (a model's
layers), which share their slot numbers. `used` is a bool tensor [slots]: which slots hold a sequence's
state. Free slots that these calls leave are clear (zero), and nothing here reads an index on the host,
so a serving loop can capture them in a graph.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import PoolRef, load
from .api import _INT32, _call, _check, _ptr


def _pools(pools, device=None):
    """(references, number, slots, device) of the checked pools."""
    if torch.is_tensor(pools):
        pools = (pools,)
    refs = (PoolRef * max(len(pools), 1))()
    slots = None
    for r, p in zip(refs, pools):
        if p.dim() < 1 or not p.is_contiguous():
            raise ValueError("a pool must be contiguous, [slots, ...]")
        n, d = p.shape[0], p.device
        if n > _INT32:
            raise ValueError(f"at most 2^31 - 1 slots (got {n})")
        if d.type != "cuda" or (device is not None and d != device):
            raise ValueError("pools must be on one HIP device")
        if slots is not None and n != slots:
            raise ValueError("pools of one call must have one number of slots")
        slots, device = n, d
        r.data = p.data_ptr()
        size = p.numel() // slots if slots else 1
        r.bytes = size * p.element_size()
        if size == 0:
            raise ValueError("a pool's slots must not be empty")
    return refs, len(pools), slots, device


def _sources(sources, pools):
    """(pointers, slots) of what is copied from: tensors like the pools, with a number of slots of their own."""
    if sources is None:
        return None, 0
    pools = (pools,) if torch.is_tensor(pools) else pools
    sources = (sources,) if torch.is_tensor(sources) else sources
    if len(sources) != len(pools) or not sources:
        raise ValueError("as many sources as pools are needed")
    for s, p in zip(sources, pools):
        _check(s, "sources", p.dtype, (sources[0].shape[0], *p.shape[1:]), p.device)
    n = sources[0].shape[0]
    if n > _INT32:
        raise ValueError(f"sources: at most 2^31 - 1 slots (got {n})")
    return (ctypes.c_void_p * len(sources))(*(s.data_ptr() for s in sources)), n


def _indices(t, name, device, n=None):
    _check(t, name, torch.int32, (t.numel() if n is None else n,), device)


def _used(used, slots, device):
    if slots is None:                       # no pools
        slots, device = used.numel(), used.device
        if slots > _INT32:
            raise ValueError(f"at most 2^31 - 1 slots (got {slots})")
        if device.type != "cuda":
            raise ValueError("used must be on a HIP device")
    _check(used, "used", torch.bool, (slots,), device)
    return slots, device


def pool_copy(pools, src=None, dst=None, sources=None):
    """Slot src[i] becomes slot dst[i], in every pool. src, dst: int32 tensors [n] (None: 0, 1, ..); a pair with an
    index out of range is skipped. sources: tensors [m, ...] like the pools to copy from (a prefill's final
    states, another pool), or None for the pools themselves. No destination may be named twice, nor be another
    pair's source in the same pool."""
    refs, n_pools, slots, dev = _pools(pools)
    if not n_pools:
        raise ValueError("at least one pool is needed")
    ptrs, m = _sources(sources, pools)
    if src is None and dst is None:
        n = m if ptrs is not None else slots
    else:
        n = (dst if src is None else src).numel()
    for t, name in ((src, "src"), (dst, "dst")):
        if t is not None:
            _indices(t, name, dev, n)
    _call(load().pool_copy, "pool_copy", dev, None, refs, n_pools, slots, ptrs, m, _ptr(src), _ptr(dst), n)


def pool_fork(pools, used, src=None, sources=None):
    """Each i whose src[i] (int32 [n]) names a used slot takes a free one, in order the lowest one left, which
    becomes a copy in every pool and used. Returns the slots, int32 [n]: -1 where src[i] names none, or where no
    free slot is left. sources as in pool_copy (src[i] is then one of theirs, and None all of them)."""
    refs, n_pools, slots, dev = _pools(pools)
    slots, dev = _used(used, slots, dev)
    ptrs, m = _sources(sources, pools)
    if src is None and ptrs is None:
        raise ValueError("src or sources are needed (pool_alloc takes slots without a copy)")
    if src is not None:
        _indices(src, "src", dev)
    n = m if src is None else src.numel()
    dst = used.new_empty(n, dtype=torch.int32)
    _call(load().pool_fork, "pool_fork", dev, None, refs, n_pools, slots, ptrs, m, used.data_ptr(), _ptr(src),
          dst.data_ptr(), n)
    return dst


def pool_alloc(used, n):
    """The n lowest free slots, which become used: int32 [n], -1 where none is left. They are as they were
    (clear, where pool_free or pool_compact left them)."""
    slots, dev = _used(used, None, None)
    if n < 0:
        raise ValueError(f"n must not be negative (got {n})")
    dst = torch.empty(n, dtype=torch.int32, device=dev)
    _call(load().pool_fork, "pool_alloc", dev, None, None, 0, slots, None, 0, used.data_ptr(), None, dst.data_ptr(), n)
    return dst


def pool_free(pools, used, indices):
    """The slots that indices (int32 [n]) name become free, and clear in every pool. An index may be named more
    than once or be out of range (skipped)."""
    refs, n_pools, slots, dev = _pools(pools)
    slots, dev = _used(used, slots, dev)
    _indices(indices, "indices", dev)
    _call(load().pool_free, "pool_free", dev, None, refs, n_pools, slots, used.data_ptr(), indices.data_ptr(),
          indices.numel())


def pool_compact(pools, used, indices):
    """The used slots move to the front of every pool, into the free ones there (in order); where they were is
    clear. indices (int32 [n], the slots of all rows in flight: a copy kept elsewhere goes stale) are renumbered in
    place. Returns the number of used slots, int32 [1] on the device."""
    refs, n_pools, slots, dev = _pools(pools)
    slots, dev = _used(used, slots, dev)
    _indices(indices, "indices", dev)
    count = indices.new_empty(1)
    ws = used.new_empty(load().pool_compact_workspace_bytes(slots) or 256, dtype=torch.uint8)
    _call(load().pool_compact, "pool_compact", dev, None, refs, n_pools, slots, used.data_ptr(), indices.data_ptr(),
          indices.numel(), count.data_ptr(), ws.data_ptr(), ws.numel())
    return count
