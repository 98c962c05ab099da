"""ctypes binding of the calls on caches in pages (spec_cache_compact and
spec_page_fork, include/specverify.h): argument marshalling only.  Streams,
devices and plans are as in beam.py.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from .beam import _DevicePlan, _vector, _workspace
from .binding import _check, _longest, _on, load_library


class PoolT(C.Structure):
    """sv_pool_t."""
    _fields_ = [("slabs", C.c_int32), ("pages", C.c_int32), ("page_size", C.c_int32), ("heads", C.c_int32),
                ("row_bytes", C.c_int64), ("slab_stride", C.c_int64), ("page_stride", C.c_int64),
                ("head_stride", C.c_int64), ("position_stride", C.c_int64)]


class CompactShapeT(C.Structure):
    """sv_compact_shape_t."""
    _fields_ = [("pool", PoolT), ("batch", C.c_int32), ("max_draft", C.c_int32), ("total_draft", C.c_int32),
                ("max_pages", C.c_int32), ("table_stride", C.c_int64), ("cu_draft", C.c_void_p),
                ("page_table", C.c_void_p)]


class ForkShapeT(C.Structure):
    """sv_fork_shape_t."""
    _fields_ = [("pool", PoolT), ("old", C.c_int32), ("batch", C.c_int32), ("beams", C.c_int32),
                ("max_pages", C.c_int32), ("table_stride", C.c_int64), ("out_table_stride", C.c_int64)]


def _pool(t):
    """The C pool of [slabs, pages, page_size, row], the same with heads before page_size, or one slab of [pages,
    page_size, row]."""
    if t.dim() not in (3, 4, 5):
        raise ValueError("pool must be [pages, page_size, row], [slabs, pages, page_size, row] or [slabs, pages, heads, "
                         "page_size, row]")
    if t.device.type != "cuda":
        raise ValueError("pool must be on a GPU")
    if t.numel() == 0:
        raise ValueError(f"pool is empty: {tuple(t.shape)}")
    v = t[None, :, None] if t.dim() == 3 else t[:, :, None] if t.dim() == 4 else t
    if v.shape[4] > 1 and v.stride(4) != 1:
        raise ValueError("pool must have unit stride in its last dimension")
    slabs, pages, heads, size, row = v.shape
    es = t.element_size()
    st = [v.stride(i) * es for i in range(4)]
    return PoolT(slabs, pages, size, heads, row * es, st[0], st[1], st[2], st[3])


def _table(t, name, rows, dev):
    """Pointer, entries per row and row stride of a page table [rows, max_pages]."""
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or t.shape[0] < 1 or t.shape[1] < 1:
        raise ValueError(f"{name} must be [{'sequences' if rows is None else rows}, max_pages], got {tuple(t.shape)}")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be {torch.int32}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device} but the call runs on {dev}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return C.c_void_p(t.data_ptr()), t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _batch(rows, cu_draft, max_draft, batch, stream):
    """(max_draft, total_draft) of `rows` packed rows of `batch` sequences."""
    total = rows - batch
    if total < 0:
        raise ValueError(f"{rows} rows; {batch} sequences need one each at least")
    if cu_draft is None:
        if total % batch != 0:
            raise ValueError("rows must be batch * (K + 1); pass cu_draft for ragged K")
        if max_draft is not None and max_draft != total // batch:
            raise ValueError("max_draft does not match the uniform draft length")
        return total // batch, total
    return int(_longest(cu_draft, stream) if max_draft is None else max_draft), total


class CompactCachePlan(_DevicePlan):
    """spec_cache_compact with every argument marshalled once: __call__
    enqueues one call and returns the new lengths, the same tensor every time.
    See compact_cache."""

    name = "spec_cache_compact"

    def __init__(self, pool, path, num_accepted, lengths=None, page_table=None, cu_draft=None, max_draft=None, out=None,
                 stream=None):
        lib = load_library()
        shape = CompactShapeT(pool=_pool(pool))
        dev, batch = pool.device, num_accepted.numel()
        if batch < 1:
            raise ValueError("num_accepted needs one entry per sequence")
        accepted = _vector(num_accepted, "num_accepted", batch, torch.int32, dev)
        cu = None if cu_draft is None else _vector(cu_draft, "cu_draft", batch + 1, torch.int32, dev)
        kmax, total = _batch(path.numel(), cu_draft, max_draft, batch, stream)
        shape.batch, shape.max_draft, shape.total_draft, shape.cu_draft = batch, kmax, total, cu
        if page_table is None:
            if shape.pool.pages < batch:
                raise ValueError(f"pool holds {shape.pool.pages} sequences; {batch} are needed without a page_table")
            shape.max_pages = 1
        else:
            shape.page_table, shape.max_pages, shape.table_stride = _table(page_table, "page_table", batch, dev)
        before = None if lengths is None else _vector(lengths, "lengths", batch, torch.int32, dev)
        rows = _vector(path, "path", total + batch, torch.int32, dev)
        with _on(dev, stream):
            if out is None:
                out = torch.empty(batch, dtype=torch.int32, device=dev)
        self.out, self.shape = out, shape
        self._own(dev, stream, out)
        self._keep = (pool, path, num_accepted, lengths, page_table, cu_draft)
        self.args = (C.byref(shape), C.c_void_p(pool.data_ptr()), before, rows, accepted,
                     _vector(out, "out", batch, torch.int32, dev))
        self.fn, self.fn_profiled = lib.spec_cache_compact, lib.spec_cache_compact_profiled


def compact_cache(pool: torch.Tensor, path: torch.Tensor, num_accepted: torch.Tensor,
                  lengths: Optional[torch.Tensor] = None, page_table: Optional[torch.Tensor] = None,
                  cu_draft: Optional[torch.Tensor] = None, max_draft: Optional[int] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The accepted rows of a verify moved behind the context, in place, on the
    GPU (spec_cache_compact).

    pool: any dtype, [slabs, pages, page_size, row], [slabs, pages, heads,
    page_size, row] or [pages, page_size, row], any strides without overlap (last
    dimension contiguous); path int32 [sum(K_b + 1)] and num_accepted int32
    [batch], as verify_tree_greedy and verify_tree_sample return them; lengths int32 [batch], the
    positions in use with the newest K_b + 1 rows (None: all); page_table int32
    [batch, max_pages], or None: page b is sequence b's whole cache.  cu_draft
    int32 [batch + 1] or None (uniform K); max_draft is read back from the device
    where it is needed and not given.  Returns the new lengths, int32 [batch]
    (`out`, which may not be `lengths`).
    """
    return CompactCachePlan(pool, path, num_accepted, lengths, page_table, cu_draft, max_draft, out, stream)()


class ForkPagesPlan(_DevicePlan):
    """spec_page_fork with every argument marshalled once: __call__ enqueues one
    call and returns {"page_table", "refs", "free"}, the same tensors every time.
    See fork_pages."""

    name = "spec_page_fork"

    def __init__(self, pool, page_table, lengths, parents, refs, new_lengths=None, beams=None, out=None, workspace=None,
                 stream=None):
        lib = load_library()
        shape = ForkShapeT(pool=_pool(pool))
        dev = pool.device
        table, max_pages, stride = _table(page_table, "page_table", None, dev)
        old = page_table.shape[0]
        batch = old if parents is None else parents.numel()
        if batch < 1:
            raise ValueError("parents needs one entry per place")
        beams = 0 if beams is None else int(beams)
        if beams < 0 or (beams > 0 and (batch % beams != 0 or old % beams != 0)):
            raise ValueError(f"{old} sequences and {batch} places; a multiple of beams = {beams} is needed")
        before = _vector(lengths, "lengths", old, torch.int32, dev)
        counts = _vector(refs, "refs", shape.pool.pages, torch.int32, dev)
        who, room = [None if t is None else _vector(t, n, batch, torch.int32, dev)
                     for n, t in (("parents", parents), ("new_lengths", new_lengths))]
        with _on(dev, stream):
            if out is None:
                out = {"page_table": torch.empty((batch, max_pages), dtype=torch.int32, device=dev),
                       "refs": torch.empty(shape.pool.pages, dtype=torch.int32, device=dev),
                       "free": torch.empty(1, dtype=torch.int32, device=dev)}
        new, entries, out_stride = _table(out["page_table"], "out['page_table']", batch, dev)
        if entries != max_pages:
            raise ValueError(f"out['page_table'] has {entries} entries a row; {max_pages} are needed")
        outs = (new, _vector(out["refs"], "out['refs']", shape.pool.pages, torch.int32, dev),
                _vector(out["free"], "out['free']", 1, torch.int32, dev))
        shape.old, shape.batch, shape.beams, shape.max_pages = old, batch, beams, max_pages
        shape.table_stride, shape.out_table_stride = stride, out_stride
        need = C.c_size_t(0)
        _check(lib.spec_page_fork(C.byref(shape), C.c_void_p(pool.data_ptr()), *[None] * 9, C.byref(need), None),
               "spec_page_fork(workspace query)")
        with _on(dev, stream):
            self.workspace = _workspace(workspace, need.value, dev)
        self.out, self.shape = out, shape
        self._own(dev, stream, self.workspace, *out.values())
        self.have = C.c_size_t(self.workspace.numel())
        self._keep = (pool, page_table, lengths, parents, refs, new_lengths)
        self.args = (C.byref(shape), C.c_void_p(pool.data_ptr()), table, before, who, room, counts, *outs,
                     C.c_void_p(self.workspace.data_ptr()), C.byref(self.have))
        self.fn, self.fn_profiled = lib.spec_page_fork, lib.spec_page_fork_profiled


def fork_pages(pool: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor, parents: Optional[torch.Tensor],
               refs: torch.Tensor, new_lengths: Optional[torch.Tensor] = None, beams: Optional[int] = None,
               out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """The page tables of sequences that continue others, on the GPU
    (spec_page_fork): whole pages shared, a page that is still written copied
    where a second place takes it, pages for new positions given, pages that
    nobody holds any more freed.

    pool as for compact_cache; page_table int32 [old, max_pages] and lengths int32
    [old], the tables and positions in use so far; parents int32 [places], the
    sequence that each place continues (-1: none; with `beams` within its group,
    as beam_select returns them; None: its own); refs int32 [pages], the holders of
    each page; new_lengths int32 [places], the positions to hold pages for.
    Returns page_table [places, max_pages], refs [pages] and free [1], the pages
    left (below 0: so many were missing).  out["refs"] may be `refs`.
    """
    return ForkPagesPlan(pool, page_table, lengths, parents, refs, new_lengths, beams, out, workspace, stream)()
