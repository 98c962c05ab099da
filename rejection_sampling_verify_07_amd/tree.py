"""ctypes binding of the calls on trees of guesses (spec_tree_attention,
spec_adjust_logits, spec_verify_tree_greedy, spec_verify_tree_sample;
include/specverify.h): argument marshalling only.  Streams, devices and plans are
as in beam.py.  A cu_draft may end before the rows do (a step of fixed size that
holds fewer guesses): rows behind the last sequence's are left as they were.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import binding as _b
from .beam import CacheT, _DevicePlan, _rows3, _vector, _workspace
from .binding import _check, _on, load_library
from .pages import _batch, _table


class AdjustShapeT(C.Structure):
    """sv_adjust_shape_t."""
    _fields_ = [("batch", C.c_int32), ("max_draft", C.c_int32), ("total_draft", C.c_int32), ("vocab", C.c_int32),
                ("dtype", C.c_int32), ("row_stride", C.c_int64), ("out_row_stride", C.c_int64), ("cu_draft", C.c_void_p),
                ("draft_ids", C.c_void_p), ("parents", C.c_void_p)]


class AdjustT(C.Structure):
    """sv_adjust_t."""
    _fields_ = ([("tokens", C.c_void_p), ("token_stride", C.c_int64), ("max_tokens", C.c_int32),
                 ("total_bias", C.c_int32)]
                + [(n, C.c_void_p) for n in ("lengths", "prompt_lengths", "repetition", "presence", "frequency",
                                             "bias_ids", "bias_values", "cu_bias", "masks")]
                + [("mask_stride", C.c_int64), ("num_masks", C.c_int32), ("mask_rows", C.c_void_p)])


def _matrix(t, name, dtype, dev):
    """Row stride of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device} but the call runs on {dev}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    # (a single row may report any stride)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class AdjustLogitsPlan(_DevicePlan):
    """spec_adjust_logits with every argument marshalled once: __call__ enqueues
    one call and returns `out`, the same tensor every time.  See adjust_logits."""

    name = "spec_adjust_logits"

    def __init__(self, logits, tokens=None, lengths=None, prompt_lengths=None, repetition=None, presence=None,
                 frequency=None, bias_ids=None, bias_values=None, cu_bias=None, masks=None, mask_rows=None,
                 draft_ids=None, parents=None, cu_draft=None, max_draft=None, out=None, stream=None):
        lib = load_library()
        if logits.dim() != 2 or logits.shape[0] < 1 or logits.shape[1] < 1:
            raise ValueError("logits must be a 2-D tensor [sum(K_b + 1), vocab]")
        dev = logits.device
        if dev.type != "cuda":
            raise ValueError("logits must be on a GPU")
        rows, vocab = logits.shape
        # sequences: what tells their number first
        counts = [("cu_draft", cu_draft, -1), ("tokens", tokens, 0), ("lengths", lengths, 0), ("repetition", repetition, 0),
                  ("presence", presence, 0), ("frequency", frequency, 0), ("cu_bias", cu_bias, -1)]
        batch = next((t.shape[0] + extra for _, t, extra in counts if t is not None),
                     rows if draft_ids is None else rows - draft_ids.numel())
        if batch < 1 or batch > rows:
            raise ValueError(f"{rows} rows do not fit {batch} sequences")
        total = rows - batch
        if cu_draft is None:
            if total % batch != 0:
                raise ValueError("logits must have batch * (K + 1) rows; pass cu_draft for ragged K")
            if max_draft is not None and max_draft != total // batch:
                raise ValueError("max_draft does not match the uniform draft length")
            max_draft = total // batch
        sizes = {"cu_draft": batch + 1, "draft_ids": total, "parents": total, "lengths": batch, "prompt_lengths": batch,
                 "repetition": batch, "presence": batch, "frequency": batch, "cu_bias": batch + 1, "mask_rows": rows}
        real = ("repetition", "presence", "frequency")
        given = dict(cu_draft=cu_draft, draft_ids=draft_ids, parents=parents, lengths=lengths,
                     prompt_lengths=prompt_lengths, repetition=repetition, presence=presence, frequency=frequency,
                     cu_bias=cu_bias, mask_rows=mask_rows)
        at = {n: None if t is None else _vector(t, n, sizes[n], torch.float32 if n in real else torch.int32, dev)
              for n, t in given.items()}
        if max_draft is None:
            max_draft = _b._longest(cu_draft, stream)
        adjust = AdjustT(**{n: at[n] for n in ("lengths", "prompt_lengths", *real, "cu_bias", "mask_rows")})
        if tokens is not None:
            if tokens.dim() == 2 and tokens.shape[0] != batch:
                raise ValueError(f"tokens holds {tokens.shape[0]} sequences; {batch} are needed")
            adjust.token_stride = _matrix(tokens, "tokens", torch.int32, dev)
            adjust.tokens, adjust.max_tokens = tokens.data_ptr(), tokens.shape[1]
        if (bias_ids is None) != (bias_values is None):
            raise ValueError("bias_ids and bias_values go together")
        if bias_ids is not None:
            n = bias_ids.numel()
            adjust.bias_ids = _vector(bias_ids, "bias_ids", n, torch.int32, dev)
            adjust.bias_values = _vector(bias_values, "bias_values", n, torch.float32, dev)
            adjust.total_bias = n
        if masks is not None:
            adjust.mask_stride = _matrix(masks, "masks", torch.int32, dev)
            if masks.shape[1] < (vocab + 31) // 32:
                raise ValueError(f"masks has {masks.shape[1]} words a row; {(vocab + 31) // 32} are needed")
            if mask_rows is None and masks.shape[0] < rows:
                raise ValueError(f"masks has {masks.shape[0]} rows; {rows} are needed without mask_rows")
            adjust.masks, adjust.num_masks = masks.data_ptr(), masks.shape[0]
        elif mask_rows is not None:
            raise ValueError("mask_rows needs masks")
        with _on(dev, stream):
            if out is None:
                out = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
        if tuple(out.shape) != (rows, vocab):
            raise ValueError(f"out must be [{rows}, {vocab}], got {tuple(out.shape)}")
        code = _b._dtype_code(logits)
        shape = AdjustShapeT(batch, int(max_draft), total, vocab, code, _matrix(logits, "logits", logits.dtype, dev),
                             _matrix(out, "out", logits.dtype, dev), at["cu_draft"], at["draft_ids"], at["parents"])
        self.out, self.shape = out, shape
        self._own(dev, stream, out)
        self._keep = (logits, tokens, bias_ids, bias_values, masks, *given.values(), adjust)
        self.args = (C.byref(shape), C.byref(adjust), C.c_void_p(logits.data_ptr()), C.c_void_p(out.data_ptr()))
        self.fn, self.fn_profiled = lib.spec_adjust_logits, lib.spec_adjust_logits_profiled


def adjust_logits(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                  prompt_lengths: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                  presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                  bias_ids: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                  cu_bias: Optional[torch.Tensor] = None, masks: Optional[torch.Tensor] = None,
                  mask_rows: Optional[torch.Tensor] = None, draft_ids: Optional[torch.Tensor] = None,
                  parents: Optional[torch.Tensor] = None, cu_draft: Optional[torch.Tensor] = None,
                  max_draft: Optional[int] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Penalties, biases and grammar masks on logits, on the GPU (spec_adjust_logits).

    logits [sum(K_b + 1), V] float32, bfloat16 or float16, rows packed as the
    target rows of a verify (one row per sequence at a plain step).  tokens int32
    [batch, max_tokens], each sequence's text so far, lengths int32 [batch] of it
    in use (None: all), prompt_lengths int32 [batch] of those that count for
    repetition alone (None: 0); draft_ids int32 [sum(K_b)]: the guesses, which count as written in
    the rows behind them, along parents (as for verify_tree_greedy; None: chains).
    repetition, presence, frequency float32 [batch].  bias_ids int32 and bias_values
    float32 [n], sequence b's at cu_bias[b] .. cu_bias[b + 1] (None: all for every
    sequence).  masks int32 [num_masks, words], bit v % 32 of word v // 32 set
    where token v is allowed; mask_rows int32 [rows], each row's mask (-1: none;
    None: row r goes by mask r).  cu_draft int32 [batch + 1] or None (uniform K);
    max_draft is read back from the device where it is needed and not given.
    Returns `out` (may be `logits` itself: in place; None: a new tensor).
    """
    return AdjustLogitsPlan(logits, tokens, lengths, prompt_lengths, repetition, presence, frequency, bias_ids,
                            bias_values, cu_bias, masks, mask_rows, draft_ids, parents, cu_draft, max_draft, out, stream)()


class _TreeVerifyPlan(_DevicePlan):
    """What both verifies of a tree marshal; `filters`: the arguments between parents and the outputs."""

    def __init__(self, target_logits, draft_ids, parents, cu_draft, max_draft, out, workspace, stream, filters):
        lib = load_library()
        fn = getattr(lib, self.name)
        if target_logits.dim() != 2:
            raise ValueError("target_logits must be a 2-D tensor with unit column stride")
        dev = target_logits.device
        if cu_draft is not None and (cu_draft.dim() != 1 or cu_draft.device != dev):
            raise ValueError(f"cu_draft must be a 1-D tensor on {dev}")
        batch, kmax, total = _b._batch_geometry(target_logits, draft_ids, cu_draft, max_draft, stream)
        # (a single row may report any stride)
        shape = _b.make_shape(target_logits, None, batch, kmax, total, cu_draft, total + batch)
        if target_logits.shape[0] == 1:
            shape.target_row_stride = max(shape.target_row_stride, shape.vocab)
        cu = None if cu_draft is None else _vector(cu_draft, "cu_draft", batch + 1, torch.int32, dev)
        ids = _vector(draft_ids, "draft_ids", total, torch.int32, dev)
        ups = None if parents is None else _vector(parents, "parents", total, torch.int32, dev)
        need = C.c_size_t(0)
        _check(fn(C.byref(shape), None, None, None, *filters, None, None, None, None, C.byref(need), None),
               self.name + "(workspace query)")
        sizes = (("tokens", total + batch), ("num_accepted", batch), ("path", total + batch))
        with _on(dev, stream):
            self.workspace = _workspace(workspace, need.value, dev)
            if out is None:
                out = {k: torch.empty(n, dtype=torch.int32, device=dev) for k, n in sizes}
        outs = [None if k == "path" and out.get(k) is None else _vector(out[k], f"out[{k!r}]", n, torch.int32, dev)
                for k, n in sizes]
        self.out, self.shape = out, shape
        self._own(dev, stream, self.workspace, *(t for t in out.values() if t is not None))
        self.have = C.c_size_t(self.workspace.numel())
        self._keep = (target_logits, draft_ids, parents, cu_draft, cu)
        self.args = (C.byref(shape), C.c_void_p(target_logits.data_ptr()), ids, ups, *filters, *outs,
                     C.c_void_p(self.workspace.data_ptr()), C.byref(self.have))
        self.fn, self.fn_profiled = fn, getattr(lib, self.name + "_profiled")


class TreeGreedyPlan(_TreeVerifyPlan):
    """spec_verify_tree_greedy with every argument marshalled once: __call__
    enqueues one call and returns the outputs, the same tensors every time.  See
    verify_tree_greedy."""

    name = "spec_verify_tree_greedy"

    def __init__(self, target_logits, draft_ids, parents=None, cu_draft=None, max_draft=None, out=None, workspace=None,
                 stream=None):
        super().__init__(target_logits, draft_ids, parents, cu_draft, max_draft, out, workspace, stream, ())


class TreeSamplePlan(_TreeVerifyPlan):
    """spec_verify_tree_sample with every argument marshalled once: __call__(offset)
    enqueues one call and returns the outputs, the same tensors every time.  Each
    step of a decoding loop takes another `offset` (default: the plan's).  See
    verify_tree_sample."""

    name = "spec_verify_tree_sample"

    def __init__(self, target_logits, draft_ids, parents=None, cu_draft=None, temperature=1.0, top_k=0, top_p=1.0,
                 seed=0, offset=0, max_draft=None, out=None, workspace=None, stream=None):
        super().__init__(target_logits, draft_ids, parents, cu_draft, max_draft, out, workspace, stream,
                         (C.c_float(temperature), C.c_int32(top_k), C.c_float(top_p), C.c_uint64(seed),
                          C.c_uint32(offset)))

    def __call__(self, offset=None):
        if offset is not None:
            self.args = (*self.args[:8], C.c_uint32(offset), *self.args[9:])
        return super().__call__()


def verify_tree_greedy(target_logits: torch.Tensor, draft_ids: torch.Tensor, parents: Optional[torch.Tensor] = None,
                       cu_draft: Optional[torch.Tensor] = None, max_draft: Optional[int] = None,
                       out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Greedy verify of a tree of guesses on the GPU (spec_verify_tree_greedy).

    target_logits [sum(K_b + 1), V] float32, bfloat16 or float16: row 0 of a
    sequence scores what follows its newest token, row j + 1 what follows guess j;
    draft_ids int32 [sum(K_b)]; parents int32 [sum(K_b)], the row (0 .. j) that
    guess j extends, or None (a chain); cu_draft int32 [batch + 1] or None (uniform
    K); max_draft is read back from the device where it is needed and not given.
    Returns tokens [sum(K_b + 1)], num_accepted [batch] and path [sum(K_b + 1)], the
    accepted rows.
    """
    return TreeGreedyPlan(target_logits, draft_ids, parents, cu_draft, max_draft, out, workspace, stream)()


def verify_tree_sample(target_logits: torch.Tensor, draft_ids: torch.Tensor, parents: Optional[torch.Tensor] = None,
                       cu_draft: Optional[torch.Tensor] = None, temperature: float = 1.0, top_k: int = 0,
                       top_p: float = 1.0, seed: int = 0, offset: int = 0, max_draft: Optional[int] = None,
                       out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Sampling verify of a tree of guesses on the GPU (spec_verify_tree_sample):
    every row draws its own token from the target's filtered softmax, and guesses
    are accepted as far as they equal the draws.  Arguments and outputs as for
    verify_tree_greedy; temperature, top_k, top_p, seed and offset as for
    verify_sample.
    """
    return TreeSamplePlan(target_logits, draft_ids, parents, cu_draft, temperature, top_k, top_p, seed, offset,
                          max_draft, out, workspace, stream)()


class TreeShapeT(C.Structure):
    """sv_tree_shape_t."""
    _fields_ = ([(n, C.c_int32) for n in ("batch", "max_draft", "total_draft", "q_heads", "kv_heads", "head_dim", "pages",
                                          "page_size", "max_pages", "dtype")]
                + [(n, C.c_int64) for n in ("table_stride", "q_row_stride", "q_head_stride", "out_row_stride",
                                            "out_head_stride")]
                + [(n, C.c_void_p) for n in ("cu_draft", "parents", "lengths", "page_table")])


def _pages(t, name, q, shape):
    """The C cache of [pages, page_size, kv_heads, head_dim]."""
    if t.dtype != q.dtype:
        raise TypeError(f"{name} is {t.dtype} but q is {q.dtype}")
    if t.device != q.device:
        raise ValueError(f"{name} is on {t.device} but q is on {q.device}")
    if t.dim() != 4 or tuple(t.shape) != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}; [pages, page_size, kv_heads, head_dim] = {shape} is needed")
    if t.stride(3) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return CacheT(t.data_ptr(), *[t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)])


class TreeAttentionPlan(_DevicePlan):
    """spec_tree_attention with every argument marshalled once: __call__ enqueues
    one call and returns {"out"} and, with return_lse, {"lse"}, the same tensors
    every time.  See tree_attention."""

    name = "spec_tree_attention"

    def __init__(self, q, k, v, page_table=None, lengths=None, parents=None, cu_draft=None, max_draft=None, scale=None,
                 return_lse=False, out=None, workspace=None, stream=None):
        lib = load_library()
        if q.dim() != 3:
            raise ValueError("q must be [rows, q_heads, head_dim]")
        if k.dim() != 4:
            raise ValueError("k must be [pages, page_size, kv_heads, head_dim]")
        rows, q_heads, dim = q.shape
        pages, page_size, kv_heads, _ = k.shape
        if q.numel() == 0 or k.numel() == 0 or q_heads % kv_heads != 0:
            raise ValueError(f"{rows} rows, {q_heads} query heads, {pages} pages of {page_size} positions and {kv_heads} "
                             "key/value heads do not fit together")
        code = _b._dtype_code(q)
        dev, dtype = q.device, q.dtype
        if dev.type != "cuda":
            raise ValueError("q must be on a GPU")
        caches = [_pages(t, n, q, (pages, page_size, kv_heads, dim)) for n, t in (("k", k), ("v", v))]
        # sequences: what tells their number first
        counts = [("cu_draft", cu_draft, -1), ("page_table", page_table, 0), ("lengths", lengths, 0)]
        batch = next((t.shape[0] + extra for _, t, extra in counts if t is not None),
                     rows if parents is None else rows - parents.numel())
        if batch < 1:
            raise ValueError(f"{rows} rows do not fit {batch} sequences")
        kmax, total = _batch(rows, cu_draft, max_draft, batch, stream)
        if page_table is None:
            if pages < batch:
                raise ValueError(f"k holds {pages} sequences; {batch} are needed without a page_table")
            table, max_pages, stride = None, 1, 1
        else:
            table, max_pages, stride = _table(page_table, "page_table", batch, dev)
        cu, ups, used = [None if t is None else _vector(t, n, c, torch.int32, dev) for n, t, c in (
            ("cu_draft", cu_draft, batch + 1), ("parents", parents, total), ("lengths", lengths, batch))]
        with _on(dev, stream):
            if out is None:
                out = {"out": torch.empty((rows, q_heads, dim), dtype=dtype, device=dev)}
            if return_lse and out.get("lse") is None:
                out = {**out, "lse": torch.empty((rows, q_heads), dtype=torch.float32, device=dev)}
        o = out["out"]
        if tuple(o.shape) != (rows, q_heads, dim) or o.dtype != dtype or o.device != dev:
            raise ValueError(f"out['out'] must be {dtype} [{rows}, {q_heads}, {dim}] on {dev}")
        lse = None
        if out.get("lse") is not None:
            lse = _vector(out["lse"], "out['lse']", rows * q_heads, torch.float32, dev)
        shape = TreeShapeT(batch, kmax, total, q_heads, kv_heads, dim, pages, page_size, max_pages, code, stride,
                           *_rows3(q, "q"), *_rows3(o, "out['out']"), cu, ups, used, table)
        scale = dim ** -0.5 if scale is None else float(scale)
        args = (C.byref(shape), C.c_void_p(q.data_ptr()), *[C.byref(c) for c in caches], C.c_float(scale),
                C.c_void_p(o.data_ptr()), lse)
        need = C.c_size_t(0)
        _check(lib.spec_tree_attention(*args, None, C.byref(need), None), "spec_tree_attention(workspace query)")
        with _on(dev, stream):
            self.workspace = _workspace(workspace, need.value, dev)
        self.out, self.shape = out, shape
        self._own(dev, stream, self.workspace, *(t for t in out.values() if t is not None))
        self.have = C.c_size_t(self.workspace.numel())
        self._keep = (q, k, v, page_table, lengths, parents, cu_draft, caches)
        self.args = (*args, C.c_void_p(self.workspace.data_ptr()), C.byref(self.have))
        self.fn, self.fn_profiled = lib.spec_tree_attention, lib.spec_tree_attention_profiled


def tree_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, page_table: Optional[torch.Tensor] = None,
                   lengths: Optional[torch.Tensor] = None, parents: Optional[torch.Tensor] = None,
                   cu_draft: Optional[torch.Tensor] = None, max_draft: Optional[int] = None,
                   scale: Optional[float] = None, return_lse: bool = False, out: Optional[dict] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Attention of every sequence's newest rows over its cache in pages, on the GPU
    (spec_tree_attention).

    q [sum(K_b + 1), q_heads, D], bfloat16 or float16, rows packed as the target
    rows of a verify (one row per sequence at a plain decode step); k and v [pages,
    page_size, kv_heads, D], the newest rows' keys and values written; page_table
    int32 [batch, max_pages] (page_size a multiple of 16), or None: page b is
    sequence b's whole cache; lengths int32 [batch], the positions in use with the
    newest rows (None: all); parents int32 [sum(K_b)], the row (0 .. j) that guess
    j extends, or None (chains); cu_draft int32 [batch + 1] or None (uniform K);
    max_draft is read back from the device, on the call's stream, where it is
    needed and not given.  scale defaults to D ** -0.5.  Returns out [rows, q_heads,
    D] and, with return_lse, lse [rows, q_heads]; `out` may hold both, or out alone.
    """
    return TreeAttentionPlan(q, k, v, page_table, lengths, parents, cu_draft, max_draft, scale, return_lse, out,
                             workspace, stream)()
