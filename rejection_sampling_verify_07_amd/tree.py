"""ctypes binding of the calls on trees of guesses (spec_verify_tree_greedy,
spec_verify_tree_sample; include/specverify.h): argument marshalling only.
Streams, devices and plans are as in beam.py.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import binding as _b
from .beam import _DevicePlan, _vector, _workspace
from .binding import _check, _on, load_library


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
