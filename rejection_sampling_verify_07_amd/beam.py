"""ctypes binding of the beam-decoding calls (spec_beam_select and its
companions, include/specverify.h): argument marshalling only, as in binding.py.

A call runs on the device of its tensors, whichever device is current, and on
`stream` (default: that device's current stream); what it allocates itself is
allocated for that stream.  Each call has a plan class that marshals the
arguments once, for tight loops and graph capture.
"""
from __future__ import annotations

import contextlib
import ctypes as C
from typing import Optional

import torch

from . import binding as _b
from .binding import SpecVerifyError, _check, _dtype_code, _Plan, load_library


class BeamShapeT(C.Structure):
    """sv_beam_shape_t."""
    _fields_ = [("groups", C.c_int32), ("beams", C.c_int32), ("vocab", C.c_int32), ("num_select", C.c_int32),
                ("dtype", C.c_int32), ("row_stride", C.c_int64)]


class StateShapeT(C.Structure):
    """sv_state_shape_t."""
    _fields_ = [("slabs", C.c_int32), ("groups", C.c_int32), ("beams", C.c_int32), ("heads", C.c_int32),
                ("positions", C.c_int32), ("row_bytes", C.c_int64), ("slab_stride", C.c_int64),
                ("beam_stride", C.c_int64), ("head_stride", C.c_int64), ("position_stride", C.c_int64)]


def _on(dev, stream):
    """A context in which `dev` is the current device and `stream` (default:
    the device's current one) its current stream, and that stream."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return contextlib.nullcontext(), torch.cuda.current_stream()
        stream = torch.cuda.current_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device} but the tensors are on {dev}")
    return torch.cuda.stream(stream), stream


def _vector(t, name, numel, dtype, dev):
    """A contiguous 1-D view's pointer, after its checks."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} entries; {numel} are needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device} but the call runs on {dev}")
    return C.c_void_p(t.data_ptr())


def _workspace(workspace, need, dev):
    if workspace is not None:
        if workspace.device != dev:
            raise ValueError(f"workspace is on {workspace.device} but the call runs on {dev}")
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        if workspace.numel() >= need:
            return workspace
    return torch.empty(max(need, 1), dtype=torch.uint8, device=dev)


class _DevicePlan(_Plan):
    """A plan that makes its tensors' device current around the launch."""

    def __call__(self):
        if self.dev.index == torch.cuda.current_device():
            return super().__call__()
        with torch.cuda.device(self.dev):
            return super().__call__()

    def profiled(self, events):
        with torch.cuda.device(self.dev):
            return super().profiled(events)


class BeamSelectPlan(_DevicePlan):
    """spec_beam_select with every argument marshalled once.

    Holds references to the tensors it was built from; __call__ enqueues one
    selection on `stream` (default: the current stream at construction) and
    returns the outputs, the same tensors every time.  See beam_select.
    """

    name = "spec_beam_select"

    def __init__(self, logits, scores, beams, num_select=None, temperature=1.0, finished=None, pad_token=0, out=None,
                 workspace=None, stream=None):
        lib = load_library()
        if logits.dim() != 2:
            raise ValueError("logits must be a 2-D tensor [groups * beams, vocab]")
        beams = int(beams)
        rows, vocab = logits.shape
        if beams < 1 or rows < 1 or rows % beams != 0:
            raise ValueError(f"logits has {rows} rows; a multiple of beams = {beams} is needed")
        num_select = beams if num_select is None else int(num_select)
        if num_select < 1:
            raise ValueError("num_select must be at least 1")
        groups = rows // beams
        code = _dtype_code(logits)
        stride = _b._rows(logits, "logits")
        dev = logits.device
        if finished is not None and finished.dtype == torch.bool:
            finished = finished.view(torch.uint8)
        # (a single row may report any stride)
        shape = BeamShapeT(groups, beams, vocab, num_select, code, stride if rows > 1 else max(stride, vocab))
        args = (C.byref(shape), C.c_void_p(logits.data_ptr()), _vector(scores, "scores", rows, torch.float32, dev),
                None if finished is None else _vector(finished, "finished", rows, torch.uint8, dev),
                C.c_float(temperature), C.c_int32(pad_token))
        need = C.c_size_t(0)
        _check(lib.spec_beam_select(*args, None, None, None, None, C.byref(need), None),
               "spec_beam_select(workspace query)")
        ctx, s = _on(dev, stream)
        with ctx:
            self.workspace = _workspace(workspace, need.value, dev)
            if out is None:
                out = {k: torch.empty((groups, num_select), dtype=d, device=dev)
                       for k, d in (("scores", torch.float32), ("tokens", torch.int32), ("parents", torch.int32))}
        outs = [_vector(out[k], f"out[{k!r}]", groups * num_select, d, dev)
                for k, d in (("scores", torch.float32), ("tokens", torch.int32), ("parents", torch.int32))]
        self.out, self.dev, self.shape = out, dev, shape
        self.have = C.c_size_t(self.workspace.numel())
        self._keep = (logits, scores, finished, s)
        self.args = (*args, *outs, C.c_void_p(self.workspace.data_ptr()), C.byref(self.have),
                     C.c_void_p(s.cuda_stream))
        self.fn, self.fn_profiled = lib.spec_beam_select, lib.spec_beam_select_profiled


def beam_select(logits: torch.Tensor, scores: torch.Tensor, beams: int, num_select: Optional[int] = None,
                temperature: float = 1.0, finished: Optional[torch.Tensor] = None, pad_token: int = 0,
                workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None, stream=None) -> dict:
    """Beam search's selection on the GPU (spec_beam_select).

    logits [groups * beams, V] float32, bfloat16 or float16 (row g * beams + w
    is beam w of group g); scores float32 [groups * beams] or [groups, beams],
    the beams' log-probabilities so far; finished (uint8 or bool, same shape):
    ended beams, whose one candidate is pad_token at their own score.
    num_select defaults to `beams`; twice that lets a caller set ended ones
    aside.  Returns scores, tokens and parents [groups, num_select], best first.
    """
    return BeamSelectPlan(logits, scores, beams, num_select, temperature, finished, pad_token, out, workspace,
                          stream)()


class StateReorderPlan(_DevicePlan):
    """spec_state_reorder with every argument marshalled once: __call__
    enqueues one reorder and returns `states`.  See reorder_states."""

    name = "spec_state_reorder"

    def __init__(self, states, parents, beams, lengths=None, stream=None):
        lib = load_library()
        beams = int(beams)
        if states.dim() not in (2, 3, 4, 5):
            raise ValueError("states must be [batch, row], [batch, positions, row], [slabs, batch, positions, row] or "
                             "[slabs, batch, heads, positions, row]")
        if states.device.type != "cuda":
            raise ValueError("states must be on a GPU")
        # every form as [slabs, batch, heads, positions, row]
        v = states
        if v.dim() == 2:
            v = v[None, :, None, None, :]
        elif v.dim() == 3:
            v = v[None, :, None, :, :]
        elif v.dim() == 4:
            v = v[:, :, None, :, :]
        slabs, batch, heads, positions, row = v.shape
        if beams < 1 or batch < 1 or batch % beams != 0:
            raise ValueError(f"states holds {batch} beams; a multiple of beams = {beams} is needed")
        if slabs < 1 or heads < 1:
            raise ValueError("states needs at least one slab and one head")
        if row > 1 and v.stride(4) != 1:
            raise ValueError("states must have unit stride in its last dimension")
        dev = states.device
        es = states.element_size()
        shape = StateShapeT(slabs, batch // beams, beams, heads, positions, row * es,
                            *(v.stride(i) * es for i in range(4)))
        ctx, s = _on(dev, stream)
        self.out, self.dev, self.shape = states, dev, shape
        self._keep = (parents, lengths, s)
        self.args = (C.byref(shape), C.c_void_p(states.data_ptr()),
                     _vector(parents, "parents", batch, torch.int32, dev),
                     None if lengths is None else _vector(lengths, "lengths", batch, torch.int32, dev),
                     C.c_void_p(s.cuda_stream))
        self.fn, self.fn_profiled = lib.spec_state_reorder, lib.spec_state_reorder_profiled


def reorder_states(states: torch.Tensor, parents: torch.Tensor, beams: int, lengths: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Beam states put in the order of their parents, in place, on the GPU
    (spec_state_reorder).

    states: any dtype, [batch, row], [batch, positions, row], [slabs, batch,
    positions, row] or [slabs, batch, heads, positions, row], batch = groups *
    beams, any strides without overlap (last dimension contiguous); parents int32
    [groups * beams] or [groups, beams], as beam_select returns them; lengths
    int32, the positions that each beam holds (as before the reorder).
    Returns `states`.
    """
    return StateReorderPlan(states, parents, beams, lengths, stream)()
