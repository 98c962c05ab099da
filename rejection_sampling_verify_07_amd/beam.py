"""ctypes binding of the beam-decoding calls (spec_beam_select and its
companions, include/specverify.h): argument marshalling only, as in binding.py.

A call runs on the device of its tensors, whichever device is current, and on
`stream` (default: that device's current stream); what it allocates itself is
allocated for that stream.  Each call has a plan class that marshals the
arguments once, for tight loops and graph capture.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import binding as _b
from .binding import SpecVerifyError, _check, _dtype_code, _longest, _on, _Plan, load_library


class BeamShapeT(C.Structure):
    """sv_beam_shape_t."""
    _fields_ = [("groups", C.c_int32), ("beams", C.c_int32), ("vocab", C.c_int32), ("num_select", C.c_int32),
                ("dtype", C.c_int32), ("row_stride", C.c_int64)]


class StateShapeT(C.Structure):
    """sv_state_shape_t."""
    _fields_ = [("slabs", C.c_int32), ("groups", C.c_int32), ("beams", C.c_int32), ("heads", C.c_int32),
                ("positions", C.c_int32), ("row_bytes", C.c_int64), ("slab_stride", C.c_int64),
                ("beam_stride", C.c_int64), ("head_stride", C.c_int64), ("position_stride", C.c_int64)]


class CacheT(C.Structure):
    """sv_cache_t."""
    _fields_ = [("data", C.c_void_p), ("batch_stride", C.c_int64), ("position_stride", C.c_int64),
                ("head_stride", C.c_int64)]


class AttentionShapeT(C.Structure):
    """sv_attention_shape_t."""
    _fields_ = ([(n, C.c_int32) for n in ("groups", "batch", "max_group", "max_draft", "total_draft", "q_heads",
                                          "kv_heads", "head_dim", "max_prefix", "max_suffix", "dtype")]
                + [(n, C.c_int64) for n in ("q_row_stride", "q_head_stride", "out_row_stride", "out_head_stride")]
                + [(n, C.c_void_p) for n in ("cu_draft", "cu_groups", "prefix_lengths", "suffix_lengths")])


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
    """A plan that launches on `stream` or, without one, on the stream that is
    current for its tensors' device at each call (so a graph capture on another
    stream than the plan was made on records it), whichever device is current.
    A plan that a graph has captured has to outlive the graph."""

    def _launch(self, fn, name, *lead):
        # (the raw handle: making a torch.cuda.Stream object takes 2 us of a call's 5)
        s = self.stream.cuda_stream if self.stream is not None else torch._C._cuda_getCurrentRawStream(self.dev.index)
        if s not in self._streams:
            self._meet(s)
        st = fn(*lead, *self.args, s)
        if st != _b.SV_OK:
            raise SpecVerifyError(st, name)
        return self.out

    def _own(self, dev, stream, *tensors):
        """The device and stream of the calls, and the tensors that this plan
        allocated for them (on that stream, or the one current now)."""
        self.dev, self.stream, self._mine = dev, stream, tensors
        self._streams = {stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev.index)}

    def _meet(self, s):
        """The plan's tensors are used on a stream that they were not allocated
        on: their memory must not be reused before its work is done.  (A capture
        keeps its plan's tensors itself as long as the graph is replayed: the
        plan has to outlive the graph.)"""
        if not torch.cuda.is_current_stream_capturing():
            for t in self._mine:
                t.record_stream(torch.cuda.ExternalStream(s, device=self.dev))
            self._streams.add(s)

    def __call__(self):
        if self.dev.index == torch._C._cuda_getDevice():
            return self._launch(self.fn, self.name)
        with torch.cuda.device(self.dev):
            return self._launch(self.fn, self.name)

    def profiled(self, events):
        with torch.cuda.device(self.dev):
            return self._launch(self.fn_profiled, self.name + "_profiled", events)


class BeamSelectPlan(_DevicePlan):
    """spec_beam_select with every argument marshalled once.

    Holds references to the tensors it was built from; __call__ enqueues one
    selection on `stream` (default: the stream current at the call) and returns
    the outputs, the same tensors every time.  See beam_select.
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
        with _on(dev, stream):
            self.workspace = _workspace(workspace, need.value, dev)
            if out is None:
                out = {k: torch.empty((groups, num_select), dtype=d, device=dev)
                       for k, d in (("scores", torch.float32), ("tokens", torch.int32), ("parents", torch.int32))}
        outs = [_vector(out[k], f"out[{k!r}]", groups * num_select, d, dev)
                for k, d in (("scores", torch.float32), ("tokens", torch.int32), ("parents", torch.int32))]
        self.out, self.shape = out, shape
        self._own(dev, stream, self.workspace, *out.values())
        self.have = C.c_size_t(self.workspace.numel())
        self._keep = (logits, scores, finished)
        self.args = (*args, *outs, C.c_void_p(self.workspace.data_ptr()), C.byref(self.have))
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
        _on(dev, stream)
        self.out, self.shape = states, shape
        self._own(dev, stream)
        self._keep = (parents, lengths)
        self.args = (C.byref(shape), C.c_void_p(states.data_ptr()),
                     _vector(parents, "parents", batch, torch.int32, dev),
                     None if lengths is None else _vector(lengths, "lengths", batch, torch.int32, dev))
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


def _rows3(t, name):
    """Row and head stride of [rows, heads, dim] (a dimension of one place may report any stride)."""
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    dim = t.shape[2]
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else dim)


def _cache(t, name, count, kv_heads, dim, dtype, dev):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [{'groups' if name.startswith('prefix') else 'batch'}, positions, kv_heads, "
                         "head_dim]")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype} but q is {dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device} but q is on {dev}")
    if t.shape[0] != count or t.shape[2] != kv_heads or t.shape[3] != dim:
        raise ValueError(f"{name} is {tuple(t.shape)}; [{count}, positions, {kv_heads}, {dim}] is needed")
    if t.numel() > 0 and t.stride(3) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    st = [t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)]
    return CacheT(t.data_ptr() or None, *st)


class PrefixAttentionPlan(_DevicePlan):
    """spec_prefix_attention with every argument marshalled once: __call__
    enqueues one call and returns {"out"} and, with return_lse, {"lse"}, the
    same tensors every time.  See prefix_attention."""

    name = "spec_prefix_attention"

    def __init__(self, q, prefix_k, prefix_v, suffix_k, suffix_v, prefix_lengths=None, suffix_lengths=None,
                 cu_draft=None, max_draft=None, cu_groups=None, max_group=None, scale=None, return_lse=False, out=None,
                 workspace=None, stream=None):
        lib = load_library()
        if q.dim() != 3:
            raise ValueError("q must be [rows, q_heads, head_dim]")
        for name, t in (("prefix_k", prefix_k), ("prefix_v", prefix_v), ("suffix_k", suffix_k),
                        ("suffix_v", suffix_v)):
            if t.dim() != 4:
                raise ValueError(f"{name} must be a 4-D tensor [groups or batch, positions, kv_heads, head_dim]")
        rows, q_heads, dim = q.shape
        groups, max_prefix, kv_heads, _ = prefix_k.shape
        batch, max_suffix = suffix_k.shape[:2]
        if batch < 1 or groups < 1 or kv_heads < 1 or q_heads % kv_heads != 0:
            raise ValueError(f"{batch} sequences, {groups} groups, {q_heads} query heads and {kv_heads} key/value heads "
                             "do not fit together")
        if prefix_v.shape[1] != max_prefix or suffix_v.shape[1] != max_suffix:
            raise ValueError("keys and values must hold the same number of positions")
        total = rows - batch
        if total < 0:
            raise ValueError(f"q has {rows} rows; {batch} sequences need one each at least")
        code = _dtype_code(q)
        dev, dtype = q.device, q.dtype
        if dev.type != "cuda":
            raise ValueError("q must be on a GPU")
        caches = [_cache(t, n, c, kv_heads, dim, dtype, dev) for n, t, c in (
            ("prefix_k", prefix_k, groups), ("prefix_v", prefix_v, groups), ("suffix_k", suffix_k, batch),
            ("suffix_v", suffix_v, batch))]
        if cu_draft is None:
            if total % batch != 0:
                raise ValueError("q must have batch * (K + 1) rows; pass cu_draft for ragged K")
            if max_draft is not None and max_draft != total // batch:
                raise ValueError("max_draft does not match the uniform draft length")
            max_draft = total // batch
        if cu_groups is None and batch % groups != 0:
            raise ValueError(f"{batch} sequences do not divide into {groups} groups; pass cu_groups")
        vectors = [None if t is None else _vector(t, n, c, torch.int32, dev) for n, t, c in (
            ("cu_draft", cu_draft, batch + 1), ("cu_groups", cu_groups, groups + 1),
            ("prefix_lengths", prefix_lengths, groups), ("suffix_lengths", suffix_lengths, batch))]
        if max_draft is None:
            max_draft = _longest(cu_draft, stream)
        if cu_groups is not None and max_group is None:
            max_group = _longest(cu_groups, stream)
        lse = None
        with _on(dev, stream):
            if out is None:
                out = {"out": torch.empty((rows, q_heads, dim), dtype=dtype, device=dev)}
            if return_lse and out.get("lse") is None:
                out = {**out, "lse": torch.empty((rows, q_heads), dtype=torch.float32, device=dev)}
        o = out["out"]
        if tuple(o.shape) != (rows, q_heads, dim) or o.dtype != dtype or o.device != dev:
            raise ValueError(f"out['out'] must be {dtype} [{rows}, {q_heads}, {dim}] on {dev}")
        if out.get("lse") is not None:
            lse = _vector(out["lse"], "out['lse']", rows * q_heads, torch.float32, dev)
        shape = AttentionShapeT(groups, batch, int(max_group or 0), int(max_draft), total, q_heads, kv_heads, dim,
                                max_prefix, max_suffix, code, *_rows3(q, "q"), *_rows3(o, "out['out']"), *vectors)
        scale = dim ** -0.5 if scale is None else float(scale)
        args = (C.byref(shape), C.c_void_p(q.data_ptr()), *[C.byref(c) for c in caches], C.c_float(scale),
                C.c_void_p(o.data_ptr()), lse)
        need = C.c_size_t(0)
        _check(lib.spec_prefix_attention(*args, None, C.byref(need), None), "spec_prefix_attention(workspace query)")
        with _on(dev, stream):
            self.workspace = _workspace(workspace, need.value, dev)
        self.out, self.shape = out, shape
        self._own(dev, stream, self.workspace, *(t for t in out.values() if t is not None))
        self.have = C.c_size_t(self.workspace.numel())
        self._keep = (q, prefix_k, prefix_v, suffix_k, suffix_v, prefix_lengths, suffix_lengths, cu_draft, cu_groups,
                      caches)
        self.args = (*args, C.c_void_p(self.workspace.data_ptr()), C.byref(self.have))
        self.fn, self.fn_profiled = lib.spec_prefix_attention, lib.spec_prefix_attention_profiled


def prefix_attention(q: torch.Tensor, prefix_k: torch.Tensor, prefix_v: torch.Tensor, suffix_k: torch.Tensor,
                     suffix_v: torch.Tensor, prefix_lengths: Optional[torch.Tensor] = None,
                     suffix_lengths: Optional[torch.Tensor] = None, cu_draft: Optional[torch.Tensor] = None,
                     max_draft: Optional[int] = None, cu_groups: Optional[torch.Tensor] = None,
                     max_group: Optional[int] = None, scale: Optional[float] = None, return_lse: bool = False,
                     out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Attention over group-shared prefixes and own suffixes on the GPU
    (spec_prefix_attention).

    q [sum(K_b + 1), q_heads, D], bfloat16 or float16, rows packed as the target
    rows of a verify (one row per sequence at a plain decode step); prefix_k and
    prefix_v [groups, positions, kv_heads, D]; suffix_k and suffix_v [batch,
    positions, kv_heads, D], the newest rows' keys and values written; lengths
    int32, the positions in use (None: all).  cu_draft int32 [batch + 1] or None
    (uniform K); cu_groups int32 [groups + 1], the groups' first sequences, or
    None (equal groups).  max_draft and max_group are read back from the device,
    on the call's stream, where they are needed and not given.  scale defaults to D ** -0.5.
    Returns out [rows, q_heads, D] and, with return_lse, lse [rows, q_heads]; `out`
    may hold both, or out alone.
    """
    return PrefixAttentionPlan(q, prefix_k, prefix_v, suffix_k, suffix_v, prefix_lengths, suffix_lengths, cu_draft,
                               max_draft, cu_groups, max_group, scale, return_lse, out, workspace, stream)()
