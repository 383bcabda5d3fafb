"""Python binding of include/ssu_delta.h: the gated delta rule (prompts in
chunks, replayed steps, flushes) beside the selective state update.

Argument marshalling only, as in the package's front end.  A cache or a call
description is checked once, when it is made; it keeps its tensors alive, and
their contents (slots, counts, inputs) may change between calls.  Tensors given
to a call itself (slot_idx, num_fold, states) are not kept: on a `stream` that
is not torch's current one they have to live until the call has run there.
"""
from __future__ import annotations

import ctypes
import dataclasses

from . import (DTYPE_CODES, SSU_BF16, SSU_F32, _check, _lib, _on_device, _packed, _ptr, _slot_pages, _I32, _I64, _P)

SSU_DELTA_MAX_PAIRS = 1 << 21


class SsuDeltaCache(ctypes.Structure):
    _fields_ = [
        ("num_slots", _I32), ("nheads_k", _I32), ("nheads_v", _I32), ("dim_k", _I32), ("dim_v", _I32),
        ("ring_len", _I32), ("state_dtype", ctypes.c_int), ("io_dtype", ctypes.c_int), ("no_qk_norm", _I32),
        ("state", _P), ("state_slot_stride", _I64), ("k_cache", _P), ("k_slot_stride", _I64),
        ("v_cache", _P), ("v_slot_stride", _I64), ("gate_cache", _P), ("gate_slot_stride", _I64),
        ("ring_start", _P), ("status", _P),
    ]


class SsuDeltaStep(ctypes.Structure):
    _fields_ = [
        ("batch", _I32), ("max_seqlen", _I32), ("slot_idx", _P), ("prev_num_accepted", _P), ("cu_seqlens", _P),
        ("q", _P), ("k", _P), ("v", _P), ("q_row_stride", _I64), ("k_row_stride", _I64), ("v_row_stride", _I64),
        ("dt", _P), ("beta", _P), ("A", _P), ("dt_bias", _P), ("scale", ctypes.c_float),
        ("no_dt_softplus", _I32), ("no_beta_sigmoid", _I32), ("out", _P), ("out_dtype", ctypes.c_int),
    ]


class SsuDeltaPrefill(ctypes.Structure):
    _fields_ = [
        ("num_seqs", _I32), ("rows", _I32), ("nheads_k", _I32), ("nheads_v", _I32), ("dim_k", _I32), ("dim_v", _I32),
        ("io_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("cu_seqlens", _P), ("q", _P), ("k", _P), ("v", _P),
        ("q_row_stride", _I64), ("k_row_stride", _I64), ("v_row_stride", _I64),
        ("dt", _P), ("beta", _P), ("A", _P), ("dt_bias", _P), ("scale", ctypes.c_float),
        ("no_dt_softplus", _I32), ("no_beta_sigmoid", _I32), ("no_qk_norm", _I32),
        ("initial_states", _P), ("final_states", _P), ("out", _P), ("workspace", _P),
        ("workspace_bytes", ctypes.c_size_t), ("status", _P),
    ]


_lib.ssu_delta_replay_step.restype = ctypes.c_int
_lib.ssu_delta_replay_step.argtypes = [ctypes.POINTER(SsuDeltaCache), ctypes.POINTER(SsuDeltaStep), _P]
_lib.ssu_delta_flush.restype = ctypes.c_int
_lib.ssu_delta_flush.argtypes = [ctypes.POINTER(SsuDeltaCache), _P, _P, _I32, _P]
for _name in ("ssu_delta_init_state", "ssu_delta_read_state"):
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = [ctypes.POINTER(SsuDeltaCache), _P, _I64, _P, _I32, _P]
_lib.ssu_delta_prefill_workspace_size.restype = ctypes.c_size_t
_lib.ssu_delta_prefill_workspace_size.argtypes = [_I32, _I32, _I32]
_lib.ssu_delta_prefill.restype = ctypes.c_int
_lib.ssu_delta_prefill.argtypes = [ctypes.POINTER(SsuDeltaPrefill), _P]

EXPORTED = ("ssu_delta_replay_step", "ssu_delta_flush", "ssu_delta_init_state", "ssu_delta_read_state",
            "ssu_delta_prefill_workspace_size", "ssu_delta_prefill")


# raw C entry points (descriptor structs in, return code out)

def ssu_delta_replay_step(cache: SsuDeltaCache, step: SsuDeltaStep, stream: int = 0) -> int:
    return _lib.ssu_delta_replay_step(ctypes.byref(cache), ctypes.byref(step), stream)


def ssu_delta_flush(cache: SsuDeltaCache, slot_idx: int, num_fold: int, n: int, stream: int = 0) -> int:
    return _lib.ssu_delta_flush(ctypes.byref(cache), slot_idx, num_fold, n, stream)


def ssu_delta_init_state(cache: SsuDeltaCache, states: int, states_batch_stride: int, slot_idx: int, n: int,
                         stream: int = 0) -> int:
    return _lib.ssu_delta_init_state(ctypes.byref(cache), states, states_batch_stride, slot_idx, n, stream)


def ssu_delta_read_state(cache: SsuDeltaCache, states: int, states_batch_stride: int, slot_idx: int, n: int,
                         stream: int = 0) -> int:
    return _lib.ssu_delta_read_state(ctypes.byref(cache), states, states_batch_stride, slot_idx, n, stream)


def ssu_delta_prefill_workspace_size(rows: int, num_seqs: int, nheads_v: int) -> int:
    return int(_lib.ssu_delta_prefill_workspace_size(rows, num_seqs, nheads_v))


def ssu_delta_prefill(args: SsuDeltaPrefill, stream: int = 0) -> int:
    return _lib.ssu_delta_prefill(ctypes.byref(args), stream)


# torch-tensor front end

def _typed(t, name: str, dtype, shape):
    """A packed device tensor of this type and (where not None) these sizes."""
    import torch
    _packed(t, name)
    want = {"i32": torch.int32, "f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    if t.dtype != want:
        raise ValueError("%s must be %s (got %s)" % (name, want, t.dtype))
    _shape(t, name, shape)


def _shape(t, name: str, shape):
    if t.dim() != len(shape) or any(w is not None and w != h for w, h in zip(shape, t.shape)):
        raise ValueError("%s must be [%s] (got %s)" % (name, ", ".join("n" if w is None else str(w) for w in shape),
                                                       tuple(t.shape)))


def _rows(t, name: str, shape) -> int:
    """A bf16 device tensor [rows, heads, dim] whose rows are each packed; the
    elements between rows."""
    import torch
    _on_device(t, name)
    if t.dtype != torch.bfloat16:
        raise ValueError("%s must be torch.bfloat16 (got %s)" % (name, t.dtype))
    _shape(t, name, shape)
    packed = t.shape[1] * t.shape[2]
    if t.shape[0] == 0:
        return packed
    if not t[0].is_contiguous():
        raise ValueError("%s: each row must be contiguous" % name)
    return t.stride(0) if t.shape[0] > 1 else max(packed, t.stride(0) // 8 * 8)


def _one_device(tensors, device=None):
    """All tensors are on one device (`device`, if given); returns it."""
    for name, t in tensors.items():
        if t is None:
            continue
        device = device or t.device
        if t.device != device:
            raise ValueError("%s is on %s, the other tensors on %s" % (name, t.device, device))
    return device


def _launch(fn, device, stream, *args):
    """fn(*args, stream) on `device`, made the current one where it is not."""
    import torch
    if stream is None:
        handle = torch.cuda.current_stream(device).cuda_stream
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == device.index:
        _check(fn(*args, handle))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, handle))


@dataclasses.dataclass(frozen=True)
class DeltaCache:
    """Device tensors of one gated-delta-rule cache in the ssu_delta_cache
    layout: state, k_cache, v_cache and gate_cache [num_slots, ...] with packed
    slot pages (the pages may be padded), ring_start int32 [num_slots], status
    an optional int32 [1].  Raises ValueError for tensors the kernels could not
    address; the library checks the rest at each call."""
    num_slots: int
    nheads_k: int
    nheads_v: int
    ring_len: int
    state_dtype: str
    state: object
    k_cache: object
    v_cache: object
    gate_cache: object
    ring_start: object
    status: object = None
    dim_k: int = 128
    dim_v: int = 128
    qk_norm: bool = True

    def __post_init__(self):
        n = self.num_slots
        _typed(self.ring_start, "ring_start", "i32", (n,))
        if self.status is not None:
            _typed(self.status, "status", "i32", (None,))
            _packed(self.status, "status", 4)
        pages = {}
        for name in ("state", "k_cache", "v_cache", "gate_cache"):
            t = getattr(self, name)
            pages[name] = _slot_pages(t, name, n)
            pages[name + "_bytes"] = (t[0].numel() if n else 0) * t.element_size()
        size = 4 if self.state_dtype == "f32" else 2
        need = dict(state=self.nheads_v * self.dim_v * self.dim_k * size,
                    k_cache=self.nheads_k * self.ring_len * self.dim_k * 2,
                    v_cache=self.nheads_v * self.ring_len * self.dim_v * 2,
                    gate_cache=self.nheads_v * self.ring_len * 8)
        for name, nbytes in need.items():
            if pages[name + "_bytes"] < nbytes:
                raise ValueError("%s: a slot page holds %d bytes; the layout needs %d" % (name, pages[name + "_bytes"], nbytes))
            if n == 1:  # a single page has no distance to the next
                pages[name] = max(pages[name], (nbytes + 15) // 16 * 16)
        object.__setattr__(self, "device", _one_device(
            {name: getattr(self, name) for name in ("state", "k_cache", "v_cache", "gate_cache", "ring_start", "status")}))
        object.__setattr__(self, "_desc", SsuDeltaCache(
            n, self.nheads_k, self.nheads_v, self.dim_k, self.dim_v, self.ring_len, DTYPE_CODES[self.state_dtype], SSU_BF16,
            0 if self.qk_norm else 1, _ptr(self.state), pages["state"], _ptr(self.k_cache), pages["k_cache"],
            _ptr(self.v_cache), pages["v_cache"], _ptr(self.gate_cache), pages["gate_cache"], _ptr(self.ring_start),
            _ptr(self.status)))

    def desc(self) -> SsuDeltaCache:
        return self._desc


def _out_code(out, shape) -> int:
    import torch
    _packed(out, "out")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out must be torch.bfloat16 or torch.float32 (got %s)" % out.dtype)
    _shape(out, "out", shape)
    return SSU_F32 if out.dtype == torch.float32 else SSU_BF16


def make_delta_step(cache: DeltaCache, max_seqlen, slot_idx, pnat, cu_seqlens, q, k, v, dt, beta, A, dt_bias, out,
                    scale=None, dt_softplus=True, beta_sigmoid=True) -> SsuDeltaStep:
    """The ssu_delta_step descriptor of one step, from device tensors.

    slot_idx, pnat: int32 [batch]; cu_seqlens: int32 [batch + 1] or None (entry
    b then has rows b * max_seqlen ...); q, k: bf16 [rows, nheads_k, dim_k] and
    v: bf16 [rows, nheads_v, dim_v], possibly slices of wider rows; dt, beta:
    f32 [rows, nheads_v]; A, dt_bias: f32 [nheads_v]; out: bf16 or f32 [rows,
    nheads_v, dim_v].  scale: of q, dim_k ** -0.5 where None.  dt_softplus and
    beta_sigmoid False take dt + dt_bias and beta as they are.  With cu_seqlens
    the lengths lie on the device: rows must hold them."""
    b, Hk, Hv, dk, dv = slot_idx.numel(), cache.nheads_k, cache.nheads_v, cache.dim_k, cache.dim_v
    _typed(slot_idx, "slot_idx", "i32", (None,))
    _typed(pnat, "pnat", "i32", (b,))
    if cu_seqlens is not None:
        _typed(cu_seqlens, "cu_seqlens", "i32", (b + 1,))
    rows = q.shape[0]
    if cu_seqlens is None and rows < b * max_seqlen:
        raise ValueError("q has %d rows; %d entries of %d tokens need %d" % (rows, b, max_seqlen, b * max_seqlen))
    strides = (_rows(q, "q", (rows, Hk, dk)), _rows(k, "k", (rows, Hk, dk)), _rows(v, "v", (rows, Hv, dv)))
    for t, name, shape in ((dt, "dt", (rows, Hv)), (beta, "beta", (rows, Hv)), (A, "A", (Hv,)), (dt_bias, "dt_bias", (Hv,))):
        _typed(t, name, "f32", shape)
    code = _out_code(out, (rows, Hv, dv))
    desc = SsuDeltaStep(b, max_seqlen, _ptr(slot_idx), _ptr(pnat), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), *strides,
                        _ptr(dt), _ptr(beta), _ptr(A), _ptr(dt_bias), dk ** -0.5 if scale is None else float(scale),
                        0 if dt_softplus else 1, 0 if beta_sigmoid else 1, _ptr(out), code)
    desc._tensors = dict(slot_idx=slot_idx, pnat=pnat, cu_seqlens=cu_seqlens, q=q, k=k, v=v, dt=dt, beta=beta, A=A,
                         dt_bias=dt_bias, out=out)
    _one_device(desc._tensors, cache.device)
    desc._dims = (Hk, Hv, dk, dv)
    return desc


def delta_replay_step(cache: DeltaCache, step: SsuDeltaStep, stream=None):
    """ssu_delta_replay_step: read out the step's tokens into its `out` and
    append them to the rings; the checkpoint stays."""
    if step._dims != (cache.nheads_k, cache.nheads_v, cache.dim_k, cache.dim_v):
        raise ValueError("the step was made for a cache of other heads or dims")
    _one_device({"slot_idx": step._tensors["slot_idx"]}, cache.device)
    _launch(ssu_delta_replay_step, cache.device, stream, cache._desc, step)


def delta_flush(cache: DeltaCache, slot_idx, num_fold, stream=None):
    """ssu_delta_flush: fold the first num_fold[j] live ring tokens of slot
    slot_idx[j] into its checkpoint and advance ring_start (int32 [n])."""
    n = slot_idx.numel()
    _typed(slot_idx, "slot_idx", "i32", (None,))
    _typed(num_fold, "num_fold", "i32", (n,))
    _one_device({"slot_idx": slot_idx, "num_fold": num_fold}, cache.device)
    _launch(ssu_delta_flush, cache.device, stream, cache._desc, _ptr(slot_idx), _ptr(num_fold), n)


def _states(cache: DeltaCache, states, slot_idx, read: bool) -> int:
    import torch
    n = slot_idx.numel()
    _typed(slot_idx, "slot_idx", "i32", (None,))
    _on_device(states, "states")
    if states.dtype != torch.float32:
        raise ValueError("states must be torch.float32 (got %s)" % states.dtype)
    _shape(states, "states", (n, cache.nheads_v, cache.dim_v, cache.dim_k))
    if n and not states[0].is_contiguous():
        raise ValueError("states: each entry must be contiguous")
    _one_device({"states": states, "slot_idx": slot_idx}, cache.device)
    packed = cache.nheads_v * cache.dim_v * cache.dim_k
    return packed if n <= 1 else states.stride(0)


def delta_init_state(cache: DeltaCache, states, slot_idx, stream=None):
    """ssu_delta_init_state: states f32 [n, nheads_v, dim_v, dim_k] (a prompt's
    final states; an expanded entry is broadcast) into the checkpoints of
    slot_idx, rings cleared."""
    stride = _states(cache, states, slot_idx, False)
    _launch(ssu_delta_init_state, cache.device, stream, cache._desc, _ptr(states), stride, _ptr(slot_idx), slot_idx.numel())


def delta_read_state(cache: DeltaCache, states, slot_idx, stream=None):
    """ssu_delta_read_state: the checkpoints of slot_idx into states (f32 [n,
    nheads_v, dim_v, dim_k])."""
    stride = _states(cache, states, slot_idx, True)
    _launch(ssu_delta_read_state, cache.device, stream, cache._desc, _ptr(states), stride, _ptr(slot_idx), slot_idx.numel())


def delta_prefill_workspace_size(rows: int, num_seqs: int, nheads_v: int) -> int:
    """Bytes of scratch a prefill of `rows` rows in num_seqs sequences needs (0
    for sizes outside the library's limits)."""
    return ssu_delta_prefill_workspace_size(rows, num_seqs, nheads_v)


def make_delta_prefill(cu_seqlens, q, k, v, dt, beta, A, dt_bias, out, initial_states=None, final_states=None,
                       workspace=None, scale=None, dt_softplus=True, beta_sigmoid=True, qk_norm=True,
                       status=None) -> SsuDeltaPrefill:
    """The ssu_delta_prefill_args descriptor, from device tensors.

    cu_seqlens: int32 [num_seqs + 1] (sequence s owns rows cu[s] .. cu[s + 1]);
    q, k: bf16 [rows, nheads_k, dim_k], v: bf16 [rows, nheads_v, dim_v],
    possibly slices of wider rows; dt, beta: f32 [rows, nheads_v]; A, dt_bias:
    f32 [nheads_v]; out: bf16 or f32 [rows, nheads_v, dim_v]; initial_states,
    final_states: f32 [num_seqs, nheads_v, dim_v, dim_k] or None, possibly the
    same; workspace: at least delta_prefill_workspace_size(rows, num_seqs,
    nheads_v) bytes; status: an optional int32 [1]."""
    n, rows = cu_seqlens.numel() - 1, q.shape[0]
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [rows, heads, dim]")
    Hk, dk, Hv, dv = q.shape[1], q.shape[2], v.shape[1], v.shape[2]
    _typed(cu_seqlens, "cu_seqlens", "i32", (None,))
    if n < 0:
        raise ValueError("cu_seqlens must hold num_seqs + 1 values")
    strides = (_rows(q, "q", (rows, Hk, dk)), _rows(k, "k", (rows, Hk, dk)), _rows(v, "v", (rows, Hv, dv)))
    for t, name, shape in ((dt, "dt", (rows, Hv)), (beta, "beta", (rows, Hv)), (A, "A", (Hv,)), (dt_bias, "dt_bias", (Hv,))):
        _typed(t, name, "f32", shape)
    for t, name in ((initial_states, "initial_states"), (final_states, "final_states")):
        if t is not None:
            _typed(t, name, "f32", (n, Hv, dv, dk))
    _packed(workspace, "workspace")
    if status is not None:
        _typed(status, "status", "i32", (None,))
        _packed(status, "status", 4)
    code = _out_code(out, (rows, Hv, dv))
    desc = SsuDeltaPrefill(n, rows, Hk, Hv, dk, dv, SSU_BF16, code, _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), *strides,
                           _ptr(dt), _ptr(beta), _ptr(A), _ptr(dt_bias), dk ** -0.5 if scale is None else float(scale),
                           0 if dt_softplus else 1, 0 if beta_sigmoid else 1, 0 if qk_norm else 1, _ptr(initial_states),
                           _ptr(final_states), _ptr(out), _ptr(workspace),
                           0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status))
    desc._tensors = dict(cu_seqlens=cu_seqlens, q=q, k=k, v=v, dt=dt, beta=beta, A=A, dt_bias=dt_bias, out=out,
                         initial_states=initial_states, final_states=final_states, workspace=workspace, status=status)
    desc._device = _one_device(desc._tensors)
    return desc


def delta_prefill(prefill: SsuDeltaPrefill, stream=None):
    """ssu_delta_prefill: outputs of every row of the sequences into `out`,
    their final states into final_states."""
    _launch(ssu_delta_prefill, prefill._device, stream, prefill)
