"""Python binding of include/ssu_prefill.h: whole prompts under the selective
state update, and the checkpoints of a cache read back as fp32 states.

Argument marshalling only; a description is checked once, when it is made, and
keeps its tensors alive.  Tensors given to a call itself (states, slot_idx) are
not kept: on a `stream` that is not torch's current one they have to live until
the call has run there.
"""
from __future__ import annotations

import ctypes

from . import SSU_BF16, DeviceCache, SsuCache, _lib, _on_device, _packed, _ptr, _I32, _I64, _P
from .delta import _launch, _one_device, _out_code, _rows, _shape, _typed


class SsuPrefill(ctypes.Structure):
    _fields_ = [
        ("num_seqs", _I32), ("rows", _I32), ("nheads", _I32), ("ngroups", _I32), ("headdim", _I32), ("dstate", _I32),
        ("io_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("cu_seqlens", _P), ("x", _P), ("B", _P), ("C", _P), ("z", _P),
        ("x_row_stride", _I64), ("B_row_stride", _I64), ("C_row_stride", _I64), ("z_row_stride", _I64),
        ("dt", _P), ("A", _P), ("D", _P), ("dt_bias", _P), ("no_dt_softplus", _I32),
        ("initial_states", _P), ("final_states", _P), ("out", _P), ("workspace", _P),
        ("workspace_bytes", ctypes.c_size_t), ("status", _P),
    ]


_lib.ssu_prefill_workspace_size.restype = ctypes.c_size_t
_lib.ssu_prefill_workspace_size.argtypes = [_I32, _I32, _I32]
_lib.ssu_prefill.restype = ctypes.c_int
_lib.ssu_prefill.argtypes = [ctypes.POINTER(SsuPrefill), _P]
_lib.ssu_read_state.restype = ctypes.c_int
_lib.ssu_read_state.argtypes = [ctypes.POINTER(SsuCache), _P, _I64, _P, _I32, _I32, _P]

EXPORTED = ("ssu_prefill_workspace_size", "ssu_prefill", "ssu_read_state")


# raw C entry points (descriptor structs in, return code out)

def ssu_prefill_workspace_size(rows: int, num_seqs: int, nheads: int) -> int:
    return int(_lib.ssu_prefill_workspace_size(rows, num_seqs, nheads))


def ssu_prefill(args: SsuPrefill, stream: int = 0) -> int:
    return _lib.ssu_prefill(ctypes.byref(args), stream)


def ssu_read_state(cache: SsuCache, states: int, states_batch_stride: int, slot_idx: int, n: int, recur: int = 0,
                   stream: int = 0) -> int:
    return _lib.ssu_read_state(ctypes.byref(cache), states, states_batch_stride, slot_idx, n, recur, stream)


# torch-tensor front end

def prefill_workspace_size(rows: int, num_seqs: int, nheads: int) -> int:
    """Bytes of scratch a prefill of `rows` rows in num_seqs sequences needs (0
    where it needs none, and for sizes outside the library's limits)."""
    return ssu_prefill_workspace_size(rows, num_seqs, nheads)


def make_prefill(cu_seqlens, x, B, C, dt, A, D, dt_bias, out, z=None, initial_states=None, final_states=None, workspace=None,
                 dt_softplus=True, status=None) -> SsuPrefill:
    """The ssu_prefill_args descriptor, from device tensors.

    cu_seqlens: int32 [num_seqs + 1] (sequence s owns rows cu[s] .. cu[s + 1]);
    x, z (or None): bf16 [rows, H, 64] and B, C: bf16 [rows, G, 128], possibly
    slices of wider rows; dt: f32 [rows, H]; A, D, dt_bias: f32 [H]; out: bf16
    or f32 [rows, H, 64]; initial_states, final_states: f32 [num_seqs, H, 64,
    128] or None, possibly the same; workspace: at least
    prefill_workspace_size(rows, num_seqs, H) bytes (None where that is 0);
    dt_softplus False takes dt + dt_bias as it is; status: an optional int32
    [1]."""
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x, B and C must be [rows, heads or groups, dim]")
    n, (rows, H, P), (G, N) = cu_seqlens.numel() - 1, x.shape, B.shape[1:]
    _typed(cu_seqlens, "cu_seqlens", "i32", (None,))
    if n < 0:
        raise ValueError("cu_seqlens must hold num_seqs + 1 values")
    strides = [_rows(x, "x", (rows, H, P)), _rows(B, "B", (rows, G, N)), _rows(C, "C", (rows, G, N)), 0]
    if z is not None:
        strides[3] = _rows(z, "z", (rows, H, P))
    for t, name, shape in ((dt, "dt", (rows, H)), (A, "A", (H,)), (D, "D", (H,)), (dt_bias, "dt_bias", (H,))):
        _typed(t, name, "f32", shape)
    for t, name in ((initial_states, "initial_states"), (final_states, "final_states")):
        if t is not None:
            _typed(t, name, "f32", (n, H, P, N))
    _packed(workspace, "workspace")
    if status is not None:
        _typed(status, "status", "i32", (None,))
        _packed(status, "status", 4)
    code = _out_code(out, (rows, H, P))
    desc = SsuPrefill(n, rows, H, G, P, N, SSU_BF16, code, _ptr(cu_seqlens), _ptr(x), _ptr(B), _ptr(C), _ptr(z), *strides,
                      _ptr(dt), _ptr(A), _ptr(D), _ptr(dt_bias), 0 if dt_softplus else 1, _ptr(initial_states),
                      _ptr(final_states), _ptr(out), _ptr(workspace),
                      0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status))
    desc._tensors = dict(cu_seqlens=cu_seqlens, x=x, B=B, C=C, z=z, dt=dt, A=A, D=D, dt_bias=dt_bias, out=out,
                         initial_states=initial_states, final_states=final_states, workspace=workspace, status=status)
    desc._device = _one_device(desc._tensors)
    return desc


def prefill(args: SsuPrefill, stream=None):
    """ssu_prefill: outputs of every row of the sequences into `out`, their
    final states (what init_state takes) into final_states."""
    _launch(ssu_prefill, args._device, stream, args)


def read_state(cache: DeviceCache, states, slot_idx, recur=False, stream=None):
    """ssu_read_state: the checkpoints of slot_idx (int32 [n]) into states (f32
    [n, H, 64, 128]); recur: the FP16 recurrence checkpoints instead of the
    ones that steps read.  Ring tokens are not folded in: flush them first."""
    import torch
    n = slot_idx.numel()
    _typed(slot_idx, "slot_idx", "i32", (None,))
    _on_device(states, "states")
    if states.dtype != torch.float32:
        raise ValueError("states must be torch.float32 (got %s)" % states.dtype)
    _shape(states, "states", (n, cache.nheads, cache.headdim, cache.dstate))
    packed = cache.nheads * cache.headdim * cache.dstate
    stride = packed if n <= 1 else states.stride(0)
    if n and not states.is_contiguous() and not states[0].is_contiguous():
        raise ValueError("states: each entry must be contiguous")
    if stride < packed:
        raise ValueError("states: its entries overlap (%d elements apart, of %d)" % (stride, packed))
    device = _one_device({"state": cache.state, "states": states, "slot_idx": slot_idx})
    _launch(ssu_read_state, device, stream, cache.desc(), _ptr(states), stride, _ptr(slot_idx), n, 1 if recur else 0)
