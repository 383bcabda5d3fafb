"""Python binding of include/ssu_verify.h: which drafted tokens the target
accepts, the token drawn after them, and the ring bookkeeping of the next step.

Argument marshalling only; a description is checked once, when it is made, and
keeps its tensors alive.
"""
from __future__ import annotations

import ctypes

from . import SSU_BF16, SSU_F16, SSU_F32, _lib, _on_device, _packed, _ptr, _I32, _I64, _P
from .delta import _launch, _one_device, _shape, _typed

SSU_STATUS_BAD_TOKEN, SSU_STATUS_BAD_PROBS = 16, 32


class SsuVerify(ctypes.Structure):
    _fields_ = [
        ("batch", _I32), ("max_seqlen", _I32), ("vocab", _I32), ("ring_len", _I32), ("reserve", _I32), ("probs_dtype", ctypes.c_int),
        ("cu_seqlens", _P), ("tokens", _P), ("target_probs", _P), ("target_row_stride", _I64), ("draft_probs", _P),
        ("draft_row_stride", _I64), ("u", _P), ("u_final", _P), ("out_tokens", _P), ("num_accepted", _P),
        ("live", _P), ("fold", _P), ("next_live", _P), ("next_fold", _P), ("next_left", _P), ("workspace", _P),
        ("workspace_bytes", ctypes.c_size_t), ("status", _P),
    ]


_lib.ssu_verify_workspace_size.restype = ctypes.c_size_t
_lib.ssu_verify_workspace_size.argtypes = [_I32, _I32]
_lib.ssu_verify.restype = ctypes.c_int
_lib.ssu_verify.argtypes = [ctypes.POINTER(SsuVerify), _P]

EXPORTED = ("ssu_verify_workspace_size", "ssu_verify")


def ssu_verify_workspace_size(batch: int, vocab: int) -> int:
    return int(_lib.ssu_verify_workspace_size(batch, vocab))


def ssu_verify(args: SsuVerify, stream: int = 0) -> int:
    return _lib.ssu_verify(ctypes.byref(args), stream)


def verify_workspace_size(batch: int, vocab: int) -> int:
    """Bytes of scratch a verification needs (0 for sizes outside the
    library's limits)."""
    return ssu_verify_workspace_size(batch, vocab)


def _probs(t, name: str, rows: int, vocab: int) -> int:
    import torch
    _on_device(t, name)
    if t.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError("%s must be float32, bfloat16 or float16 (got %s)" % (name, t.dtype))
    _shape(t, name, (rows, vocab))
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError("%s: each row must be contiguous" % name)
    if rows > 1 and t.stride(0) < vocab:
        raise ValueError("%s: its rows overlap (%d elements apart, of %d)" % (name, t.stride(0), vocab))
    return t.stride(0) if rows > 1 else vocab


def make_verify(tokens, target_probs, draft_probs, u, u_final, out_tokens, num_accepted, workspace, cu_seqlens=None,
                live=None, fold=None, ring_len=0, reserve=0, next_live=None, next_fold=None, next_left=None, status=None) -> SsuVerify:
    """The ssu_verify_args descriptor, from device tensors.

    tokens: int32 [rows], what the step was fed; target_probs, draft_probs (or
    None): f32, bf16 or f16 [rows, vocab]; u: f32 [rows]; u_final: f32 [batch];
    out_tokens: int32 [batch, max_seqlen]; num_accepted: int32 [batch];
    cu_seqlens: int32 [batch + 1], or None where every entry has max_seqlen
    rows; live, fold, next_live, next_fold, next_left: int32 [batch] or None;
    reserve: the tokens next_fold keeps room for (0: max_seqlen; 2 max_seqlen
    towards a fused step);
    workspace: at least verify_workspace_size(batch, vocab) bytes."""
    import torch
    _shape(out_tokens, "out_tokens", (None, None))
    b, T = out_tokens.shape
    _shape(target_probs, "target_probs", (None, None))
    rows, vocab = target_probs.shape
    for t, name, dtype, shape in ((tokens, "tokens", "i32", (rows,)), (u, "u", "f32", (rows,)), (u_final, "u_final", "f32", (b,)),
                                  (out_tokens, "out_tokens", "i32", (b, T)), (num_accepted, "num_accepted", "i32", (b,))):
        _typed(t, name, dtype, shape)
    if cu_seqlens is not None:
        _typed(cu_seqlens, "cu_seqlens", "i32", (b + 1,))
    elif rows < b * T:
        raise ValueError("target_probs has %d rows; %d entries of %d tokens need %d" % (rows, b, T, b * T))
    for t, name in ((live, "live"), (fold, "fold"), (next_live, "next_live"), (next_fold, "next_fold"), (next_left, "next_left")):
        if t is not None:
            _typed(t, name, "i32", (b,))
    strides = [_probs(target_probs, "target_probs", rows, vocab), 0]
    if draft_probs is not None:
        strides[1] = _probs(draft_probs, "draft_probs", rows, vocab)
        if draft_probs.dtype != target_probs.dtype:
            raise ValueError("draft_probs must be %s like target_probs (got %s)" % (target_probs.dtype, draft_probs.dtype))
    _packed(workspace, "workspace")
    if status is not None:
        _typed(status, "status", "i32", (None,))
        _packed(status, "status", 4)
    code = {torch.float32: SSU_F32, torch.bfloat16: SSU_BF16, torch.float16: SSU_F16}[target_probs.dtype]
    desc = SsuVerify(b, T, vocab, ring_len, reserve, code, _ptr(cu_seqlens), _ptr(tokens), _ptr(target_probs), strides[0],
                     _ptr(draft_probs), strides[1], _ptr(u), _ptr(u_final), _ptr(out_tokens), _ptr(num_accepted), _ptr(live),
                     _ptr(fold), _ptr(next_live), _ptr(next_fold), _ptr(next_left), _ptr(workspace),
                     0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status))
    desc._tensors = dict(tokens=tokens, target_probs=target_probs, draft_probs=draft_probs, u=u, u_final=u_final,
                         out_tokens=out_tokens, num_accepted=num_accepted, cu_seqlens=cu_seqlens, live=live, fold=fold,
                         next_live=next_live, next_fold=next_fold, next_left=next_left, workspace=workspace, status=status)
    desc._device = _one_device(desc._tensors)
    return desc


def verify(args: SsuVerify, stream=None):
    """ssu_verify: accepted drafts and the drawn token into out_tokens, their
    number into num_accepted, the next step's ring counts into next_*."""
    _launch(ssu_verify, args._device, stream, args)
