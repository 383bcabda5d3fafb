"""Python binding of include/ssu_logits.h: token histories of the requests in a
cache, and a step's logits as the probabilities that verification takes
(penalties, biases, grammar masks, temperature, softmax).

Argument marshalling only; a description is checked once, when it is made, and
keeps its tensors alive.
"""
from __future__ import annotations

import ctypes
import dataclasses

from . import SSU_BF16, SSU_F16, SSU_F32, _lib, _on_device, _packed, _ptr, _slot_pages, _I32, _I64, _P
from .delta import _launch, _one_device, _shape, _typed

SSU_STATUS_EMPTY_ROW, SSU_STATUS_BAD_BIAS = 64, 128


class SsuHistory(ctypes.Structure):
    _fields_ = [
        ("num_slots", _I32), ("vocab", _I32), ("counts", _P), ("counts_slot_stride", _I64), ("seen", _P),
        ("seen_slot_stride", _I64), ("status", _P),
    ]


class SsuCount(ctypes.Structure):
    _fields_ = [
        ("batch", _I32), ("max_seqlen", _I32), ("rows", _I32), ("slot_idx", _P), ("tokens", _P), ("num_tokens", _P),
        ("cu_seqlens", _P), ("prompt", _I32), ("reset", _I32),
    ]


class SsuLogits(ctypes.Structure):
    _fields_ = [
        ("batch", _I32), ("max_seqlen", _I32), ("rows", _I32), ("vocab", _I32), ("logits_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int), ("logits", _P), ("logits_row_stride", _I64), ("out", _P), ("out_row_stride", _I64),
        ("cu_seqlens", _P), ("slot_idx", _P), ("tokens", _P), ("temperature", _P), ("repetition", _P), ("frequency", _P),
        ("presence", _P), ("bias_offsets", _P), ("bias_tokens", _P), ("bias_values", _P), ("bias_count", _I32), ("mask", _P),
        ("mask_row_stride", _I64), ("no_softmax", _I32), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t), ("status", _P),
    ]


_lib.ssu_history_count.restype = ctypes.c_int
_lib.ssu_history_count.argtypes = [ctypes.POINTER(SsuHistory), ctypes.POINTER(SsuCount), _P]
_lib.ssu_logits_workspace_size.restype = ctypes.c_size_t
_lib.ssu_logits_workspace_size.argtypes = [_I32, _I32, _I32]
_lib.ssu_logits.restype = ctypes.c_int
_lib.ssu_logits.argtypes = [ctypes.POINTER(SsuHistory), ctypes.POINTER(SsuLogits), _P]

EXPORTED = ("ssu_history_count", "ssu_logits_workspace_size", "ssu_logits")


# raw C entry points (descriptor structs in, return code out)

def ssu_history_count(history: SsuHistory, args: SsuCount, stream: int = 0) -> int:
    return _lib.ssu_history_count(ctypes.byref(history), ctypes.byref(args), stream)


def ssu_logits_workspace_size(batch: int, max_seqlen: int, vocab: int) -> int:
    return int(_lib.ssu_logits_workspace_size(batch, max_seqlen, vocab))


def ssu_logits(history, args: SsuLogits, stream: int = 0) -> int:
    return _lib.ssu_logits(None if history is None else ctypes.byref(history), ctypes.byref(args), stream)


# torch-tensor front end

@dataclasses.dataclass(frozen=True)
class TokenHistory:
    """Device tensors of the token histories of a cache's slots, in the layout
    of ssu_history: counts int32 [num_slots, vocab], seen int32 [num_slots,
    ceil(vocab / 32)] (rows may be padded), status an optional int32 [1].  A slot's
    page begins with a count whose reset is set."""
    num_slots: int
    vocab: int
    counts: object
    seen: object
    status: object = None

    def __post_init__(self):
        import torch
        n, strides = self.num_slots, []
        for name, words in (("counts", self.vocab), ("seen", (self.vocab + 31) // 32)):
            t = getattr(self, name)
            _on_device(t, name)
            if t.dtype != torch.int32:
                raise ValueError("%s must be torch.int32 (got %s)" % (name, t.dtype))
            _shape(t, name, (n, words))
            stride = _slot_pages(t, name, n) if n else 4 * words
            strides.append(stride if n > 1 else max(stride, 4 * words))
        if self.status is not None:
            _typed(self.status, "status", "i32", (None,))
            _packed(self.status, "status", 4)
        object.__setattr__(self, "device", _one_device(dict(counts=self.counts, seen=self.seen, status=self.status)))
        object.__setattr__(self, "_desc", SsuHistory(n, self.vocab, _ptr(self.counts), strides[0], _ptr(self.seen), strides[1],
                                                     _ptr(self.status)))

    def desc(self) -> SsuHistory:
        return self._desc


def make_count(history: TokenHistory, slot_idx, tokens, num_tokens=None, cu_seqlens=None, prompt=False, reset=False) -> SsuCount:
    """The ssu_count_args descriptor, from device tensors.

    slot_idx: int32 [batch]; tokens: int32 [batch, max_seqlen] with num_tokens
    int32 [batch] of them (None: all) as verify leaves out_tokens and
    num_accepted, or int32 [rows] with cu_seqlens int32 [batch + 1].  prompt:
    they are the prompt's tokens, else generated ones; reset: the slots'
    histories begin here."""
    b = slot_idx.numel()
    _typed(slot_idx, "slot_idx", "i32", (None,))
    if cu_seqlens is not None:
        if num_tokens is not None:
            raise ValueError("cu_seqlens and num_tokens exclude each other")
        _typed(cu_seqlens, "cu_seqlens", "i32", (b + 1,))
        _typed(tokens, "tokens", "i32", (None,))
        T = 1
    else:
        _typed(tokens, "tokens", "i32", (b, None))
        T = tokens.shape[1]
        if num_tokens is not None:
            _typed(num_tokens, "num_tokens", "i32", (b,))
    desc = SsuCount(b, T, tokens.numel(), _ptr(slot_idx), _ptr(tokens), _ptr(num_tokens), _ptr(cu_seqlens), 1 if prompt else 0,
                    1 if reset else 0)
    desc._tensors = dict(slot_idx=slot_idx, tokens=tokens, num_tokens=num_tokens, cu_seqlens=cu_seqlens)
    _one_device(desc._tensors, history.device)
    desc._history = history
    return desc


def count(args: SsuCount, stream=None):
    """ssu_history_count: the tokens into the history that the description was
    made for."""
    _launch(ssu_history_count, args._history.device, stream, args._history._desc, args)


def logits_workspace_size(batch: int, max_seqlen: int, vocab: int) -> int:
    """Bytes of scratch that the logits of batch entries of up to max_seqlen
    rows need (0 for sizes outside the library's limits)."""
    return ssu_logits_workspace_size(batch, max_seqlen, vocab)


def _values(t, name: str, rows: int, vocab: int):
    """(dtype code, elements between rows) of a device tensor of values."""
    import torch
    _on_device(t, name)
    codes = {torch.float32: SSU_F32, torch.bfloat16: SSU_BF16, torch.float16: SSU_F16}
    if t.dtype not in codes:
        raise ValueError("%s must be float32, bfloat16 or float16 (got %s)" % (name, t.dtype))
    _shape(t, name, (rows, vocab))
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError("%s: each row must be contiguous" % name)
    if rows > 1 and t.stride(0) < vocab:
        raise ValueError("%s: its rows overlap (%d elements apart, of %d)" % (name, t.stride(0), vocab))
    return codes[t.dtype], t.stride(0) if rows > 1 else vocab


def make_logits(logits, out, batch, max_seqlen, cu_seqlens=None, history=None, slot_idx=None, tokens=None, temperature=None,
                repetition=None, frequency=None, presence=None, bias_offsets=None, bias_tokens=None, bias_values=None, mask=None,
                softmax=True, workspace=None, status=None) -> SsuLogits:
    """The ssu_logits_args descriptor, from device tensors.

    logits, out (possibly the same): f32, bf16 or f16 [rows, vocab]; cu_seqlens:
    int32 [batch + 1], or None where every entry has max_seqlen rows; history (a
    TokenHistory) with slot_idx int32 [batch] and tokens int32 [rows] (what the
    step was fed; None: no drafts are counted); temperature, repetition,
    frequency, presence: f32 [batch] or None; bias_offsets int32 [batch + 1],
    bias_tokens int32 [n], bias_values f32 [n]; mask: int32 [rows, ceil(vocab /
    32)], a bit for each token that may be taken (an expanded row serves all);
    softmax False: out gets x / temperature instead of probabilities;
    workspace: at least logits_workspace_size(batch, max_seqlen, vocab) bytes
    (none without softmax)."""
    import torch
    if bias_offsets is not None and (bias_tokens is None or bias_values is None):
        raise ValueError("bias_offsets needs bias_tokens and bias_values")
    _shape(logits, "logits", (None, None))
    rows, vocab = logits.shape
    it, in_stride = _values(logits, "logits", rows, vocab)
    ot, out_stride = _values(out, "out", rows, vocab)
    if cu_seqlens is not None:
        _typed(cu_seqlens, "cu_seqlens", "i32", (batch + 1,))
    elif rows < batch * max_seqlen:
        raise ValueError("logits has %d rows; %d entries of %d tokens need %d" % (rows, batch, max_seqlen, batch * max_seqlen))
    if history is not None:
        if slot_idx is None:
            raise ValueError("a history needs slot_idx")
        _typed(slot_idx, "slot_idx", "i32", (batch,))
    if tokens is not None:
        _typed(tokens, "tokens", "i32", (rows,))
    for t, name in ((temperature, "temperature"), (repetition, "repetition"), (frequency, "frequency"), (presence, "presence")):
        if t is not None:
            _typed(t, name, "f32", (batch,))
    biases = 0
    if bias_offsets is not None:
        _typed(bias_offsets, "bias_offsets", "i32", (batch + 1,))
        _typed(bias_tokens, "bias_tokens", "i32", (None,))
        biases = bias_tokens.numel()
        _typed(bias_values, "bias_values", "f32", (biases,))
    mask_stride = 0
    if mask is not None:
        _on_device(mask, "mask")
        words = (vocab + 31) // 32
        if mask.dtype != torch.int32:
            raise ValueError("mask must be torch.int32 (got %s)" % mask.dtype)
        _shape(mask, "mask", (rows, words))
        if words > 1 and mask.stride(1) != 1:
            raise ValueError("mask: each row must be contiguous")
        mask_stride = mask.stride(0) if rows > 1 else words
    _packed(workspace, "workspace")
    if status is not None:
        _typed(status, "status", "i32", (None,))
        _packed(status, "status", 4)
    desc = SsuLogits(batch, max_seqlen, rows, vocab, it, ot, _ptr(logits), in_stride, _ptr(out), out_stride, _ptr(cu_seqlens),
                     _ptr(slot_idx), _ptr(tokens), _ptr(temperature), _ptr(repetition), _ptr(frequency), _ptr(presence),
                     _ptr(bias_offsets), _ptr(bias_tokens), _ptr(bias_values), biases, _ptr(mask), mask_stride,
                     0 if softmax else 1, _ptr(workspace),
                     0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status))
    desc._tensors = dict(logits=logits, out=out, cu_seqlens=cu_seqlens, slot_idx=slot_idx, tokens=tokens, temperature=temperature,
                         repetition=repetition, frequency=frequency, presence=presence, bias_offsets=bias_offsets,
                         bias_tokens=bias_tokens, bias_values=bias_values, mask=mask, workspace=workspace, status=status)
    desc._device = _one_device(desc._tensors, None if history is None else history.device)
    desc._history = history
    return desc


def logits(args: SsuLogits, stream=None):
    """ssu_logits: probabilities (without softmax: processed logits) of every
    row of the entries into `out`."""
    _launch(ssu_logits, args._device, stream, None if args._history is None else args._history._desc, args)
