"""Python binding of libw12.so's verification of drafted tokens
(include/draft.h), the end of a verify step of speculative decoding.

As mx4.py this marshals arguments only; outputs and workspaces come from
torch's allocator on the current stream of the tensors' device, one per call.

    logits = w12.w12_gemm(x, head)              # [B * (D + 1), V], fp32
    tokens, accepted = draft_verify(logits.view(B, D + 1, V), drafts, uniforms,
                                    draft_probs=probs, temperature=tau)
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import w12
from .mx4 import _away, _gpu, _raw_stream, _same, _type_of, _workspace
from .w12 import STATUS, W12Error

MAX_D = 1023


class DraftError(W12Error):
    def __init__(self, status: int, what: str):
        self.status = status
        RuntimeError.__init__(self, "%s: %s (%s)" % (what, STATUS.get(status, status),
                                                     draft_status_string(status)))


_lib = None


def lib() -> ctypes.CDLL:
    """libw12.so with the draft calls' signatures set."""
    global _lib
    if _lib is not None:
        return _lib
    L = w12.lib()
    i64, i32, p, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    L.draft_status_string.argtypes = [i32]
    L.draft_status_string.restype = ctypes.c_char_p
    L.draft_workspace_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
    L.draft_workspace_bytes.restype = i32
    L.draft_verify.argtypes = [p, i32, i64, i64, i64, i64, i64, p, i32, p, p, i32, i64, i64, p, p,
                               p, p, p, sz, p]
    L.draft_verify.restype = i32
    _lib = L
    return L


def draft_status_string(status: int) -> str:
    return lib().draft_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise DraftError(status, what)


@functools.lru_cache(maxsize=4096)
def draft_workspace_bytes(B: int, D: int, V: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().draft_workspace_bytes(int(B), int(D), int(V), ctypes.byref(n)),
           "draft_workspace_bytes")
    return int(n.value)


def _words(t: torch.Tensor, what: str) -> tuple:
    """(strides of sequences and of rows) of a 3-D tensor with contiguous words."""
    ldb, ldd, unit = t.stride()
    if unit != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError("%s must have contiguous words" % what)
    return ldb, ldd


_F32 = (torch.float32,)
_I32 = (torch.int32,)
_INTS = (torch.int32, torch.int64)


def _small(t: torch.Tensor, what: str, shape: tuple, dtypes: tuple, dev: int) -> int:
    """The pointer of a contiguous tensor of the given shape and types."""
    if t.get_device() != dev or t.dtype not in dtypes or t.shape != shape \
            or not t.is_contiguous():
        _same(dev, _gpu(t, what))
        if t.dtype not in dtypes:
            raise TypeError("%s must be %s, got %s"
                            % (what, " or ".join(map(str, dtypes)), t.dtype))
        raise ValueError("%s must be contiguous %s, got %s" % (what, shape, tuple(t.shape)))
    return t.data_ptr()


def draft_verify(logits: torch.Tensor, drafts: torch.Tensor, uniforms: torch.Tensor,
                 draft_probs: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                 temperature: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                 accepted: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> tuple:
    """(tokens int32 [B, D + 1], accepted int32 [B]) of include/draft.h's
    draft_verify: logits [B, D + 1, V] BF16 or fp32, drafts [B, D] int32 or int64,
    uniforms fp32 [B, D + 1], draft_probs [B, D, V] BF16 or fp32, lengths int32
    [B], temperature fp32 [B]."""
    dev = _gpu(logits, "logits")
    if _away(dev):
        with torch.cuda.device(dev):
            return draft_verify(logits, drafts, uniforms, draft_probs, lengths, temperature,
                                tokens, accepted, workspace)
    if logits.dim() != 3 or logits.shape[1] < 1:
        raise ValueError("logits must be [B, D + 1, V], got %s" % (tuple(logits.shape),))
    B, rows, V = logits.shape
    D = rows - 1
    ldb, ldd = _words(logits, "logits")
    lt = _type_of(logits.dtype)
    dp = _small(drafts, "drafts", (B, D), _INTS, dev)
    up = _small(uniforms, "uniforms", (B, rows), _F32, dev)
    np_ = None if lengths is None else _small(lengths, "lengths", (B,), _I32, dev)
    tp = None if temperature is None else _small(temperature, "temperature", (B,), _F32, dev)
    qp, qt, pdb, pdd = None, 0, 0, 0
    if draft_probs is not None:
        if draft_probs.get_device() != dev or draft_probs.shape != (B, D, V):
            _same(dev, _gpu(draft_probs, "draft_probs"))
            raise ValueError("draft_probs must be %s, got %s"
                             % ((B, D, V), tuple(draft_probs.shape)))
        qp, qt = draft_probs.data_ptr(), _type_of(draft_probs.dtype)
        pdb, pdd = _words(draft_probs, "draft_probs")
    if tokens is None:
        tokens = logits.new_empty((B, rows), dtype=torch.int32)
        op = tokens.data_ptr()
    else:
        op = _small(tokens, "tokens", (B, rows), _I32, dev)
    if accepted is None:
        accepted = logits.new_empty(B, dtype=torch.int32)
        ap = accepted.data_ptr()
    else:
        ap = _small(accepted, "accepted", (B,), _I32, dev)
    keep, wsp, wsb = _workspace(draft_workspace_bytes(B, D, V), workspace, logits)
    _check(lib().draft_verify(logits.data_ptr(), lt, B, D, V, ldb, ldd, dp,
                              int(drafts.dtype is torch.int64), up, qp, qt, pdb, pdd, np_, tp, op,
                              ap, wsp, wsb, _raw_stream(dev)), "draft_verify")
    return tokens, accepted
