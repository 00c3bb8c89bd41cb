"""Python binding of libw12.so's MX4 calls (include/mx4.h): 4-bit floating
point under a shared scale per 32 values, the products with weights stored
that way, and an expert layer on them.

As w12.py this marshals arguments only: every function hands torch tensors'
device pointers and torch's current HIP stream of the tensors' device to the
C ABI, and raises if the library is missing or a tensor is not on the GPU.
Outputs and workspaces come from torch's allocator on that stream, one per
call, so calls on different streams, and captured graphs, share nothing.

    wq = mx4_quantize(w)                    # [N, K] -> 4.25 bits a value
    y = mx4_gemm(x, wq)                     # x BF16 [M, K], any M
    y = mx4_gemm(mx4_quantize(x), wq)       # both sides in 4 bits
    y = mx4_moe(x, logits, w13q, w2q, 6)    # an expert layer, up to 128 tokens
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import w12
from .w12 import OUT_BF16, OUT_F32, STATUS, W12Error

BLOCK = 32
MAX_T = 128
MAX_E = 1024
MAX_TOP_K = 32

_BF16_TYPES = (torch.bfloat16, torch.int16, torch.uint16)
_u8 = torch.uint8


class MX4Error(W12Error):
    def __init__(self, status: int, what: str):
        self.status = status
        RuntimeError.__init__(self, "%s: %s (%s)" % (what, STATUS.get(status, status),
                                                     mx4_status_string(status)))


_lib = None


def lib() -> ctypes.CDLL:
    """libw12.so with the MX4 calls' signatures set."""
    global _lib
    if _lib is not None:
        return _lib
    L = w12.lib()
    i64, i32, p, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    psz = ctypes.POINTER(sz)
    L.mx4_status_string.argtypes = [i32]
    L.mx4_status_string.restype = ctypes.c_char_p
    for name in ("mx4_codes_bytes", "mx4_scales_bytes"):
        getattr(L, name).argtypes = [i64, i64, i64]
        getattr(L, name).restype = sz
    L.mx4_quantize.argtypes = [p, i32, i64, i64, i64, i64, i64, p, p, p]
    L.mx4_dequantize.argtypes = [p, p, i64, i64, i64, p, i32, i64, i64, p]
    L.mx4_gemm_workspace_bytes.argtypes = [i64, i64, i64, i32, psz]
    L.mx4_gemm.argtypes = [p, i64, i64, p, p, i64, i64, p, i64, i32, p, sz, p]
    L.mx4_gemm_mx4.argtypes = [p, p, i64, p, p, i64, i64, p, i64, i32, p, sz, p]
    L.mx4_moe_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i32, psz]
    L.mx4_moe.argtypes = [p, i64, i64, p, i64, p, p, p, p, i64, i64, i64, i64, i32, p, i64, i32,
                          p, sz, p]
    for name in ("mx4_quantize", "mx4_dequantize", "mx4_gemm_workspace_bytes", "mx4_gemm",
                 "mx4_gemm_mx4", "mx4_moe_workspace_bytes", "mx4_moe"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def mx4_status_string(status: int) -> str:
    return lib().mx4_status_string(int(status)).decode()


def mx4_codes_bytes(B: int, R: int, K: int) -> int:
    return int(lib().mx4_codes_bytes(int(B), int(R), int(K)))


def mx4_scales_bytes(B: int, R: int, K: int) -> int:
    return int(lib().mx4_scales_bytes(int(B), int(R), int(K)))


@functools.lru_cache(maxsize=4096)
def mx4_gemm_workspace_bytes(M: int, N: int, K: int, x_mx4: bool = False) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mx4_gemm_workspace_bytes(int(M), int(N), int(K), int(bool(x_mx4)),
                                          ctypes.byref(n)), "mx4_gemm_workspace_bytes")
    return int(n.value)


@functools.lru_cache(maxsize=4096)
def mx4_moe_workspace_bytes(T: int, H: int, I: int, E: int, top_k: int,
                            out_dtype: torch.dtype = torch.bfloat16) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mx4_moe_workspace_bytes(int(T), int(H), int(I), int(E), int(top_k),
                                         _type_of(out_dtype), ctypes.byref(n)),
           "mx4_moe_workspace_bytes")
    return int(n.value)


@functools.lru_cache(maxsize=4096)
def _sizes(R: int, K: int, batch: int) -> tuple:
    tiles = batch * ((R + 15) // 16)
    return tiles * ((K + 127) // 128) * 1024, tiles * ((K + 511) // 512) * 256


@dataclass
class MX4Tensor:
    """A container of one [R, K] matrix (batch None) or of `batch` of them: one
    flat uint8 tensor that holds the codes (mx4_codes_bytes) and then the
    scales (mx4_scales_bytes) of include/mx4.h's layout."""
    data: torch.Tensor
    R: int
    K: int
    batch: int | None = None

    def __post_init__(self):
        self._code_bytes, self._scale_bytes = _sizes(self.R, self.K, self.batch or 1)

    @property
    def shape(self) -> tuple:
        return (self.R, self.K) if self.batch is None else (self.batch, self.R, self.K)

    @property
    def codes(self) -> torch.Tensor:
        return self.data[:self._code_bytes]

    @property
    def scales(self) -> torch.Tensor:
        return self.data[self._code_bytes:self._code_bytes + self._scale_bytes]

    @property
    def nbytes(self) -> int:
        return self._code_bytes + self._scale_bytes

    def ptrs(self, what: str) -> tuple:
        """(codes, scales) device pointers and the device's index."""
        d = self.data
        dev = d.get_device()
        if dev < 0:
            raise ValueError("%s must be on the GPU" % what)
        if d.dtype is not _u8 or d.numel() < self._code_bytes + self._scale_bytes \
                or not d.is_contiguous():
            raise ValueError("%s: data must be %d contiguous bytes" % (what, self.nbytes))
        p = d.data_ptr()
        return p, p + self._code_bytes, dev


# ---- marshalling helpers ---------------------------------------------------

def _check(status: int, what: str) -> None:
    if status != 0:
        raise MX4Error(status, what)


_TYPES = {torch.float32: OUT_F32, **{t: OUT_BF16 for t in _BF16_TYPES}}


def _type_of(dtype: torch.dtype) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise TypeError("expected float32 or BF16, got %s" % dtype)
    return t


# torch's current stream of a device as the pointer itself (torch.cuda.current_stream
# builds an object around it, which costs a small call more than its launch)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


_current = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device


# Every call launches with its tensors' device current: a function that finds another
# one current calls itself again under it.
def _away(device: int) -> bool:
    return _current() != device


def _same(device: int, *others: int) -> None:
    for o in others:
        if o != device:
            raise ValueError("tensors on devices %d and %d in one call" % (device, o))


def _gpu(t: torch.Tensor, what: str) -> int:
    """The index of the tensor's GPU."""
    device = t.get_device()
    if device < 0:
        raise ValueError("%s must be a GPU tensor" % what)
    return device


def _rows(t: torch.Tensor, what: str) -> tuple:
    """(rows, width, row stride) of a 2-D tensor with contiguous rows (one row:
    its width, as its stride says nothing)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D" % what)
    R, K = shape
    ld, unit = t.stride()
    if unit != 1 and K > 1:
        raise ValueError("%s must have unit column stride" % what)
    return R, K, ld if R > 1 else K


def _batched(t: torch.Tensor, what: str) -> tuple:
    """(batch or None, R, K, row stride, matrix stride) of a 2-D or 3-D tensor."""
    shape = t.shape
    if len(shape) == 2:
        R, K, ld = _rows(t, what)
        return None, R, K, ld, 0
    if len(shape) != 3:
        raise ValueError("%s must be 2-D or 3-D" % what)
    B, R, K = shape
    ldb, ld, unit = t.stride()
    if unit != 1 and K > 1:
        raise ValueError("%s must have unit column stride" % what)
    return B, R, K, ld if R > 1 else K, ldb


# (new_empty on a tensor at hand takes 0.4 us less of the host than torch.empty with
# its device)
def _output(y, M: int, N: int, out_dtype: torch.dtype, device: int, like: torch.Tensor) -> tuple:
    """(y, row stride, type) of a given [M, N] output or a new one beside `like`."""
    if y is None:
        if out_dtype is torch.float32:
            return like.new_empty((M, N), dtype=out_dtype), N, OUT_F32
        if out_dtype is torch.bfloat16:
            return like.new_empty((M, N), dtype=out_dtype), N, OUT_BF16
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    _same(device, _gpu(y, "y"))
    R, K, ld = _rows(y, "y")
    if R != M or K != N:
        raise ValueError("y is %s, this call writes (%d, %d)" % (tuple(y.shape), M, N))
    return y, ld, _type_of(y.dtype)


def _workspace(need: int, given, like: torch.Tensor) -> tuple:
    """(tensor to keep until the launch, pointer, bytes)."""
    if need == 0:
        return None, None, 0
    if given is None:
        given = like.new_empty(need, dtype=_u8)
        return given, given.data_ptr(), need
    if given.device != like.device or not given.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % like.device)
    return given, given.data_ptr(), given.numel() * given.element_size()


# ---- the C ABI, by name ----------------------------------------------------

def empty_mx4(R: int, K: int, batch: int | None = None, device="cuda") -> MX4Tensor:
    """A container of the given shape, contents undefined."""
    t = _container(R, K, batch)
    t.data = torch.empty(t.nbytes, dtype=_u8, device=device)
    return t


def _container(R: int, K: int, batch: int | None) -> MX4Tensor:
    if R < 0 or K < BLOCK or K % BLOCK or (batch is not None and batch < 1):
        raise MX4Error(-2, "container of (%s, %d, %d)" % (batch, R, K))
    return MX4Tensor(None, R, K, batch)


def mx4_quantize(x: torch.Tensor, out: MX4Tensor | None = None) -> MX4Tensor:
    """x [R, K] or [B, R, K] (BF16 or fp32, unit column stride) as MX4."""
    dev = _gpu(x, "x")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx4_quantize(x, out)
    xt = _type_of(x.dtype)
    B, R, K, ld, ldb = _batched(x, "x")
    if out is None:
        out = _container(R, K, B)
        out.data = x.new_empty(out.nbytes, dtype=_u8)
        codes = out.data.data_ptr()
        scales = codes + out._code_bytes
    else:
        if out.shape != tuple(x.shape):
            raise ValueError("out holds %s, x is %s" % (out.shape, tuple(x.shape)))
        codes, scales, out_dev = out.ptrs("out")
        _same(dev, out_dev)
    _check(lib().mx4_quantize(x.data_ptr(), xt, B or 1, R, K, ld, ldb, codes, scales,
                              _raw_stream(dev)), "mx4_quantize")
    return out


def mx4_dequantize(q: MX4Tensor, out_dtype: torch.dtype = torch.bfloat16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """The values a container stands for, [R, K] or [B, R, K]."""
    codes, scales, dev = q.ptrs("q")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx4_dequantize(q, out_dtype, out)
    if out is None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
        out = q.data.new_empty(q.shape, dtype=out_dtype)
        B, R, K = q.batch, q.R, q.K
        ld, ldb = K, R * K
    else:
        _same(dev, _gpu(out, "out"))
        if tuple(out.shape) != q.shape:
            raise ValueError("out is %s, q holds %s" % (tuple(out.shape), q.shape))
        B, R, K, ld, ldb = _batched(out, "out")
    yt = _type_of(out.dtype)
    _check(lib().mx4_dequantize(codes, scales, B or 1, R, K, out.data_ptr(), yt, ld, ldb,
                                _raw_stream(dev)), "mx4_dequantize")
    return out


def mx4_gemm(x, w: MX4Tensor, out_dtype: torch.dtype = torch.float32,
             y: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m, n] = sum_k x[m, k] W[n, k] for a container w of one [N, K]: x BF16
    [M, K] (mx4_gemm) or a container of one [M, K] (mx4_gemm_mx4)."""
    if w.batch is not None:
        raise ValueError("w must hold one matrix")
    wc, wsc, dev = w.ptrs("w")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx4_gemm(x, w, out_dtype, y, workspace)
    N, K = w.R, w.K
    x_mx4 = isinstance(x, MX4Tensor)
    if x_mx4:
        M = x.R
        if x.batch is not None or x.K != K:
            raise ValueError("x %s does not multiply w %s" % (x.shape, w.shape))
        xc, xsc, x_dev = x.ptrs("x")
        a0, a1, a2 = xc, xsc, M
    else:
        x_dev = _gpu(x, "x")
        if x.dtype not in _BF16_TYPES:
            raise TypeError("x must hold BF16 bits (bfloat16/int16/uint16), got %s" % x.dtype)
        M, xk, ldx = _rows(x, "x")
        if xk != K:
            raise ValueError("x %s does not multiply w %s" % (tuple(x.shape), w.shape))
        a0, a1, a2 = x.data_ptr(), M, ldx
    _same(dev, x_dev)
    y, ldy, yt = _output(y, M, N, out_dtype, dev, w.data)
    keep, wsp, wsb = _workspace(mx4_gemm_workspace_bytes(M, N, K, x_mx4), workspace, w.data)
    if x_mx4:
        _check(lib().mx4_gemm_mx4(a0, a1, a2, wc, wsc, N, K, y.data_ptr(), ldy, yt, wsp, wsb,
                                  _raw_stream(dev)), "mx4_gemm_mx4")
    else:
        _check(lib().mx4_gemm(a0, a1, a2, wc, wsc, N, K, y.data_ptr(), ldy, yt, wsp, wsb,
                              _raw_stream(dev)), "mx4_gemm")
    return y


def mx4_moe(x: torch.Tensor, logits: torch.Tensor, w13: MX4Tensor, w2: MX4Tensor, top_k: int,
            renormalize: bool = True, out_dtype: torch.dtype = torch.bfloat16,
            y: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The expert layer of include/mx4.h: x BF16 [T, H], router logits fp32
    [T, E], w13 a container of E matrices [2 I, H] (gate rows, then up rows),
    w2 of E matrices [H, I]; T <= 128."""
    dev, logits_dev = _gpu(x, "x"), _gpu(logits, "logits")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx4_moe(x, logits, w13, w2, top_k, renormalize, out_dtype, y, workspace)
    if x.dtype not in _BF16_TYPES:
        raise TypeError("x must hold BF16 bits (bfloat16/int16/uint16), got %s" % x.dtype)
    if logits.dtype is not torch.float32:
        raise TypeError("logits must be float32, got %s" % logits.dtype)
    T, H, ldx = _rows(x, "x")
    T_logits, E, ldl = _rows(logits, "logits")
    I = w2.K
    if T_logits != T or w13.shape != (E, 2 * I, H) or w2.shape != (E, H, I):
        raise ValueError("x %s, logits %s, w13 %s and w2 %s do not fit together"
                         % (tuple(x.shape), tuple(logits.shape), w13.shape, w2.shape))
    c13, s13, d13 = w13.ptrs("w13")
    c2, s2, d2 = w2.ptrs("w2")
    _same(dev, logits_dev, d13, d2)
    y, ldy, yt = _output(y, T, H, out_dtype, dev, x)
    need = mx4_moe_workspace_bytes(T, H, I, E, int(top_k), y.dtype)
    keep, wsp, wsb = _workspace(need, workspace, x)
    _check(lib().mx4_moe(x.data_ptr(), T, ldx, logits.data_ptr(), ldl, c13, s13, c2, s2, H, I, E,
                         int(top_k), int(bool(renormalize)), y.data_ptr(), ldy, yt, wsp, wsb,
                         _raw_stream(dev)), "mx4_moe")
    return y
