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
        tiles = (self.batch or 1) * ((self.R + 15) // 16)
        self._code_bytes = tiles * ((self.K + 127) // 128) * 1024
        self._scale_bytes = tiles * ((self.K + 511) // 512) * 256

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


def _call(device: int, fn, *args) -> None:
    """fn(*args, stream) on torch's current stream of `device`, which is made
    current for the launch."""
    if _current() == device:
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status != 0:
        raise MX4Error(status, fn.__name__)


def _same(device: int, *others: int) -> None:
    for o in others:
        if o != device:
            raise ValueError("tensors on devices %d and %d in one call" % (device, o))


def _gpu(t: torch.Tensor, what: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % what)
    return t


def _rows(t: torch.Tensor, what: str) -> int:
    """Row stride of a 2-D tensor with contiguous rows (its width if it has
    one row: such a stride says nothing)."""
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % what)
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError("%s must have unit column stride" % what)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _batched(t: torch.Tensor, what: str) -> tuple:
    """(batch or None, R, K, row stride, matrix stride) of a 2-D or 3-D tensor."""
    if t.dim() not in (2, 3):
        raise ValueError("%s must be 2-D or 3-D" % what)
    R, K = t.shape[-2:]
    if t.stride(-1) != 1 and K > 1:
        raise ValueError("%s must have unit column stride" % what)
    ld = t.stride(-2) if R > 1 else K
    if t.dim() == 2:
        return None, R, K, ld, 0
    return t.shape[0], R, K, ld, t.stride(0)


def _output(y, M: int, N: int, out_dtype: torch.dtype, device) -> tuple:
    """(y, row stride, type) of a given or new [M, N] output."""
    if y is None:
        if out_dtype is torch.float32:
            return torch.empty((M, N), dtype=out_dtype, device=device), N, OUT_F32
        if out_dtype is torch.bfloat16:
            return torch.empty((M, N), dtype=out_dtype, device=device), N, OUT_BF16
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    ld = _rows(_gpu(y, "y"), "y")
    if tuple(y.shape) != (M, N):
        raise ValueError("y is %s, this call writes (%d, %d)" % (tuple(y.shape), M, N))
    return y, ld, _type_of(y.dtype)


def _workspace(need: int, given, device) -> tuple:
    """(tensor to keep until the launch, pointer, bytes)."""
    if need == 0:
        return None, None, 0
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=device)
    elif given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % device)
    return given, given.data_ptr(), given.numel() * given.element_size()


# ---- the C ABI, by name ----------------------------------------------------

def empty_mx4(R: int, K: int, batch: int | None = None, device="cuda") -> MX4Tensor:
    """A container of the given shape, contents undefined."""
    if R < 0 or K < BLOCK or K % BLOCK or (batch is not None and batch < 1):
        raise MX4Error(-2, "empty_mx4(%s, %d, %d)" % (batch, R, K))
    t = MX4Tensor(None, R, K, batch)
    t.data = torch.empty(t._code_bytes + t._scale_bytes, dtype=_u8, device=device)
    return t


def mx4_quantize(x: torch.Tensor, out: MX4Tensor | None = None) -> MX4Tensor:
    """x [R, K] or [B, R, K] (BF16 or fp32, unit column stride) as MX4."""
    xt = _type_of(_gpu(x, "x").dtype)
    B, R, K, ld, ldb = _batched(x, "x")
    if out is None:
        out = empty_mx4(R, K, B, x.device)
    elif out.shape != tuple(x.shape):
        raise ValueError("out holds %s, x is %s" % (out.shape, tuple(x.shape)))
    codes, scales, dev = out.ptrs("out")
    _same(dev, x.get_device())
    _call(dev, lib().mx4_quantize, x.data_ptr(), xt, B or 1, R, K, ld, ldb, codes, scales)
    return out


def mx4_dequantize(q: MX4Tensor, out_dtype: torch.dtype = torch.bfloat16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """The values a container stands for, [R, K] or [B, R, K]."""
    codes, scales, dev = q.ptrs("q")
    if out is None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
        out = torch.empty(q.shape, dtype=out_dtype, device=q.data.device)
    elif tuple(out.shape) != q.shape:
        raise ValueError("out is %s, q holds %s" % (tuple(out.shape), q.shape))
    yt = _type_of(_gpu(out, "out").dtype)
    B, R, K, ld, ldb = _batched(out, "out")
    _same(dev, out.get_device())
    _call(dev, lib().mx4_dequantize, codes, scales, B or 1, R, K, out.data_ptr(), yt, ld, ldb)
    return out


def mx4_gemm(x, w: MX4Tensor, out_dtype: torch.dtype = torch.float32,
             y: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m, n] = sum_k x[m, k] W[n, k] for a container w of one [N, K]: x BF16
    [M, K] (mx4_gemm) or a container of one [M, K] (mx4_gemm_mx4)."""
    if w.batch is not None:
        raise ValueError("w must hold one matrix")
    wc, wsc, dev = w.ptrs("w")
    N, K = w.R, w.K
    device = w.data.device
    x_mx4 = isinstance(x, MX4Tensor)
    if x_mx4:
        M = x.R
        if x.batch is not None or x.K != K:
            raise ValueError("x %s does not multiply w %s" % (x.shape, w.shape))
        xc, xsc, x_dev = x.ptrs("x")
        a0, a1, a2 = xc, xsc, M
    else:
        if _gpu(x, "x").dtype not in _BF16_TYPES:
            raise TypeError("x must hold BF16 bits (bfloat16/int16/uint16), got %s" % x.dtype)
        ldx = _rows(x, "x")
        M = x.shape[0]
        if x.shape[1] != K:
            raise ValueError("x %s does not multiply w %s" % (tuple(x.shape), w.shape))
        x_dev = x.get_device()
        a0, a1, a2 = x.data_ptr(), M, ldx
    y, ldy, yt = _output(y, M, N, out_dtype, device)
    _same(dev, x_dev, y.get_device())
    keep, wsp, wsb = _workspace(mx4_gemm_workspace_bytes(M, N, K, x_mx4), workspace, device)
    L = lib()
    _call(dev, L.mx4_gemm_mx4 if x_mx4 else L.mx4_gemm, a0, a1, a2, wc, wsc, N, K, y.data_ptr(),
          ldy, yt, wsp, wsb)
    return y


def mx4_moe(x: torch.Tensor, logits: torch.Tensor, w13: MX4Tensor, w2: MX4Tensor, top_k: int,
            renormalize: bool = True, out_dtype: torch.dtype = torch.bfloat16,
            y: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The expert layer of include/mx4.h: x BF16 [T, H], router logits fp32
    [T, E], w13 a container of E matrices [2 I, H] (gate rows, then up rows),
    w2 of E matrices [H, I]; T <= 128."""
    if _gpu(x, "x").dtype not in _BF16_TYPES:
        raise TypeError("x must hold BF16 bits (bfloat16/int16/uint16), got %s" % x.dtype)
    if _gpu(logits, "logits").dtype is not torch.float32:
        raise TypeError("logits must be float32, got %s" % logits.dtype)
    ldx, ldl = _rows(x, "x"), _rows(logits, "logits")
    (T, H), E = x.shape, logits.shape[1]
    I = w2.K
    if logits.shape[0] != T or w13.shape != (E, 2 * I, H) or w2.shape != (E, H, I):
        raise ValueError("x %s, logits %s, w13 %s and w2 %s do not fit together"
                         % (tuple(x.shape), tuple(logits.shape), w13.shape, w2.shape))
    c13, s13, d13 = w13.ptrs("w13")
    c2, s2, d2 = w2.ptrs("w2")
    dev, device = x.get_device(), x.device
    y, ldy, yt = _output(y, T, H, out_dtype, device)
    _same(dev, logits.get_device(), d13, d2, y.get_device())
    need = mx4_moe_workspace_bytes(T, H, I, E, int(top_k), y.dtype)
    keep, wsp, wsb = _workspace(need, workspace, device)
    _call(dev, lib().mx4_moe, x.data_ptr(), T, ldx, logits.data_ptr(), ldl, c13, s13, c2, s2, H, I,
          E, int(top_k), int(bool(renormalize)), y.data_ptr(), ldy, yt, wsp, wsb)
    return y
