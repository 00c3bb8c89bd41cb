"""Python binding of libw12.so's MX8 calls (include/mx8.h): activations in 8-bit
floating point under a shared scale per 32 values, the residual addition and
norm that writes them, and their product with MX4 weights.  The bytes are
E4M3's; by default values are multiples of 1/4 of their block's unit, with
fine=True they take all of E4M3's steps (include/mx8.h says what either loses).

As mx4.py this marshals arguments only; outputs and workspaces come from
torch's allocator on the current stream of the tensors' device, one per call.

    y, stream = mx8_rms_norm(x, weight, residual=stream)    # MX8 for mx8_gemm
    y = mx8_gemm(y, wq)                                     # wq from mx4_quantize
    y, stream = mx8_rms_norm(x, weight, residual=stream, out_dtype=torch.bfloat16)
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import w12
from .mx4 import (MX4Tensor, _away, _gpu, _output, _raw_stream, _rows, _same, _type_of,
                  _workspace)
from .w12 import STATUS, W12Error

BLOCK = 32
MAX_NORM_K = 32768
OUT_MX8 = 2
FINE_STEPS = 16
VALUES = torch.float8_e4m3fn        # as an output type: a whole MX8Tensor

_u8 = torch.uint8


class MX8Error(W12Error):
    def __init__(self, status: int, what: str):
        self.status = status
        RuntimeError.__init__(self, "%s: %s (%s)" % (what, STATUS.get(status, status),
                                                     mx8_status_string(status)))


_lib = None


def lib() -> ctypes.CDLL:
    """libw12.so with the MX8 calls' signatures set."""
    global _lib
    if _lib is not None:
        return _lib
    L = w12.lib()
    i64, i32, p, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    L.mx8_status_string.argtypes = [i32]
    L.mx8_status_string.restype = ctypes.c_char_p
    L.mx8_scale_row_bytes.argtypes = [i64]
    L.mx8_scale_row_bytes.restype = sz
    L.mx8_quantize.argtypes = [p, i32, i64, i64, i64, p, i64, p, i64, p]
    L.mx8_dequantize.argtypes = [p, i64, p, i64, i64, i64, p, i32, i64, p]
    L.mx8_rms_norm.argtypes = [p, i32, i64, p, p, i32, i64, i64, p, i32, ctypes.c_float, i64, i64,
                               p, i32, i64, p, i64, p]
    L.mx8_gemm_workspace_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
    L.mx8_gemm.argtypes = [p, i64, p, i64, i64, p, p, i64, i64, p, i64, i32, p, sz, p]
    L.mx8_gemm_plan.argtypes = [i64, i64, i64, ctypes.POINTER(ctypes.c_int)]
    L.mx8_gemm_plan.restype = ctypes.c_char_p
    for name in ("mx8_quantize", "mx8_dequantize", "mx8_rms_norm", "mx8_gemm_workspace_bytes",
                 "mx8_gemm"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def mx8_status_string(status: int) -> str:
    return lib().mx8_status_string(int(status)).decode()


def mx8_scale_row_bytes(K: int) -> int:
    return int(lib().mx8_scale_row_bytes(int(K)))


@functools.lru_cache(maxsize=4096)
def mx8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mx8_gemm_workspace_bytes(int(M), int(N), int(K), ctypes.byref(n)),
           "mx8_gemm_workspace_bytes")
    return int(n.value)


def mx8_gemm_plan(M: int, N: int, K: int) -> tuple:
    """(name, slices of K) of the kernel that mx8_gemm of this shape takes
    (include/mx8_plan.h)."""
    n = ctypes.c_int(0)
    name = lib().mx8_gemm_plan(int(M), int(N), int(K), ctypes.byref(n))
    if name is None:
        raise MX8Error(-2, "mx8_gemm_plan")
    return name.decode(), n.value


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MX8Error(status, what)


def _scale_bytes(K: int) -> int:
    return 16 * ((K + 511) // 512)


class MX8Tensor:
    """Rows of MX8: values [R, K] (float8_e4m3fn, unit column stride) and scales
    [R, 16 * ceil(K / 512)] (uint8, in include/mx8.h's order).  Rows may be cut
    out of both together: t[3:7].

    Made from two tensors, or by this module's calls in one allocation, the
    scales behind the values, whose views are built when they are asked for."""
    __slots__ = ("_data", "_parts", "_values", "_scales")

    def __init__(self, values: torch.Tensor, scales: torch.Tensor):
        self._data = self._parts = None
        self._values, self._scales = values, scales

    @property
    def values(self) -> torch.Tensor:
        if self._values is None:
            R, K = self._parts[:2]
            self._values = self._data[:R * K].view(VALUES).view(R, K)
        return self._values

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            R, K = self._parts[:2]
            self._scales = self._data[R * K:].view(R, _scale_bytes(K))
        return self._scales

    @property
    def shape(self) -> tuple:
        return tuple(self._values.shape) if self._parts is None else self._parts[:2]

    @property
    def block_scales(self) -> torch.Tensor:
        """The scales [R, K / 32] in the order of their blocks."""
        R, K = self.shape
        s = self.scales[:, :_scale_bytes(K)].unflatten(1, (-1, 4, 4)).transpose(2, 3)
        return s.flatten(1)[:, :K // BLOCK]

    def __getitem__(self, rows: slice) -> "MX8Tensor":
        if not isinstance(rows, slice):
            raise TypeError("an MX8Tensor is cut by a slice of rows")
        return MX8Tensor(self.values[rows], self.scales[rows])

    def __repr__(self) -> str:
        return "MX8Tensor(%d, %d)" % self.shape

    def parts(self, what: str) -> tuple:
        """(R, K, values pointer, stride, scales pointer, stride, device)."""
        if self._parts is not None:
            if self._parts[-1] < 0:
                raise ValueError("%s must be on the GPU" % what)
            return self._parts
        v, s = self._values, self._scales
        dev = _gpu(v, what)
        if v.dtype is not VALUES or s.dtype is not _u8:
            raise TypeError("%s must hold float8_e4m3fn values and uint8 scales, got %s and %s"
                            % (what, v.dtype, s.dtype))
        R, K, ldv = _rows(v, what)
        Rs, n, lds = _rows(s, what + ".scales")
        if Rs != R or n < _scale_bytes(K):
            raise ValueError("%s: scales %s do not fit values %s"
                             % (what, tuple(s.shape), tuple(v.shape)))
        _same(dev, _gpu(s, what))
        return R, K, v.data_ptr(), ldv, s.data_ptr(), lds, dev


def _new(R: int, K: int, like: torch.Tensor) -> MX8Tensor:
    if K < BLOCK or K % BLOCK:
        raise MX8Error(-2, "rows of (%d, %d)" % (R, K))
    n = _scale_bytes(K)
    t = MX8Tensor(None, None)
    t._data = data = like.new_empty(R * (K + n), dtype=_u8)
    p = data.data_ptr()
    t._parts = (R, K, p, K, p + R * K, n, data.get_device())
    return t


def empty_mx8(R: int, K: int, device="cuda") -> MX8Tensor:
    """Rows of the given shape, contents undefined."""
    if R < 0:
        raise MX8Error(-2, "rows of (%d, %d)" % (R, K))
    return _new(R, K, torch.empty(0, dtype=_u8, device=device))


def _target(out, R: int, K: int, dev: int, like: torch.Tensor) -> tuple:
    """(out or new rows, their parts)."""
    if out is None:
        out = _new(R, K, like)
        return out, out._parts
    if out.shape != (R, K):
        raise ValueError("out holds %s, this call writes %s" % (out.shape, (R, K)))
    parts = out.parts("out")
    _same(dev, parts[-1])
    return out, parts


def mx8_quantize(x: torch.Tensor, out: MX8Tensor | None = None,
                 fine: bool = False) -> MX8Tensor:
    """x [R, K] (BF16 or fp32, unit column stride) as MX8, in all of E4M3's steps if
    `fine`."""
    dev = _gpu(x, "x")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx8_quantize(x, out, fine)
    xt = _type_of(x.dtype) | (FINE_STEPS if fine else 0)
    R, K, ld = _rows(x, "x")
    out, (_, _, vp, ldv, sp, lds, _) = _target(out, R, K, dev, x)
    _check(lib().mx8_quantize(x.data_ptr(), xt, R, K, ld, vp, ldv, sp, lds, _raw_stream(dev)),
           "mx8_quantize")
    return out


def mx8_dequantize(q: MX8Tensor, out_dtype: torch.dtype = torch.bfloat16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that rows of MX8 stand for, [R, K]."""
    R, K, vp, ldv, sp, lds, dev = q.parts("q")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx8_dequantize(q, out_dtype, out)
    out, ld, yt = _output(out, R, K, out_dtype, dev, q._values if q._data is None else q._data)
    _check(lib().mx8_dequantize(vp, ldv, sp, lds, R, K, out.data_ptr(), yt, ld, _raw_stream(dev)),
           "mx8_dequantize")
    return out


def mx8_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                 out_dtype: torch.dtype = VALUES, out=None, fine: bool = False):
    """s / sqrt(mean(s^2) + eps) * weight over the rows of s = x + residual
    (rounded to the residual's type) or s = x: an MX8Tensor (in all of E4M3's
    steps if `fine`), or BF16 or fp32 as out_dtype (or `out`) says.  With a
    residual: (that, s); s goes to residual_out, which may be the residual itself,
    or to a new tensor."""
    dev = _gpu(x, "x")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx8_rms_norm(x, weight, eps, residual, residual_out, out_dtype, out, fine)
    M, K, ldx = _rows(x, "x")
    if weight.dim() != 1 or weight.shape[0] != K or (K > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be %d contiguous values" % K)
    _same(dev, _gpu(weight, "weight"))
    rp = op = None
    rt = ldr = ldo = 0
    if residual is not None:
        _same(dev, _gpu(residual, "residual"))
        rt = _type_of(residual.dtype)
        Mr, Kr, ldr = _rows(residual, "residual")
        if Mr != M or Kr != K:
            raise ValueError("residual is %s, x %s" % (tuple(residual.shape), (M, K)))
        if residual_out is None:
            residual_out, ldo = residual.new_empty((M, K)), K
        elif residual_out.dtype != residual.dtype or tuple(residual_out.shape) != (M, K):
            raise ValueError("residual_out must be %s of the residual's type" % ((M, K),))
        else:
            _same(dev, _gpu(residual_out, "residual_out"))
            _, _, ldo = _rows(residual_out, "residual_out")
        rp, op = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if isinstance(out, MX8Tensor) or (out is None and out_dtype is VALUES):
        out, (_, _, yp, ldy, sp, lds, _) = _target(out, M, K, dev, x)
        yt = OUT_MX8 | FINE_STEPS if fine else OUT_MX8
    elif fine:
        raise ValueError("fine steps are those of an MX8 output")
    else:
        out, ldy, yt = _output(out, M, K, out_dtype, dev, x)
        yp, sp, lds = out.data_ptr(), None, 0
    _check(lib().mx8_rms_norm(x.data_ptr(), _type_of(x.dtype), ldx, rp, op, rt, ldr, ldo,
                              weight.data_ptr(), _type_of(weight.dtype), float(eps), M, K, yp, yt,
                              ldy, sp, lds, _raw_stream(dev)), "mx8_rms_norm")
    return out if residual is None else (out, residual_out)


def mx8_gemm(x: MX8Tensor, w: MX4Tensor, out_dtype: torch.dtype = torch.float32,
             y: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m, n] = sum_k x[m, k] W[n, k] for x [M, K] in MX8 and a container w of
    one [N, K] in MX4."""
    if w.batch is not None:
        raise ValueError("w must hold one matrix")
    wc, wsc, dev = w.ptrs("w")
    if _away(dev):
        with torch.cuda.device(dev):
            return mx8_gemm(x, w, out_dtype, y, workspace)
    M, K, vp, ldv, sp, lds, x_dev = x.parts("x")
    if K != w.K:
        raise ValueError("x %s does not multiply w %s" % (x.shape, w.shape))
    _same(dev, x_dev)
    N = w.R
    y, ldy, yt = _output(y, M, N, out_dtype, dev, w.data)
    keep, wsp, wsb = _workspace(mx8_gemm_workspace_bytes(M, N, K), workspace, w.data)
    _check(lib().mx8_gemm(vp, ldv, sp, lds, M, wc, wsc, N, K, y.data_ptr(), ldy, yt, wsp, wsb,
                          _raw_stream(dev)), "mx8_gemm")
    return y
