"""The MX4 calls without a GPU: exports, sizes, and what they refuse before any
launch."""
import ctypes
import os
import re

import pytest
import torch

from lossless_bit_weight_amd import mx4, w12

P = ctypes.c_void_p
A = P(4096)         # a non-null, 256-byte aligned stand-in (never dereferenced:
MIS = P(4104)       # every call below fails validation before any launch)
HEADER = os.path.join(os.path.dirname(w12.HEADER_PATH), "mx4.h")


def test_exports_every_declared_symbol():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(mx4_\w+)\s*\(", text, flags=re.M)
    assert set(names) == {"mx4_status_string", "mx4_codes_bytes", "mx4_scales_bytes",
                          "mx4_quantize", "mx4_dequantize", "mx4_gemm", "mx4_gemm_mx4",
                          "mx4_gemm_workspace_bytes", "mx4_moe", "mx4_moe_workspace_bytes"}
    for n in names:
        assert hasattr(mx4.lib(), n), n


def test_sizes():
    assert mx4.mx4_codes_bytes(1, 7168, 5120) == 7168 * 5120 // 2
    assert mx4.mx4_scales_bytes(1, 7168, 5120) == 7168 * 5120 // 32
    assert mx4.mx4_codes_bytes(3, 17, 160) == 3 * 2 * 2 * 1024
    assert mx4.mx4_scales_bytes(3, 17, 160) == 3 * 2 * 256
    assert mx4.mx4_codes_bytes(1, 0, 32) == 0
    for bad in ((0, 16, 32), (1, -1, 32), (1, 16, 0), (1, 16, 48), (1, 16, 1 << 24),
                (1, 1 << 40, 32), (1 << 39, 16, 32), (1 << 20, 1 << 20, 512)):
        assert mx4.mx4_codes_bytes(*bad) == 0 and mx4.mx4_scales_bytes(*bad) == 0, bad
    for s in (0, -1, -2, -3, -4, -6, -7, -8, 99):
        assert mx4.mx4_status_string(s)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(codes=None), -1), (dict(scales=None), -1), (dict(t=2), -4),
    (dict(t=-1), -4), (dict(B=0), -2), (dict(R=-1), -2), (dict(K=0), -2), (dict(K=40), -2),
    (dict(K=1 << 24, ldx=1 << 24), -2), (dict(ldx=32), -2), (dict(ldx=68), -3),
    (dict(t=1, ldx=66), -3), (dict(x=MIS), -3), (dict(codes=MIS), -3), (dict(scales=MIS), -3),
    (dict(B=2, ldb=-8), -2), (dict(B=2, ldb=1028), -3), (dict(R=1 << 40), -2)])
@pytest.mark.parametrize("inverse", [False, True])
def test_codec_rejects(kw, status, inverse):
    a = dict(x=A, t=0, B=1, R=16, K=64, ldx=64, ldb=0, codes=A, scales=A)
    a.update(kw)
    if inverse:
        rc = mx4.lib().mx4_dequantize(a["codes"], a["scales"], a["B"], a["R"], a["K"], a["x"],
                                      a["t"], a["ldx"], a["ldb"], None)
    else:
        rc = mx4.lib().mx4_quantize(a["x"], a["t"], a["B"], a["R"], a["K"], a["ldx"], a["ldb"],
                                    a["codes"], a["scales"], None)
    assert rc == status


def test_dequantize_refuses_overlapping_matrices():
    assert mx4.lib().mx4_dequantize(A, A, 2, 16, 64, A, 0, 64, 512, None) == -2


def test_zero_rows_launch_nothing():
    L = mx4.lib()
    assert L.mx4_quantize(None, 0, 1, 0, 64, 64, 0, None, None, None) == 0
    assert L.mx4_dequantize(None, None, 1, 0, 64, None, 0, 64, 0, None) == 0
    assert L.mx4_gemm(None, 0, 64, A, A, 16, 64, None, 16, 0, None, 0, None) == 0
    assert L.mx4_gemm_mx4(None, None, 0, A, A, 16, 64, None, 16, 0, None, 0, None) == 0
    assert L.mx4_moe(None, 0, 64, None, 4, A, A, A, A, 64, 32, 4, 2, 1, None, 64, 0, None, 0,
                     None) == 0


GEMM_BAD = [(dict(w=None), -1), (dict(ws=None), -1), (dict(y=None), -1), (dict(M=-1), -2),
            (dict(M=(1 << 24) + 1), -2), (dict(N=0), -2), (dict(K=33), -2), (dict(ldy=31), -2),
            (dict(yt=2), -4), (dict(w=MIS), -3), (dict(ws=MIS), -3), (dict(y=P(4097)), -3),
            (dict(yt=1, y=P(4098)), -3), (dict(x=None), -1), (dict(x=MIS), -3),
            (dict(N=1 << 40, ldy=1 << 40), -2), (dict(N=(1 << 27) + 1, ldy=1 << 29), -2),
            (dict(M=1 << 24, N=(1 << 13) + 1, ldy=1 << 14), -2)]


@pytest.mark.parametrize("kw,status", GEMM_BAD + [(dict(ldx=60), -2), (dict(ldx=68), -3)])
def test_gemm_rejects(kw, status):
    a = dict(x=A, M=3, ldx=64, w=A, ws=A, N=32, K=64, y=A, ldy=32, yt=0)
    a.update(kw)
    assert mx4.lib().mx4_gemm(a["x"], a["M"], a["ldx"], a["w"], a["ws"], a["N"], a["K"], a["y"],
                              a["ldy"], a["yt"], None, 0, None) == status


@pytest.mark.parametrize("kw,status", GEMM_BAD + [(dict(xs=None), -1), (dict(xs=MIS), -3)])
def test_gemm_mx4_rejects(kw, status):
    a = dict(x=A, xs=A, M=3, w=A, ws=A, N=32, K=64, y=A, ldy=32, yt=0)
    a.update(kw)
    assert mx4.lib().mx4_gemm_mx4(a["x"], a["xs"], a["M"], a["w"], a["ws"], a["N"], a["K"],
                                  a["y"], a["ldy"], a["yt"], None, 0, None) == status


@pytest.mark.parametrize("x_mx4", [False, True])
def test_gemm_workspace(x_mx4):
    """A shape that splits K asks for a workspace and refuses to run without."""
    L = mx4.lib()
    need = mx4.mx4_gemm_workspace_bytes(33, 512, 17408, x_mx4)
    if need:
        for ws, n in ((None, need), (A, need - 1), (P(4096 + 16), need)):
            if x_mx4:
                rc = L.mx4_gemm_mx4(A, A, 33, A, A, 512, 17408, A, 512, 0, ws, n, None)
            else:
                rc = L.mx4_gemm(A, 33, 17408, A, A, 512, 17408, A, 512, 0, ws, n, None)
            assert rc == -8
    n = ctypes.c_size_t(7)
    assert L.mx4_gemm_workspace_bytes(1, 16, 33, 0, ctypes.byref(n)) == -2 and n.value == 0
    assert L.mx4_gemm_workspace_bytes(1, 16, 32, 0, None) == -1
    assert mx4.mx4_gemm_workspace_bytes(0, 16, 32) == 0
    assert mx4.mx4_gemm_workspace_bytes(1, 1 << 27, 32, x_mx4) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(l=None), -1), (dict(a=None), -1), (dict(b=None), -1),
    (dict(c=None), -1), (dict(d=None), -1), (dict(y=None), -1), (dict(T=-1), -2),
    (dict(T=129), -6), (dict(H=0), -2), (dict(H=40, ldx=40, ldy=40), -2), (dict(I=0), -2),
    (dict(I=48), -2), (dict(E=0), -2), (dict(E=1025, ldl=1025), -6), (dict(k=0), -2),
    (dict(k=5), -2), (dict(E=64, ldl=64, k=33), -6), (dict(ldx=32), -2), (dict(ldx=68), -3),
    (dict(ldl=3), -2), (dict(ldy=63), -2), (dict(yt=2), -4), (dict(x=MIS), -3),
    (dict(l=P(4098)), -3), (dict(a=MIS), -3), (dict(b=MIS), -3), (dict(c=MIS), -3),
    (dict(d=MIS), -3), (dict(y=P(4097)), -3), (dict(w=None), -8), (dict(w=MIS), -8),
    (dict(n=100), -8), (dict(I=1 << 24), -2),
    (dict(H=1 << 23, ldx=1 << 23, ldy=1 << 23, T=128, E=64, ldl=64, k=32), -2)])
def test_moe_rejects(kw, status):
    a = dict(x=A, T=2, ldx=64, l=A, ldl=4, a=A, b=A, c=A, d=A, H=64, I=32, E=4, k=2, y=A, ldy=64,
             yt=0, w=A, n=1 << 30)
    a.update(kw)
    assert mx4.lib().mx4_moe(a["x"], a["T"], a["ldx"], a["l"], a["ldl"], a["a"], a["b"], a["c"],
                             a["d"], a["H"], a["I"], a["E"], a["k"], 1, a["y"], a["ldy"], a["yt"],
                             a["w"], a["n"], None) == status


def test_moe_workspace():
    n = ctypes.c_size_t(7)
    L = mx4.lib()
    assert L.mx4_moe_workspace_bytes(1, 64, 32, 4, 5, 0, ctypes.byref(n)) == -2 and n.value == 0
    assert L.mx4_moe_workspace_bytes(1, 64, 32, 4, 2, 3, ctypes.byref(n)) == -4
    assert mx4.mx4_moe_workspace_bytes(0, 64, 32, 4, 2) == 0
    small = mx4.mx4_moe_workspace_bytes(16, 64, 1280, 64, 6)
    assert 16 * 6 * 1280 * 4 <= small < mx4.mx4_moe_workspace_bytes(16, 64, 1280, 64, 6,
                                                                    torch.float32)


def test_binding_refuses_before_the_library():
    """Types, shapes and places that the binding turns down; CPU tensors never
    reach a launch."""
    cpu = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mx4.mx4_quantize(cpu)
    with pytest.raises(mx4.MX4Error):
        mx4.empty_mx4(4, 40, device="cpu")
    with pytest.raises(mx4.MX4Error):
        mx4.empty_mx4(4, 64, batch=0, device="cpu")
    q = mx4.empty_mx4(4, 64, device="cpu")
    assert q.nbytes == 1024 + 256 and q.shape == (4, 64)
    assert q.codes.numel() == 1024 and q.scales.numel() == 256
    with pytest.raises(ValueError):
        mx4.mx4_dequantize(q)
    with pytest.raises(ValueError):
        mx4.mx4_gemm(cpu, q)
    with pytest.raises(ValueError):
        mx4.mx4_moe(cpu, torch.zeros((4, 2)), q, q, 1)
    assert issubclass(mx4.MX4Error, w12.W12Error)
