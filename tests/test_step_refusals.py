"""What the MX8, routing and draft calls refuse before any launch, and their
exports and sizes, without a GPU."""
import ctypes
import os
import re

import pytest
import torch

from lossless_bit_weight_amd import draft, mx4, mx8, w12

P = ctypes.c_void_p
A, MIS = P(4096), P(4104)       # never dereferenced: every call here fails validation


@pytest.mark.parametrize("header,lib,names", [
    ("mx8.h", mx8.lib, {"mx8_status_string", "mx8_scale_row_bytes", "mx8_quantize",
                        "mx8_dequantize", "mx8_rms_norm", "mx8_gemm",
                        "mx8_gemm_workspace_bytes"}),
    ("mx4_route.h", mx4.lib, {"mx4_route", "mx4_moe_routed"}),
    ("draft.h", draft.lib, {"draft_status_string", "draft_verify", "draft_workspace_bytes"})])
def test_exports_every_declared_symbol(header, lib, names):
    with open(os.path.join(os.path.dirname(w12.HEADER_PATH), header)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    found = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*((?:mx8|mx4|draft)_\w+)\s*\(", text,
                       flags=re.M)
    assert set(found) == names
    for n in names:
        assert hasattr(lib(), n), n


def test_sizes_and_status():
    assert mx8.mx8_scale_row_bytes(5120) == 160 and mx8.mx8_scale_row_bytes(32) == 16
    assert mx8.mx8_scale_row_bytes(544) == 32
    for bad in (0, -32, 33, 1 << 24):
        assert mx8.mx8_scale_row_bytes(bad) == 0
    for s in (0, -1, -2, -3, -4, -6, -7, -8, 99):
        assert mx8.mx8_status_string(s) and draft.draft_status_string(s)
    assert mx8.mx8_gemm_workspace_bytes(0, 16, 32) == 0
    assert draft.draft_workspace_bytes(0, 4, 100) == 0
    assert draft.draft_workspace_bytes(1, 0, 1) > 0
    n = ctypes.c_size_t(7)
    assert mx8.lib().mx8_gemm_workspace_bytes(1, 16, 33, ctypes.byref(n)) == -2 and n.value == 0
    assert mx8.lib().mx8_gemm_workspace_bytes(1, 16, 32, None) == -1
    assert draft.lib().draft_workspace_bytes(1, 1, 0, ctypes.byref(n)) == -2 and n.value == 0
    assert draft.lib().draft_workspace_bytes(1, 1, 1, None) == -1


def test_zero_rows_launch_nothing():
    assert mx8.lib().mx8_quantize(None, 0, 0, 64, 64, None, 64, None, 16, None) == 0
    assert mx8.lib().mx8_dequantize(None, 64, None, 16, 0, 64, None, 0, 64, None) == 0
    assert mx8.lib().mx8_rms_norm(None, 0, 64, None, None, 0, 0, 0, A, 0, 1e-6, 0, 64, None, 2, 64,
                                  None, 16, None) == 0
    assert mx8.lib().mx8_gemm(None, 64, None, 16, 0, A, A, 16, 64, None, 16, 0, None, 0, None) == 0
    assert mx4.lib().mx4_route(None, 1, 0, 8, 8, None, 0, 1, 1, 1, 2, 1, 1.0, None, None, None) == 0
    assert mx4.lib().mx4_moe_routed(None, 0, 64, None, None, A, A, A, A, 64, 32, 4, 2, None, 64, 0,
                                    None, 0, None) == 0
    assert draft.lib().draft_verify(None, 1, 0, 3, 9, 36, 9, None, 0, None, None, 0, 0, 0, None,
                                    None, None, None, None, 0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(v=None), -1), (dict(s=None), -1), (dict(t=2), -4), (dict(t=-1), -4),
    (dict(R=-1), -2), (dict(K=0), -2), (dict(K=40), -2), (dict(K=1 << 24, ldx=1 << 24), -2),
    (dict(ldx=32), -2), (dict(ldx=68), -3), (dict(t=1, ldx=66), -3), (dict(x=MIS), -3),
    (dict(v=MIS), -3), (dict(s=MIS), -3), (dict(ldv=48), -2), (dict(ldv=72), -3),
    (dict(lds=0), -2), (dict(lds=24), -3), (dict(R=1 << 40), -2), (dict(K=544, ldx=544, ldv=544),
                                                                   -2)])
@pytest.mark.parametrize("inverse", [False, True])
def test_codec_rejects(kw, status, inverse):
    a = dict(x=A, t=0, R=16, K=64, ldx=64, v=A, ldv=64, s=A, lds=16)
    a.update(kw)
    if inverse:
        rc = mx8.lib().mx8_dequantize(a["v"], a["ldv"], a["s"], a["lds"], a["R"], a["K"], a["x"],
                                      a["t"], a["ldx"], None)
    else:
        rc = mx8.lib().mx8_quantize(a["x"], a["t"], a["R"], a["K"], a["ldx"], a["v"], a["ldv"],
                                    a["s"], a["lds"], None)
    assert rc == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(ys=None), -1),
    (dict(ro=None), -1), (dict(M=-1), -2), (dict(M=(1 << 24) + 1), -2), (dict(K=48), -2),
    (dict(K=32800, ldx=32800, ldr=32800, ldo=32800, ldy=32800, lds=2048), -6),
    (dict(xt=2), -4), (dict(rt=2), -4), (dict(wt=2), -4), (dict(yt=3), -4), (dict(yt=-1), -4),
    (dict(ldx=32), -2), (dict(ldr=32), -2), (dict(ldo=32), -2), (dict(ldy=32), -2),
    (dict(lds=8), -2), (dict(lds=24), -3), (dict(ldr=66), -3), (dict(x=MIS), -3),
    (dict(r=MIS), -3), (dict(ro=MIS), -3), (dict(w=MIS), -3), (dict(y=MIS), -3),
    (dict(ys=MIS), -3), (dict(yt=0, ldy=68), -3)])
def test_norm_rejects(kw, status):
    a = dict(x=A, xt=0, ldx=64, r=A, ro=A, rt=0, ldr=64, ldo=64, w=A, wt=0, M=3, K=64, y=A, yt=2,
             ldy=64, ys=A, lds=16)
    a.update(kw)
    rc = mx8.lib().mx8_rms_norm(a["x"], a["xt"], a["ldx"], a["r"], a["ro"], a["rt"], a["ldr"],
                                a["ldo"], a["w"], a["wt"], 1e-6, a["M"], a["K"], a["y"], a["yt"],
                                a["ldy"], a["ys"], a["lds"], None)
    assert rc == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(xs=None), -1), (dict(w=None), -1), (dict(ws=None), -1),
    (dict(y=None), -1), (dict(M=-1), -2), (dict(M=(1 << 24) + 1), -2), (dict(N=0), -2),
    (dict(K=33), -2), (dict(ldy=31), -2), (dict(yt=2), -4), (dict(w=MIS), -3), (dict(ws=MIS), -3),
    (dict(x=MIS), -3), (dict(xs=MIS), -3), (dict(y=P(4097)), -3), (dict(yt=1, y=P(4098)), -3),
    (dict(ldv=48), -2), (dict(ldv=72), -3), (dict(lds=8), -2), (dict(lds=24), -3),
    (dict(ldv=1 << 31), -2), (dict(lds=1 << 31), -2),
    (dict(N=(1 << 27) + 1, ldy=1 << 29), -2), (dict(M=1 << 24, N=(1 << 13) + 1, ldy=1 << 14), -2)])
def test_gemm_rejects(kw, status):
    a = dict(x=A, ldv=64, xs=A, lds=16, M=3, w=A, ws=A, N=32, K=64, y=A, ldy=32, yt=0)
    a.update(kw)
    assert mx8.lib().mx8_gemm(a["x"], a["ldv"], a["xs"], a["lds"], a["M"], a["w"], a["ws"], a["N"],
                              a["K"], a["y"], a["ldy"], a["yt"], None, 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(l=None), -1), (dict(e=None), -1), (dict(s=None), -1), (dict(lt=2), -4), (dict(kind=2), -4),
    (dict(T=-1), -2), (dict(E=0), -2), (dict(k=0), -2), (dict(k=65), -2), (dict(k=33), -6),
    (dict(E=1025, ldl=1025), -6), (dict(T=(1 << 24) + 1), -6), (dict(ldl=63), -2),
    (dict(groups=0), -2), (dict(groups=3), -2), (dict(kept=0), -2), (dict(groups=4, kept=5), -2),
    (dict(E=128, ldl=128, groups=128), -6), (dict(terms=0), -2), (dict(terms=3), -2),
    (dict(l=P(4098)), -3), (dict(lt=0, l=P(4097)), -3), (dict(b=P(4098)), -3),
    (dict(e=P(4098)), -3), (dict(s=P(4098)), -3)])
def test_route_rejects(kw, status):
    a = dict(l=A, lt=1, T=3, E=64, ldl=64, b=None, kind=0, groups=1, kept=1, terms=1, k=4, e=A, s=A)
    a.update(kw)
    assert mx4.lib().mx4_route(a["l"], a["lt"], a["T"], a["E"], a["ldl"], a["b"], a["kind"],
                               a["groups"], a["kept"], a["terms"], a["k"], 1, 1.0, a["e"], a["s"],
                               None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(e=None), -1), (dict(p=None), -1), (dict(a=None), -1),
    (dict(d=None), -1), (dict(y=None), -1), (dict(T=-1), -2), (dict(T=129), -6), (dict(k=0), -2),
    (dict(k=5), -2), (dict(H=48), -2), (dict(I=16), -2), (dict(e=P(4098)), -3),
    (dict(p=P(4098)), -3), (dict(x=MIS), -3), (dict(ldy=63), -2), (dict(yt=2), -4), (dict(), -8)])
def test_moe_routed_rejects(kw, status):
    a = dict(x=A, T=3, e=A, p=A, a=A, d=A, H=64, I=32, E=4, k=2, y=A, ldy=64, yt=0)
    a.update(kw)
    assert mx4.lib().mx4_moe_routed(a["x"], a["T"], 64, a["e"], a["p"], a["a"], A, A, a["d"],
                                    a["H"], a["I"], a["E"], a["k"], a["y"], a["ldy"], a["yt"],
                                    None, 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(l=None), -1), (dict(d=None), -1), (dict(u=None), -1), (dict(t=None), -1),
    (dict(a=None), -1), (dict(lt=2), -4), (dict(q=A, qt=2), -4), (dict(B=-1), -2), (dict(D=-1), -2),
    (dict(V=0), -2), (dict(V=(1 << 30) + 1), -2), (dict(D=1024), -6), (dict(B=1 << 24), -2),
    (dict(B=1 << 20, V=1 << 20), -2), (dict(ldd=8), -2), (dict(ldb=-1), -2), (dict(q=A, pdd=8), -2),
    (dict(q=A, pdb=-1), -2), (dict(l=P(4098)), -3), (dict(lt=0, l=P(4097)), -3),
    (dict(q=P(4097), qt=0), -3), (dict(d=P(4098)), -3), (dict(d64=1, d=P(4100)), -3),
    (dict(u=P(4097)), -3), (dict(n=P(4097)), -3), (dict(tau=P(4097)), -3), (dict(t=P(4097)), -3),
    (dict(a=P(4097)), -3), (dict(), -8), (dict(ws=P(4096 + 16)), -8), (dict(ws=A, wb=8), -8)])
def test_verify_rejects(kw, status):
    a = dict(l=A, lt=1, B=2, D=3, V=9, ldb=36, ldd=9, d=A, d64=0, u=A, q=None, qt=1, pdb=27, pdd=9,
             n=None, tau=None, t=A, a=A, ws=None, wb=1 << 20)
    a.update(kw)
    assert draft.lib().draft_verify(a["l"], a["lt"], a["B"], a["D"], a["V"], a["ldb"], a["ldd"],
                                    a["d"], a["d64"], a["u"], a["q"], a["qt"], a["pdb"], a["pdd"],
                                    a["n"], a["tau"], a["t"], a["a"], a["ws"], a["wb"],
                                    None) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: mx8.mx8_quantize(x), lambda: mx8.mx8_rms_norm(x, x[0]),
                 lambda: mx4.mx4_route(x.float(), 2),
                 lambda: draft.draft_verify(torch.zeros(1, 2, 8), torch.zeros(1, 1, dtype=torch.int32),
                                            torch.zeros(1, 2))):
        with pytest.raises(ValueError):
            call()
