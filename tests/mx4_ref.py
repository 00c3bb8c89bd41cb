"""Plain 64-bit numpy form of the MX4 operators for the tests: the encoding from
its formula, the container's layout from its description, the products and the
expert layer with bounds on what fp32 sums may be off by."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16_bits(v: np.ndarray) -> np.ndarray:
    """Nearest BF16 (ties to even) of finite fp32-exact values."""
    u = v.astype(np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def encode(v: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(codes uint8 [..., K], scale bytes uint8 [..., K / 32]) of fp32 values
    held in float64."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    fin = np.where(np.isfinite(b), b, 0.0)
    top = np.abs(fin).max(-1)
    # floor(log2(top)) exactly: top = m 2^x with m in [1/2, 1)
    x = np.frexp(top)[1] - 1
    e = np.where(top > 0, np.maximum(x - 2 + 127, 0), 0)
    t = np.abs(fin) / np.ldexp(1.0, e - 127)[..., None]
    # nearest grid value; a tie goes to the even index
    i = np.clip(np.searchsorted(GRID, t, side="right") - 1, 0, 6)
    lo, hi = t - GRID[i], GRID[i + 1] - t
    code = np.where(lo < hi, i, np.where(lo > hi, i + 1, np.where(i % 2 == 0, i, i + 1)))
    code = np.where(t > 6.0, 7, code).astype(np.uint8) | (np.signbit(fin).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    e = np.where(bad, 255, e).astype(np.uint8)
    return code.reshape(v.shape), e


def decode(code: np.ndarray, e: np.ndarray) -> np.ndarray:
    s = np.where(e == 255, np.nan, np.ldexp(1.0, e.astype(int) - 127))
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(*e.shape, 32) * s[..., None]).reshape(code.shape)


def rounded(v: np.ndarray) -> np.ndarray:
    return decode(*encode(v))


def container(code: np.ndarray, e: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(code bytes, scale bytes), flat, of codes [B, R, K] in the documented
    layout, written with plain loops over its indices."""
    B, R, K = code.shape
    T, G, Q = (R + 15) // 16, (K + 127) // 128, (K + 511) // 512
    full = np.zeros((B, T * 16, G * 128), np.uint8)
    full[:, :R, :K] = code
    sc = np.full((B, T * 16, Q * 16), 127, np.uint8)
    sc[:, :R, :K // 32] = e
    codes = np.zeros((B, T, G, 64, 16), np.uint8)
    scales = np.zeros((B, T, Q, 64, 4), np.uint8)
    for L in range(64):
        c, q = L % 16, L // 16
        rows = full[:, c::16].reshape(B, T, G, 4, 32)[:, :, :, q]
        codes[:, :, :, L] = rows[..., 0::2] | (rows[..., 1::2] << 4)
        scales[:, :, :, L] = sc[:, c::16].reshape(B, T, Q, 4, 4)[..., q]
    return codes.reshape(-1), scales.reshape(-1)


def gamma(n: int) -> float:
    """Relative error of a sum of n products in fp32, any order, each step off by
    at most one last place (2^-23)."""
    return (n + 8) * 2.0 ** -23


def matmul(x: np.ndarray, w: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(x w^T, bound on an fp32 sum's error)."""
    return x @ w.T, gamma(x.shape[1]) * (np.abs(x) @ np.abs(w).T) + 1e-37


def moe(x, logits, w13, w2, k, renormalize, parts):
    """(y, bound): the expert layer in 64 bits and what its fp32 form with hidden
    values in `parts` BF16 parts may be off by."""
    T, E = logits.shape
    I, H = w2.shape[2], w2.shape[1]
    y, tol = np.zeros((T, H)), np.full((T, H), 1e-37)
    for t in range(T):
        order = sorted((e for e in range(E) if logits[t, e] != -np.inf),
                       key=lambda e: (-logits[t, e], e))[:k]
        if not order:
            continue
        l = logits[t].astype(np.float64)
        top = l[order[0]]
        total = sum(np.exp(l[e] - top) for e in (order if renormalize else range(E)))
        for e in order:
            p = np.exp(l[e] - top) / total
            gu, d = matmul(x[t:t + 1], w13[e])
            g, u, dg, du = gu[0, :I], gu[0, I:], d[0, :I], d[0, I:]
            silu = g / (1 + np.exp(-g))
            h = silu * u
            # |silu'| <= 1.1; exp, division and products in fp32: a few last places,
            # exp's argument adding |g| of them; the parts leave 2^-8 each
            dh = (1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du
                  + np.abs(h) * ((8 + np.abs(g)) * 2.0 ** -23 + 2.0 ** (-8 * parts)))
            o, do = matmul(h[None], w2[e])
            y[t] += p * o[0]
            # the waves' split adds partial sums: within gamma's n + 8; the share's own
            # exp and division: a few last places and |l - top|
            rel = (16 + abs(l[e] - top) + k) * 2.0 ** -23
            tol[t] += p * (do[0] * parts + dh @ np.abs(w2[e]).T
                           + rel * (np.abs(h) @ np.abs(w2[e]).T))
    return y, tol


def assert_close(got: np.ndarray, ref: np.ndarray, tol: np.ndarray, out: str, what: str) -> None:
    """|got - ref| <= tol, plus half a step of the output type; NaN meets NaN."""
    got = got.astype(np.float64)
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what + ": NaN positions differ"
    bound = tol + (np.abs(ref) + tol) * (2.0 ** -8 if out == "bf16" else 2.0 ** -24)
    fin = ~np.isnan(ref)
    err = np.abs(got - ref)[fin]
    bad = err > bound[fin]
    assert not bad.any(), "%s: %d of %d off; worst %.3e against %.3e" % (
        what, bad.sum(), bad.size, err[np.argmax(err - bound[fin])],
        bound[fin][np.argmax(err - bound[fin])])
