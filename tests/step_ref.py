"""Plain 64-bit numpy forms, for the tests, of what stands between the products
of a verify step: the MX8 format from its description, the residual addition and
norm, the routing of tokens to experts and the verification of drafted tokens,
written with plain loops over their definitions."""
from __future__ import annotations

import numpy as np

from tests.mx4_ref import bf16_to_f64, f64_to_bf16_bits


def e4m3_table() -> np.ndarray:
    """The value of every E4M3 byte."""
    v = np.zeros(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = np.nan if e == 15 and m == 7 else (-x if s else x)
    return v


TABLE = e4m3_table()


def nearest_e4m3(t: np.ndarray) -> np.ndarray:
    """Bytes 0..126 nearest to magnitudes t >= 0 among the multiples of 1/4, ties to the
    even multiple (from 4 on: the even byte), 448 at most."""
    grid = TABLE[:127]
    t = np.where(t < 4.0, np.rint(t * 4.0) / 4.0, t)
    i = np.clip(np.searchsorted(grid, t, side="right") - 1, 0, 125)
    lo, hi = t - grid[i], grid[i + 1] - t
    up = (hi < lo) | ((hi == lo) & (i % 2 == 1))
    return np.where(t >= 448.0, 126, i + up).astype(np.uint8)


def exponent(top: np.ndarray) -> np.ndarray:
    """The scale byte of blocks whose largest magnitude is top (0 and up, finite)."""
    x = np.frexp(top)[1] - 1
    return np.where(top > 0, np.maximum(x - 8 + 127, 0), 0)


def encode8(v: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(bytes [..., K], scale bytes [..., K / 32]) of fp32 values in float64."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    fin = np.where(np.isfinite(b), b, 0.0)
    e = exponent(np.abs(fin).max(-1))
    code = nearest_e4m3(np.abs(fin) / np.ldexp(1.0, e - 127)[..., None])
    code = code | (np.signbit(fin).astype(np.uint8) << 7)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    return code.reshape(v.shape), np.where(bad, 255, e).astype(np.uint8)


def decode8(code: np.ndarray, e: np.ndarray) -> np.ndarray:
    s = np.where(e == 255, np.nan, np.ldexp(1.0, e.astype(int) - 127))
    return (TABLE[code].reshape(*e.shape, 32) * s[..., None]).reshape(code.shape)


def scale_rows(e: np.ndarray) -> np.ndarray:
    """Scales [R, K / 32] in the order they are kept in: [R, 16 * ceil(K / 512)]."""
    R, n = e.shape
    out = np.full((R, 16 * ((n + 15) // 16)), 127, np.uint8)
    for block in range(n):
        k = 32 * block
        out[:, 16 * (k // 512) + 4 * (k % 128 // 32) + k % 512 // 128] = e[:, block]
    return out


def norm(x, res, w, eps, res_bf16):
    """(y, s): x, res (or None) and w in float64 that hold BF16 or fp32 values."""
    s = x
    if res is not None:
        s = (x.astype(np.float32) + res.astype(np.float32)).astype(np.float64)
        if res_bf16:
            s = bf16_to_f64(f64_to_bf16_bits(s))
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s * r * w, s


def route(logits, k, scores="softmax", bias=None, groups=1, kept=1, terms=1, renorm=True,
          scale=1.0):
    """(experts int [T, k], shares [T, k])."""
    T, E = logits.shape
    experts, shares = np.full((T, k), -1), np.zeros((T, k))
    inf = np.inf
    with np.errstate(all="ignore"):
        for t in range(T):
            l = logits[t].astype(np.float64)
            if scores == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-l))
            else:
                p = np.exp(l - l.max()) if not np.isnan(l).any() else np.full(E, np.nan)
                s = p / p.sum()
            b = np.zeros(E) if bias is None else bias.astype(np.float64)
            value = s + b
            rank = l if bias is None else value
            # NaN above all, what is not to be chosen below all
            order = np.where(np.isnan(rank) | np.isnan(l), inf, rank)
            tier = (np.isnan(rank) | np.isnan(l)).astype(int)
            allowed = (l != -inf) & (b != -inf)
            if kept < groups:
                per, of = E // groups, []
                for g in range(groups):
                    ids = [e for e in range(g * per, (g + 1) * per) if allowed[e]]
                    if not ids:
                        of.append((-1, 0.0))
                    elif terms == 1:
                        of.append(max((tier[e], order[e]) for e in ids))
                    elif any(np.isnan(value[e]) for e in ids):
                        of.append((1, inf))
                    else:
                        of.append((0, sum(sorted((value[e] for e in ids), reverse=True)[:2])))
                best = sorted(range(groups), key=lambda g: (-of[g][0], -of[g][1], g))[:kept]
                for g in range(groups):
                    if g not in best:
                        allowed[g * per:(g + 1) * per] = False
            ids = sorted((e for e in range(E) if allowed[e]),
                         key=lambda e: (-tier[e], -order[e], e))[:k]
            total = sum(s[e] for e in ids)
            for j, e in enumerate(ids):
                experts[t, j] = e
                shares[t, j] = scale * ((0.0 if total == 0 else s[e] / total) if renorm else s[e])
    return experts, shares


def verify(logits, drafts, uniforms, probs=None, lengths=None, tau=None):
    """(tokens [B, D + 1], accepted [B])."""
    B, rows, V = logits.shape
    D = rows - 1
    tokens, accepted = np.full((B, rows), -1), np.zeros(B, int)
    with np.errstate(all="ignore"):
        for b in range(B):
            n = D if lengths is None else min(max(int(lengths[b]), 0), D)
            temp = 1.0 if tau is None else float(tau[b])
            for i in range(n + 1):
                l = logits[b, i].astype(np.float64)
                x = int(drafts[b, i]) if i < n else None
                accepted[b] = i
                good = not np.isnan(l).any() and -np.inf < l.max() < np.inf
                if not good:
                    break
                if not temp > 0:
                    token = int(np.argmax(l))
                    if x == token:
                        tokens[b, i] = x
                        continue
                    tokens[b, i] = token
                    break
                p = np.exp((l - l.max()) / temp)
                p /= p.sum()
                q = np.zeros(V)
                if x is not None:
                    inside = 0 <= x < V
                    if probs is not None:
                        q = probs[b, i].astype(np.float64)
                    elif inside:
                        q[x] = 1.0
                    if inside and float(uniforms[b, i]) * q[x] < p[x]:
                        tokens[b, i] = x
                        continue
                w = np.maximum(p - q, 0.0)
                if not w.sum() > 0:
                    w = p
                run = np.cumsum(w)
                hit = np.nonzero((run > float(uniforms[b, D]) * run[-1]) & (w > 0))[0]
                tokens[b, i] = hit[0] if len(hit) else np.nonzero(w > 0)[0][-1]
                break
    return tokens, accepted
