"""Measured cases of the MX4 operators (lossless_bit_weight_amd.mx4):
quantisation to 4-bit blocks of 32 under a shared power-of-two scale and its
inverse, the product with 4-bit weights (activations in BF16, or quantised
too), and a mixture-of-experts layer on 4-bit experts for a few tokens.

A case names its operator in "op":

  codec   x [R, K] -> MX4 -> the values it stands for, in x's type
  linear  y = x W^T, W [N, K] in MX4, x [M, K] BF16 read as it is
  linear4 the same with x quantised to MX4 within the pass
  moe     y[t] = sum over the top_k experts e of token t of
          p[t, e] W2[e] (silu(G[e] x[t]) * U[e] x[t]), where
          W13[e] = [G[e]; U[e]] and p is the softmax of the token's router
          logits over its chosen experts

Each has its plain form (elementary torch operations in 32 bits), the calls
a program makes of the library (`own`), and the definition in 64 bits
(`exact`).
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32                      # values that share one scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # magnitudes of a 4-bit code


def listed():
    return [
        # the activations of one token before a product: latency only
        {"name": "codec_one_token", "op": "codec", "R": 1, "K": 5120, "dtype": "bf16"},
        # the activations of a prompt
        {"name": "codec_prompt", "op": "codec", "R": 4096, "K": 5120, "dtype": "bf16"},
        # a weight converted from its fp32 master, a row short of whole tiles
        {"name": "codec_weight_f32", "op": "codec", "R": 5119, "K": 17408, "dtype": "f32"},
        # QKV of one request's decode step
        {"name": "linear_qkv_m1", "op": "linear", "M": 1, "N": 7168, "K": 5120, "out": "bf16"},
        # gate+up over a drafted block of 16 tokens
        {"name": "linear_gate_up_m16", "op": "linear", "M": 16, "N": 34816, "K": 5120,
         "out": "bf16"},
        # a down projection's shard with ragged rows, an odd batch, fp32 out
        {"name": "linear_ragged_m33", "op": "linear", "M": 33, "N": 5003, "K": 17376,
         "out": "f32"},
        # QKV over a prompt
        {"name": "linear_qkv_m2048", "op": "linear", "M": 2048, "N": 7168, "K": 5120,
         "out": "bf16"},
        # the O projection of a small batch, activations in 4 bits too
        {"name": "linear4_o_m7", "op": "linear4", "M": 7, "N": 5120, "K": 5120, "out": "bf16"},
        # gate+up over a long prompt, activations in 4 bits too
        {"name": "linear4_gate_up_m4096", "op": "linear4", "M": 4096, "N": 34816, "K": 5120,
         "out": "bf16"},
        # the expert layer of one request's decode step
        {"name": "moe_t1", "op": "moe", "T": 1, "H": 5120, "I": 1280, "E": 64, "k": 6,
         "out": "bf16"},
        # the same over a drafted block of 16 tokens
        {"name": "moe_t16", "op": "moe", "T": 16, "H": 5120, "I": 1280, "E": 64, "k": 6,
         "out": "bf16"},
        # an odd batch over many narrow experts
        {"name": "moe_t61_odd", "op": "moe", "T": 61, "H": 2080, "I": 736, "E": 127, "k": 8,
         "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges: rows from one to a long prompt's, any
    number of weight rows, any K of whole blocks."""
    limit = max(work(c)["flops"] for c in listed())
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(("codec", "linear", "linear4", "moe"))
        if op == "codec":
            case = {"op": op, "R": _log(rng, 1, 8192), "K": BLOCK * _log(rng, 1, 544),
                    "dtype": rng.choice(("bf16", "f32"))}
        elif op == "moe":
            E = _log(rng, 4, 128)
            case = {"op": op, "T": _log(rng, 1, 128), "H": BLOCK * _log(rng, 4, 160),
                    "I": BLOCK * _log(rng, 2, 48), "E": E, "k": rng.randint(1, min(8, E)),
                    "out": rng.choice(("bf16", "f32"))}
        else:
            case = {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 1, 34816),
                    "K": BLOCK * _log(rng, 1, 544), "out": rng.choice(("bf16", "f32"))}
        w = work(case)
        if w["flops"] <= limit and w["bytes"] <= most:
            return case


def _stored(rows, K):
    """Bytes of rows x K values in MX4: 4 bits each and a scale byte a block."""
    return rows * (K // 2 + K // BLOCK)


def work(case):
    op = case["op"]
    if op == "codec":
        R, K = case["R"], case["K"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * R * K * size + _stored(R, K), "flops": 4 * R * K}
    size = 2 if case["out"] == "bf16" else 4
    if op == "moe":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        used = E * (1.0 - (1.0 - k / E) ** T)       # experts that some token chose
        stored = _stored(2 * I, H) + _stored(H, I)
        return {"bytes": int(used * stored) + T * (2 * H + size * H + 4 * E),
                "flops": 6 * T * k * H * I}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": _stored(N, K) + M * (2 * K + size * N), "flops": 2 * M * N * K}


# ---- plain form of the format -----------------------------------------------

def _encode(x):
    """(codes, exponents) of x [..., K] in 32 bits: per block of 32 the exponent
    floor(log2(largest magnitude)) - 2, at least -127, and per value the
    nearest code (ties to the even one; above 6 it saturates), with bit 3 the
    sign."""
    blocks = x.float().unflatten(-1, (-1, BLOCK))
    top = blocks.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(min=-127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    t = torch.ldexp(blocks.abs(), -e)
    code = torch.zeros(t.shape, dtype=torch.uint8, device=x.device)
    for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                     (3.5, True), (5.0, False)):
        code += (t >= edge) if up else (t > edge)
    code += torch.signbit(blocks).to(torch.uint8) * 8
    return code.flatten(-2), e.squeeze(-1)


def _decode(code, e, dtype=torch.float32):
    """The values of codes [..., K] under exponents [..., K / 32]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=dtype, device=code.device)
    v = grid[code.int()].unflatten(-1, (-1, BLOCK))
    return (v * torch.ldexp(torch.ones_like(e, dtype=dtype), e).unsqueeze(-1)).flatten(-2)


def _halves(code):
    """Two codes a byte, as a weight is kept."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _whole(packed):
    return torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)


# ---- inputs -------------------------------------------------------------------

def _normal(shape, sigma, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _weight(shape, seed):
    """A BF16 weight N(0, 0.02) of `shape`, its rows' sizes spread a little."""
    w = _normal(shape, 0.02, seed, torch.float32)
    w *= torch.exp(0.3 * _normal(shape[:-1] + (1,), 1.0, seed + 1, torch.float32))
    return w.to(torch.bfloat16)


def _raw_inputs(case, seed):
    op, base = case["op"], 1000003 * (seed + 1)
    if op == "codec":
        x = _normal((case["R"], case["K"]), 1.0, base, torch.float32)
        x *= torch.exp(_normal((1, case["K"]), 1.0, base + 1, torch.float32))
        return {"x": x.to(DTYPES[case["dtype"]])}
    if op == "moe":
        T, H, I, E = (case[n] for n in ("T", "H", "I", "E"))
        return {"x": _normal((T, H), 1.0, base, torch.bfloat16),
                "logits": _normal((T, E), 1.5, base + 1, torch.float32),
                "w13": [_weight((2 * I, H), base + 10 + 4 * e) for e in range(E)],
                "w2": [_weight((H, I), base + 12 + 4 * e) for e in range(E)]}
    return {"x": _normal((case["M"], case["K"]), 1.0, base, torch.bfloat16),
            "w": _weight((case["N"], case["K"]), base + 1)}


def _plain_weight(w):
    code, e = _encode(w)
    return _halves(code), e.to(torch.int16)


def prepare(case, seed):
    raw = _raw_inputs(case, seed)
    state = {"case": case, "x": raw["x"]}
    op = case["op"]
    if own and op != "codec":
        from lossless_bit_weight_amd import mx4
    if op in ("linear", "linear4"):
        state["w"] = mx4.mx4_quantize(raw["w"]) if own else _plain_weight(raw["w"])
    if op == "moe":
        state["logits"] = raw["logits"]
        for name in ("w13", "w2"):
            if own:
                state[name] = mx4.mx4_quantize(torch.stack(raw.pop(name)))
            else:
                state[name] = [_plain_weight(w) for w in raw.pop(name)]
    return state


# ---- one pass -------------------------------------------------------------------

def _choose(logits, k, dtype):
    """(experts, weights) [T, k]: the k largest logits of each token, ties to
    the lowest expert, and the softmax over them."""
    value, expert = torch.sort(logits.to(dtype), dim=-1, descending=True, stable=True)
    value, expert = value[:, :k], expert[:, :k]
    p = torch.exp(value - value[:, :1])
    return expert, p / p.sum(-1, keepdim=True)


def _silu_mul(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _run_plain(state):
    case, x = state["case"], state["x"]
    op = case["op"]
    if op == "codec":
        return _decode(*_encode(x)).to(x.dtype)
    if op == "moe":
        T, I = case["T"], case["I"]
        expert, p = _choose(state["logits"], case["k"], torch.float32)
        y = torch.zeros((T, case["H"]), device=x.device)
        xf = x.float()
        for e in torch.unique(expert).tolist():
            t, j = torch.nonzero(expert == e, as_tuple=True)
            code, ex = state["w13"][e]
            gu = xf[t] @ _decode(_whole(code), ex.int()).T
            h = _silu_mul(gu[:, :I], gu[:, I:])
            code, ex = state["w2"][e]
            y[t] += p[t, j].unsqueeze(-1) * (h @ _decode(_whole(code), ex.int()).T)
        return y.to(DTYPES[case["out"]])
    code, e = state["w"]
    xf = _decode(*_encode(x)) if op == "linear4" else x.float()
    return (xf @ _decode(_whole(code), e.int()).T).to(DTYPES[case["out"]])


def _run_own(state):
    from lossless_bit_weight_amd import mx4
    case, x = state["case"], state["x"]
    op = case["op"]
    if op == "codec":
        return mx4.mx4_dequantize(mx4.mx4_quantize(x), out_dtype=x.dtype)
    out = DTYPES[case["out"]]
    if op == "moe":
        return mx4.mx4_moe(x, state["logits"], state["w13"], state["w2"], case["k"],
                           out_dtype=out)
    if op == "linear4":
        x = mx4.mx4_quantize(x)
    return mx4.mx4_gemm(x, state["w"], out_dtype=out)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits ---------------------------------------------------

def _rounded(x):
    """x as MX4 holds it, in 64 bits: each block is divided by
    2^(floor(log2(largest magnitude)) - 2) and rounded to steps of 1/2 below
    2, 1 below 4 and 2 above, half to even, 6 at most."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    _, ex = torch.frexp(torch.where(top > 0, top, torch.full_like(top, 2.0 ** -125)))
    unit = torch.exp2((ex.double() - 3.0).clamp(min=-127.0))
    t = b.abs() / unit
    step = torch.where(t < 2.0, 0.5, torch.where(t < 4.0, 1.0, 2.0)).double()
    q = torch.round(t / step).mul_(step).clamp_(max=6.0)
    return torch.copysign(q * unit, b).flatten(-2)


def exact(case, seed):
    raw = _raw_inputs(case, seed)
    op, x = case["op"], raw["x"]
    if op == "codec":
        return _rounded(x)
    if op == "moe":
        I = case["I"]
        logits = raw["logits"].double()
        y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=x.device)
        order = torch.argsort(-logits, dim=-1, stable=True)[:, :case["k"]]
        p = torch.softmax(torch.gather(logits, 1, order), dim=-1)
        share = torch.zeros_like(logits).scatter_(1, order, p)
        for e in range(case["E"]):
            rows = [t for t, chosen in enumerate(order.tolist()) if e in chosen]
            if not rows:
                continue
            w13, w2 = _rounded(raw["w13"][e]), _rounded(raw["w2"][e])
            g = x[rows].double() @ w13[:I].T
            u = x[rows].double() @ w13[I:].T
            y[rows] += share[rows, e, None] * ((g * torch.sigmoid(g) * u) @ w2.T)
        return y
    xr = _rounded(x) if op == "linear4" else x.double()
    return xr @ _rounded(raw["w"]).T
