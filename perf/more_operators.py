"""Measured cases of what stands between the products of a decoder's verify
step: the residual's addition with the root-mean-square norm and its output in
8 bits, the product of such 8-bit activations with 4-bit weights, the routing
of tokens to experts and the expert layer on a given routing, and the
verification of drafted tokens.

A case names its operator in "op":

  norm     s = x + residual, rounded to the residual's type;
           y = s / sqrt(mean(s^2) + eps) * weight, in BF16, fp32 or MX8 (blocks
           of 32 along K under a shared power of two: E4M3 values, multiples of 1/4)
  linear8  y = x W^T, W [N, K] in MX4, x [M, K] BF16 quantised to MX8 within the
           pass
  route    a token's experts (the top_k of its scores plus a bias, from the kept
           groups of experts) and their shares
  experts  route, and then y[t] = sum over t's experts e of
           share[t, e] W2[e] (silu(G[e] x[t]) * U[e] x[t]), W13[e] = [G[e]; U[e]]
  verify   the drafted tokens of a sequence that the target's probabilities
           accept, and the token drawn behind them, from given random numbers

Each has its plain form (elementary torch operations), the calls a program
makes of the library (`own`), and the definition in 64 bits (`exact`).
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32                      # values that share one scale
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # magnitudes of a 4-bit code


def listed():
    return [
        # before the QKV product of one request's decode step: latency only
        {"name": "norm_one_token", "op": "norm", "M": 1, "K": 5120, "x": "bf16", "res": "bf16",
         "w": "bf16", "out": "mx8"},
        # before the gate+up product of a prompt, the branch's output in fp32
        {"name": "norm_prompt", "op": "norm", "M": 4096, "K": 5120, "x": "f32", "res": "bf16",
         "w": "bf16", "out": "mx8"},
        # every head's query of an odd batch, no residual
        {"name": "norm_heads", "op": "norm", "M": 40 * 517, "K": 128, "x": "bf16", "res": "none",
         "w": "f32", "out": "bf16"},
        # QKV of one request's decode step
        {"name": "linear8_qkv_m1", "op": "linear8", "M": 1, "N": 7168, "K": 5120, "out": "bf16"},
        # a down projection with ragged rows, an odd batch, fp32 out
        {"name": "linear8_down_m33", "op": "linear8", "M": 33, "N": 5003, "K": 17376,
         "out": "f32"},
        # gate+up over a long prompt
        {"name": "linear8_gate_up_m4096", "op": "linear8", "M": 4096, "N": 34816, "K": 5120,
         "out": "bf16"},
        # the routing of a drafted block of 16 tokens: latency only
        {"name": "route_block", "op": "route", "T": 16, "E": 64, "k": 6, "scores": "softmax",
         "bias": False, "groups": 1, "kept": 1, "terms": 1, "renorm": True, "logits": "f32"},
        # the routing of a long prompt, balanced by a bias and limited to groups
        {"name": "route_prompt", "op": "route", "T": 8191, "E": 256, "k": 8, "scores": "sigmoid",
         "bias": True, "groups": 8, "kept": 4, "terms": 2, "renorm": True, "logits": "f32"},
        # the expert layer over a drafted block of 16 tokens
        {"name": "experts_block", "op": "experts", "T": 16, "H": 5120, "I": 1280, "E": 64, "k": 6,
         "scores": "sigmoid", "bias": True, "groups": 1, "kept": 1, "terms": 1, "renorm": True,
         "logits": "f32", "out": "bf16"},
        # an odd batch over many narrow experts in groups
        {"name": "experts_odd", "op": "experts", "T": 61, "H": 2080, "I": 736, "E": 126, "k": 8,
         "scores": "softmax", "bias": False, "groups": 7, "kept": 3, "terms": 1, "renorm": False,
         "logits": "bf16", "out": "bf16"},
        # one request, four tokens drafted without probabilities, an odd vocabulary
        {"name": "verify_one", "op": "verify", "B": 1, "D": 4, "V": 32003, "logits": "bf16",
         "probs": "none"},
        # a batch of drafted blocks of 15 with their drafter's probabilities
        {"name": "verify_batch", "op": "verify", "B": 32, "D": 15, "V": 129280, "logits": "f32",
         "probs": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_route(rng, most_experts):
    groups = rng.choice((1, 1, rng.randint(2, 8)))
    per = _log(rng, 4 if groups == 1 else 2, most_experts // groups)
    kept = rng.randint(1, groups)
    return {"E": groups * per, "k": rng.randint(1, min(8, kept * per)),
            "scores": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5,
            "groups": groups, "kept": kept, "terms": rng.choice((1, 2)),
            "renorm": rng.random() < 0.7, "logits": rng.choice(("f32", "f32", "bf16"))}


def draw(rng):
    """One more case of the same ranges: rows from one to a long prompt's, any K
    of whole blocks, any number of weight rows, of experts and of words."""
    limit = max(work(c)["flops"] for c in listed())
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(("norm", "linear8", "route", "experts", "verify"))
        if op == "norm":
            case = {"op": op, "M": _log(rng, 1, 8192), "K": BLOCK * _log(rng, 1, 544),
                    "x": rng.choice(("bf16", "f32")), "res": rng.choice(("none", "bf16", "f32")),
                    "w": rng.choice(("bf16", "f32")), "out": rng.choice(("bf16", "f32", "mx8"))}
        elif op == "linear8":
            case = {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 1, 34816),
                    "K": BLOCK * _log(rng, 1, 544), "out": rng.choice(("bf16", "f32"))}
        elif op == "route":
            case = {"op": op, "T": _log(rng, 1, 16384), **_draw_route(rng, 512)}
        elif op == "experts":
            case = {"op": op, "T": _log(rng, 1, 128), "H": BLOCK * _log(rng, 4, 160),
                    "I": BLOCK * _log(rng, 2, 48), **_draw_route(rng, 128),
                    "out": rng.choice(("bf16", "f32"))}
        else:
            case = {"op": op, "B": _log(rng, 1, 64), "D": rng.randint(0, 16),
                    "V": _log(rng, 100, 160000), "logits": rng.choice(("bf16", "f32")),
                    "probs": rng.choice(("none", "bf16", "f32"))}
        w = work(case)
        if w["flops"] <= limit and w["bytes"] <= most:
            return case


def _stored(rows, K):
    """Bytes of rows x K values in MX4: 4 bits each and a scale byte a block."""
    return rows * (K // 2 + K // BLOCK)


def _size(name):
    return {"none": 0, "bf16": 2, "f32": 4}[name]


def work(case):
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        y = 1 + 1 / BLOCK if case["out"] == "mx8" else _size(case["out"])
        return {"bytes": int(M * K * (_size(case["x"]) + 2 * _size(case["res"]) + y)
                             + K * _size(case["w"])), "flops": 6 * M * K}
    if op == "linear8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _stored(N, K) + M * (2 * K + _size(case["out"]) * N),
                "flops": 2 * M * N * K}
    if op == "verify":
        rows, V = case["B"] * (case["D"] + 1), case["V"]
        return {"bytes": rows * V * _size(case["logits"])
                + case["B"] * (case["D"] > 0) * V * _size(case["probs"]) + rows * 16,
                "flops": 4 * rows * V}
    T, E, k = case["T"], case["E"], case["k"]
    chosen = {"bytes": T * E * _size(case["logits"]) + 8 * T * k + 4 * E, "flops": 8 * T * E}
    if op == "route":
        return chosen
    H, I = case["H"], case["I"]
    used = E * (1.0 - (1.0 - k / E) ** T)       # experts that some token chose
    return {"bytes": chosen["bytes"] + T * H * (2 + _size(case["out"]))
            + int(used * (_stored(2 * I, H) + _stored(H, I))),
            "flops": chosen["flops"] + 6 * T * k * H * I}


# ---- plain form of the formats -----------------------------------------------

def _exponents(blocks, top_exponent):
    """floor(log2(largest magnitude)) - top_exponent of blocks [..., 32], at
    least -127."""
    top = blocks.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 1 - top_exponent).clamp(min=-127)
    return torch.where(top == 0, torch.full_like(e, -127), e)


def _encode(x):
    """(4-bit codes, exponents) of x [..., K] in 32 bits: per block of 32 the
    exponent, and per value the nearest code (ties to the even one; above 6 it
    saturates), with bit 3 the sign."""
    blocks = x.float().unflatten(-1, (-1, BLOCK))
    e = _exponents(blocks, 2)
    t = torch.ldexp(blocks.abs(), -e)
    code = torch.zeros(t.shape, dtype=torch.uint8, device=x.device)
    code = code + (t > 0.25) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) \
        + (t > 5.0)
    code = code + torch.signbit(blocks).to(torch.uint8) * 8
    return code.to(torch.uint8).flatten(-2), e.squeeze(-1)


def _decode(code, e):
    """The values of codes [..., K] under exponents [..., K / 32]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=code.device)
    v = grid[code.int()].unflatten(-1, (-1, BLOCK))
    return (v * torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).unsqueeze(-1)).flatten(-2)


def _halves(code):
    """Two codes a byte, as a weight is kept."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _whole(packed):
    return torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)


def _mx8(x):
    """The values that MX8 holds for x [..., K], in 32 bits: per block of 32 the
    exponent e of its unit, and per value the nearest multiple (ties to even) of
    its binade's step, an eighth of the binade and at least 1/4; 448 at most."""
    blocks = x.float().unflatten(-1, (-1, BLOCK))
    e = _exponents(blocks, 8)
    t = torch.ldexp(blocks.abs(), -e)
    step = (torch.frexp(t).exponent - 4).clamp(min=-2)
    q = torch.ldexp(torch.round(torch.ldexp(t, -step)), step).clamp(max=448.0)
    return torch.copysign(torch.ldexp(q, e), blocks).flatten(-2)


# ---- inputs -------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, sigma, seed, dtype):
    return (torch.randn(shape, generator=_generator(seed), device="cuda") * sigma).to(dtype)


def _uniform(shape, seed):
    return torch.rand(shape, generator=_generator(seed), device="cuda")


def _weight(shape, seed):
    """A BF16 weight N(0, 0.02) of `shape`, its rows' sizes spread a little."""
    w = _normal(shape, 0.02, seed, torch.float32)
    w *= torch.exp(0.3 * _normal(shape[:-1] + (1,), 1.0, seed + 1, torch.float32))
    return w.to(torch.bfloat16)


def _block_inputs(case, seed):
    """What a block of a decoder has in hand: activations whose columns differ in
    size, weights, a router's logits."""
    op, base = case["op"], 1000003 * (seed + 1)
    if op == "norm":
        M, K = case["M"], case["K"]
        spread = torch.exp(_normal((1, K), 0.7, base, torch.float32))
        x = (_normal((M, K), 1.0, base + 1, torch.float32) * spread).to(DTYPES[case["x"]])
        raw = {"x": x, "w": (1.0 + _normal((K,), 0.2, base + 2, torch.float32)
                             ).to(DTYPES[case["w"]]), "res": None}
        if case["res"] != "none":
            raw["res"] = (_normal((M, K), 3.0, base + 4, torch.float32) * spread
                          ).to(DTYPES[case["res"]])
        return raw
    if op == "linear8":
        return {"x": _normal((case["M"], case["K"]), 1.0, base, torch.bfloat16),
                "w": _weight((case["N"], case["K"]), base + 1)}
    T, E = case["T"], case["E"]
    raw = {"logits": _normal((T, E), 1.5, base + 1, DTYPES[case["logits"]]),
           "bias": _normal((E,), 0.1, base + 2, torch.float32) if case["bias"] else None}
    if op == "experts":
        H, I = case["H"], case["I"]
        raw["x"] = _normal((T, H), 1.0, base, torch.bfloat16)
        raw["w13"] = [_weight((2 * I, H), base + 10 + 4 * e) for e in range(E)]
        raw["w2"] = [_weight((H, I), base + 12 + 4 * e) for e in range(E)]
    return raw


def _verify_inputs(case, seed):
    """A target's logits, drafts that a nearby distribution gave (or, without
    probabilities, the target's own likely words), one temperature a sequence,
    some of them 0, and sequences that drafted fewer tokens than D."""
    B, D, V = case["B"], case["D"], case["V"]
    base = 1000003 * (seed + 1)
    logits = _normal((B, D + 1, V), 2.5, base, torch.float32)
    temperature = 0.5 + _uniform((B,), base + 1)
    greedy = _uniform((B,), base + 2) < 0.25
    guess = logits[:, :D] + _normal((B, D, V), 0.4, base + 3, torch.float32)
    gumbel = -torch.log(-torch.log(_uniform((B, D, V), base + 4).clamp(1e-20, 1 - 1e-7)))
    probs = None
    if case["probs"] != "none":
        guess /= temperature[:, None, None]
        probs = torch.softmax(guess, dim=-1).to(DTYPES[case["probs"]])
        drafts = (guess + gumbel).argmax(-1)
    else:
        drafts = (2.0 * guess + 0.3 * gumbel).argmax(-1)
    least = max(0, D // 2)
    lengths = torch.randint(least, D + 1, (B,), generator=_generator(base + 5), device="cuda")
    lengths[0] = D
    return {"logits": logits.to(DTYPES[case["logits"]]), "probs": probs,
            "drafts": drafts.to(torch.int32), "lengths": lengths.to(torch.int32),
            "temperature": torch.where(greedy, torch.zeros_like(temperature), temperature),
            "uniforms": _uniform((B, D + 1), base + 6)}


def _raw_inputs(case, seed):
    return _verify_inputs(case, seed) if case["op"] == "verify" else _block_inputs(case, seed)


def _plain_weight(w):
    code, e = _encode(w)
    return _halves(code), e.to(torch.int16)


def prepare(case, seed):
    state = _raw_inputs(case, seed)
    state["case"] = case
    if own:
        from lossless_bit_weight_amd import mx4
    if case["op"] == "linear8":
        state["w"] = mx4.mx4_quantize(state["w"]) if own else _plain_weight(state["w"])
    if case["op"] == "experts":
        for name in ("w13", "w2"):
            if own:
                state[name] = mx4.mx4_quantize(torch.stack(state[name]))
            else:
                parts = [_plain_weight(w) for w in state[name]]
                state[name] = tuple(torch.stack(p) for p in zip(*parts))
    return state


# ---- one pass -------------------------------------------------------------------

def _norm_plain(state):
    case, x, res = state["case"], state["x"].float(), state["res"]
    if res is not None:
        res = (x + res.float()).to(res.dtype)
        x = res.float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * state["w"].float()
    y = _mx8(y).to(torch.bfloat16) if case["out"] == "mx8" else y.to(DTYPES[case["out"]])
    return [y] if res is None else [y, res]


def _scores(logits, kind):
    """Scores in 64 bits, so that a choice between near ones depends on no
    rounding."""
    l = logits.double()
    if kind == "sigmoid":
        return l, 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(-1, keepdim=True))
    return l, p / p.sum(-1, keepdim=True)


def _route_plain(state):
    case = state["case"]
    l, s = _scores(state["logits"], case["scores"])
    biased = s if state["bias"] is None else s + state["bias"].double()
    key = l if state["bias"] is None else biased
    if case["groups"] > 1:
        G, kept = case["groups"], case["kept"]
        if case["terms"] == 1:
            group = key.unflatten(-1, (G, -1)).amax(-1)
        else:
            two = torch.sort(biased.unflatten(-1, (G, -1)), dim=-1, descending=True).values
            group = two[..., :2].sum(-1)
        order = torch.sort(group, dim=-1, descending=True, stable=True).indices
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, order[:, :kept], True)
        key = key.unflatten(-1, (G, -1)).masked_fill(~keep.unsqueeze(-1), -math.inf).flatten(-2)
    expert = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
    share = torch.gather(s, 1, expert)
    if case["renorm"]:
        share = share / share.sum(-1, keepdim=True)
    return expert.to(torch.int32), share.float()


def _experts_plain(state):
    """Every expert on every token, weighted by its share of the token (0 where it
    is none of the token's)."""
    case, x = state["case"], state["x"].float()
    T, H, I, E = (case[n] for n in ("T", "H", "I", "E"))
    expert, share = _route_plain(state)
    table = torch.zeros((T, E), device=x.device).scatter_(1, expert.long(), share)
    code, e = state["w13"]
    gu = (x @ _decode(_whole(code), e.int()).view(E * 2 * I, H).T).view(T, E, 2 * I)
    g, u = gu[..., :I], gu[..., I:]
    h = g / (1.0 + torch.exp(-g)) * u * table.unsqueeze(-1)
    code, e = state["w2"]
    w2 = _decode(_whole(code), e.int()).transpose(1, 2).reshape(E * I, H)
    return [(h.reshape(T, E * I) @ w2).to(DTYPES[case["out"]]), expert, share]


def _verify_plain(state):
    """Probabilities and their running sums in 64 bits: a random number next to a
    word's border has to fall on the same side of it."""
    logits, drafts, u = state["logits"], state["drafts"].long(), state["uniforms"].double()
    B, rows, V = logits.shape
    D = rows - 1
    l, tau = logits.double(), state["temperature"].double()
    greedy = (tau <= 0)[:, None]
    best = logits.float().argmax(-1)
    p = torch.exp((l - l.amax(-1, keepdim=True)) / torch.where(greedy, 1.0, tau[:, None])[..., None])
    p = p / p.sum(-1, keepdim=True)
    places = torch.arange(rows, device=l.device)
    px = torch.gather(p[:, :D], 2, drafts[..., None])[..., 0]
    if state["probs"] is None:
        q = torch.zeros((B, D, V), dtype=torch.float64, device=l.device)
        q = q.scatter_(2, drafts[..., None], 1.0)
    else:
        q = state["probs"].double()
    qx = torch.gather(q, 2, drafts[..., None])[..., 0]
    ok = torch.where(greedy, drafts == best[:, :D], u[:, :D] * qx < px)
    ok = ok & (places[:D] < state["lengths"][:, None])
    n = ok.long().cumprod(-1).sum(-1)
    # what is drawn behind the accepted tokens: the target's probabilities there,
    # less the drafter's of the place where it was refused
    at = torch.arange(B, device=l.device)
    last = p[at, n]
    q = torch.cat((q, torch.zeros((B, 1, V), dtype=torch.float64, device=l.device)), 1)
    rest = (last - q[at, n] * (n < state["lengths"])[:, None]).clamp(min=0.0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, last)
    total = rest.cumsum(-1)
    hit = (total > (u[:, D] * total[:, -1])[:, None]) & (rest > 0)
    final = V - 1 - (rest > 0).flip(-1).long().argmax(-1)
    token = torch.where(hit.any(-1), hit.long().argmax(-1), final)
    token = torch.where(greedy[:, 0], best[at, n], token)[:, None]
    tokens = torch.cat((drafts, token), 1)
    tokens = torch.where(places == n[:, None], token, tokens)
    tokens = torch.where(places > n[:, None], -1, tokens)
    return [tokens.to(torch.int32), n.to(torch.int32)]


def _run_plain(state):
    op = state["case"]["op"]
    if op == "linear8":
        code, e = state["w"]
        y = _mx8(state["x"]) @ _decode(_whole(code), e.int()).T
        return y.to(DTYPES[state["case"]["out"]])
    if op == "route":
        return list(_route_plain(state))
    return {"norm": _norm_plain, "experts": _experts_plain, "verify": _verify_plain}[op](state)


def _run_own(state):
    from lossless_bit_weight_amd import draft, mx4, mx8
    case = state["case"]
    op = case["op"]
    if op == "norm":
        out = mx8.VALUES if case["out"] == "mx8" else DTYPES[case["out"]]
        y = mx8.mx8_rms_norm(state["x"], state["w"], EPS, residual=state["res"], out_dtype=out)
        y, res = y if state["res"] is not None else (y, None)
        if case["out"] == "mx8":
            y = mx8.mx8_dequantize(y, torch.bfloat16)
        return [y] if res is None else [y, res]
    if op == "linear8":
        return mx8.mx8_gemm(mx8.mx8_quantize(state["x"]), state["w"], DTYPES[case["out"]])
    if op == "verify":
        return list(draft.draft_verify(state["logits"], state["drafts"], state["uniforms"],
                                       draft_probs=state["probs"], lengths=state["lengths"],
                                       temperature=state["temperature"]))
    expert, share = mx4.mx4_route(
        state["logits"], case["k"], scores=case["scores"], bias=state["bias"],
        groups=case["groups"], kept_groups=case["kept"], group_terms=case["terms"],
        renormalize=case["renorm"])
    if op == "route":
        return [expert, share]
    y = mx4.mx4_moe_routed(state["x"], expert, share, state["w13"], state["w2"],
                           out_dtype=DTYPES[case["out"]])
    return [y, expert, share]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits ---------------------------------------------------

def _held(x, top, steps):
    """x as a block format holds it, in 64 bits: `top` is the exponent of the
    format's largest binade, `steps` its steps a binade; the smallest binade
    that has its own step starts at 2^low, and what lies past the largest value
    becomes it."""
    low, most = {2: (0, 6.0), 8: (1, 448.0)}[top]
    b = x.double().unflatten(-1, (-1, BLOCK))
    big = b.abs().amax(-1, keepdim=True)
    whole = torch.floor(torch.log2(torch.where(big > 0, big, torch.full_like(big, 2.0 ** -126))))
    whole = whole - (torch.exp2(whole) > big).double() + (torch.exp2(whole + 1) <= big).double()
    unit = torch.exp2((whole - top).clamp(min=-127.0))
    t = b.abs() / unit
    binade = torch.floor(torch.log2(t.clamp(min=2.0 ** low))).clamp(min=float(low))
    binade = binade - (torch.exp2(binade) > t.clamp(min=2.0 ** low)).double()
    step = torch.exp2(binade) / steps
    return torch.copysign((torch.round(t / step) * step).clamp(max=most) * unit, b).flatten(-2)


def _exact_route(case, raw):
    logits = raw["logits"].double()
    s = torch.sigmoid(logits) if case["scores"] == "sigmoid" else torch.softmax(logits, -1)
    rank = logits if raw["bias"] is None else s + raw["bias"].double()
    if case["groups"] > 1:
        per = case["E"] // case["groups"]
        by = rank if case["terms"] == 1 else (s if raw["bias"] is None else rank)
        value = by.view(-1, case["groups"], per).topk(min(case["terms"], per), -1).values.sum(-1)
        order = torch.argsort(-value, dim=-1, stable=True)
        out = torch.ones_like(value).scatter_(1, order[:, :case["kept"]], 0.0)
        rank = rank.masked_fill(out.repeat_interleave(per, 1) > 0, -math.inf)
    expert = torch.argsort(-rank, dim=-1, stable=True)[:, :case["k"]]
    share = s.gather(1, expert)
    if case["renorm"]:
        share = share / share.sum(-1, keepdim=True)
    return expert.to(torch.int32), share


def _exact_verify(raw):
    """Sequence by sequence."""
    tokens = torch.full(raw["uniforms"].shape, -1, dtype=torch.int32)
    lengths, tau = raw["lengths"].tolist(), raw["temperature"].tolist()
    drafts, numbers = raw["drafts"].tolist(), raw["uniforms"].tolist()
    accepted = torch.zeros(len(lengths), dtype=torch.int32)
    for b, words in enumerate(drafts):
        for i in range(lengths[b] + 1):
            l = raw["logits"][b, i].double()
            refused = None
            if tau[b] <= 0:
                token = int(torch.nonzero(l == l.max())[0])
                if i < lengths[b] and words[i] == token:
                    tokens[b, i] = token
                    continue
            else:
                p = torch.softmax(l / tau[b], -1)
                if i < lengths[b]:
                    refused = torch.zeros_like(p)
                    if raw["probs"] is None:
                        refused[words[i]] = 1.0
                    else:
                        refused = raw["probs"][b, i].double()
                    if numbers[b][i] * float(refused[words[i]]) < float(p[words[i]]):
                        tokens[b, i] = words[i]
                        continue
                left = p if refused is None else (p - refused).clamp(min=0.0)
                left = left if float(left.sum()) > 0 else p
                below = left.cumsum(-1)
                found = torch.nonzero((below > numbers[b][-1] * below[-1]) & (left > 0))
                token = int(found[0] if len(found) else torch.nonzero(left > 0)[-1])
            tokens[b, i] = token
            accepted[b] = i
            break
    return [tokens, accepted]


def exact(case, seed):
    raw = _raw_inputs(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(raw)
    if op == "norm":
        x, res = raw["x"].double(), raw["res"]
        if res is not None:
            res = (raw["x"].float() + res.float()).to(res.dtype).double()
            x = res
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * raw["w"].double()
        if case["out"] == "mx8":
            y = _held(y, 8, 8)
        return [y] if res is None else [y, res]
    if op == "linear8":
        return _held(raw["x"], 8, 8) @ _held(raw["w"], 2, 2).T
    expert, share = _exact_route(case, raw)
    if op == "route":
        return [expert, share]
    x, I = raw["x"].double(), case["I"]
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        t, j = torch.nonzero(expert == e, as_tuple=True)
        if len(t):
            w13 = _held(raw["w13"][e], 2, 2)
            g, u = x[t] @ w13[:I].T, x[t] @ w13[I:].T
            h = g * torch.sigmoid(g) * u
            y[t] += share[t, j, None] * (h @ _held(raw["w2"][e], 2, 2).T)
    return [y, expert, share]
