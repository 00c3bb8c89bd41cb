"""Routing to experts, and the expert layer on a given routing, against their
64-bit forms."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4
from tests import mx4_ref, step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _bf16(v):
    return mx4_ref.bf16_to_f64(mx4_ref.f64_to_bf16_bits(v))


def _dev(v, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).cuda().to(dtype)


def _logits(T, E, seed, dtype="f32", sigma=1.5):
    v = np.random.default_rng(seed).standard_normal((T, E)) * sigma
    return _bf16(v) if dtype == "bf16" else v.astype(np.float32).astype(np.float64)


def _check(l, k, dtype="f32", scores="softmax", bias=None, groups=1, kept=1, terms=1, renorm=True,
           scale=1.0):
    e, s = mx4.mx4_route(_dev(l, TYPES[dtype]), k, scores=scores,
                         bias=None if bias is None else _dev(bias), groups=groups,
                         kept_groups=kept, group_terms=terms, renormalize=renorm, scale=scale)
    we, ws = ref.route(l, k, scores, bias, groups, kept, terms, renorm, scale)
    assert np.array_equal(e.cpu().numpy(), we)
    got = s.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ws))
    # 64 bits rounded once to fp32 (the smallest to a subnormal)
    fin = ~np.isnan(ws)
    assert np.all(np.abs(got - ws)[fin] <= np.abs(ws[fin]) * 2.0 ** -24 * (1 + 1e-6) + 2.0 ** -150)
    return e, s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (16, 64, 6), (5, 65, 8), (3, 127, 32),
                                   (61, 128, 8), (7, 200, 9), (130, 256, 8), (2, 513, 32),
                                   (9, 1024, 32)])
def test_route(T, E, k, scores, dtype):
    l = _logits(T, E, T + E, dtype)
    bias = (0.2 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)
    _check(l, k, dtype, scores)
    _check(l, k, dtype, scores, renorm=False, scale=2.5)
    _check(l, k, dtype, scores, bias=bias, scale=0.5)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,kept", [(1, 8, 2, 4, 1), (33, 256, 8, 8, 4), (5, 126, 6, 7, 3),
                                               (4, 64, 4, 64, 9), (3, 1024, 32, 32, 2),
                                               (17, 160, 6, 5, 5), (9, 96, 32, 3, 1),
                                               (6, 40, 8, 20, 3), (2, 320, 8, 64, 63)])
def test_route_in_groups(T, E, k, groups, kept, scores):
    l = _logits(T, E, T * E + groups)
    bias = (0.2 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)
    for terms in (1, 2):
        for b in (None, bias):
            _check(l, k, "f32", scores, b, groups, kept, terms)


@pytest.mark.parametrize("E", [7, 64, 256, 1000])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest(E, scores):
    rng = np.random.default_rng(E)
    l = rng.choice([-1.0, 0.0, 1.0], (20, E))
    l[0] = 0.0
    l[1, ::2] = -0.0
    l[1, 1::2] = 0.0
    k = min(E, 8)
    _check(l, k, "f32", scores)
    _check(l, k, "bf16", scores)
    b = rng.choice([0.0, 0.5], E).astype(np.float32)
    _check(l, k, "f32", scores, b)
    if E % 8 == 0:
        for terms in (1, 2):
            _check(l, k, "f32", scores, None, 8, 3, terms)
            _check(l, k, "f32", scores, b, 8, 3, terms)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masked_experts(scores, renorm):
    """Logits and biases of -inf, down to tokens with none left and groups with one."""
    rng = np.random.default_rng(3)
    l = _logits(64, 48, 5)
    for t in range(64):
        l[t, rng.permutation(48)[:min(t, 48)]] = -np.inf
    b = (0.1 * rng.standard_normal(48)).astype(np.float32)
    _check(l, 8, "f32", scores, renorm=renorm)
    _check(l, 8, "f32", scores, b, renorm=renorm)
    b[10:20] = -np.inf
    for terms in (1, 2):
        _check(l, 8, "f32", scores, None, 12, 5, terms, renorm)
        _check(l, 8, "f32", scores, b, 12, 5, terms, renorm)
    _check(np.full((3, 48), -np.inf), 4, "f32", scores, renorm=renorm)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_nan_and_extremes(scores, renorm):
    l = _logits(12, 40, 7)
    l[0, 11] = np.nan
    l[1, [3, 30]] = np.nan
    l[2] = np.nan
    l[3] *= 1e30
    l[4] -= 1000.0
    l[5] += 1000.0
    l[6] = -3e38
    l[7] = 3e38
    l[8, 1:] = -2000.0
    l[9] = np.float32(1e-45)
    l = l.astype(np.float32).astype(np.float64)
    _check(l, 6, "f32", scores, renorm=renorm)
    b = np.linspace(-0.5, 0.5, 40).astype(np.float32)
    _check(l[[0, 1, 2, 3, 5, 9, 10]], 6, "f32", scores, b, renorm=renorm)
    b[5] = np.nan
    _check(l[9:], 6, "f32", scores, b, renorm=renorm)


def test_route_of_views_and_into_given_outputs():
    l = _logits(10, 32, 1)
    wide = torch.full((10, 45), 99.0, device="cuda")
    wide[:, 3:35] = _dev(l)
    e = torch.empty(10, 4, dtype=torch.int32, device="cuda")
    s = torch.empty(10, 4, device="cuda")
    got = mx4.mx4_route(wide[:, 3:35], 4, experts=e, shares=s)
    assert got[0] is e and got[1] is s
    we, ws = ref.route(l, 4)
    assert np.array_equal(e.cpu().numpy(), we)
    b = torch.full((10, 45), 99.0, device="cuda", dtype=torch.bfloat16)
    b[:, 3:35] = _dev(_bf16(l), torch.bfloat16)
    assert np.array_equal(mx4.mx4_route(b[:, 3:35], 4)[0].cpu().numpy(), ref.route(_bf16(l), 4)[0])


def test_route_of_many_tokens():
    """More tokens than any grid of workgroups side by side."""
    T = 100003
    l = torch.from_numpy(np.random.default_rng(1).standard_normal((T, 16)).astype(np.float32)).cuda()
    e, s = mx4.mx4_route(l, 2)
    value, want = torch.sort(l, dim=-1, descending=True, stable=True)
    assert torch.equal(e.long(), want[:, :2])
    p = torch.softmax(value[:, :2].double(), -1).float()
    assert torch.equal(s, p) or float((s - p).abs().max()) <= 2.0 ** -24


# ---- the layer on a given routing ---------------------------------------------------------

def _layer(T, H, I, E, seed):
    rng = np.random.default_rng(seed)
    x = _bf16(rng.standard_normal((T, H)))
    w13, w2 = (_bf16(0.05 * rng.standard_normal(s)) for s in ((E, 2 * I, H), (E, H, I)))
    dev = torch.bfloat16
    return (x, mx4_ref.rounded(w13), mx4_ref.rounded(w2), _dev(x, dev),
            mx4.mx4_quantize(_dev(w13, dev)), mx4.mx4_quantize(_dev(w2, dev)))


def _layer_ref(x, experts, shares, w13, w2):
    """(y, bound) as tests/mx4_ref.py's expert layer, on a given routing."""
    T, H = x.shape
    I, E = w2.shape[2], len(w2)
    y, tol = np.zeros((T, H)), np.full((T, H), 1e-37)
    for t in range(T):
        for e, p in zip(experts[t], shares[t].astype(np.float64)):
            if not 0 <= e < E:
                continue
            gu, d = mx4_ref.matmul(x[t:t + 1], w13[e])
            g, u, dg, du = gu[0, :I], gu[0, I:], d[0, :I], d[0, I:]
            silu = g / (1 + np.exp(-g))
            h = silu * u
            dh = (1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du
                  + np.abs(h) * ((8 + np.abs(g)) * 2.0 ** -23 + 2.0 ** -24))
            o, do = mx4_ref.matmul(h[None], w2[e])
            y[t] += p * o[0]
            rel = (4 + len(experts[t])) * 2.0 ** -23
            tol[t] += np.abs(p) * (do[0] * 3 + dh @ np.abs(w2[e]).T
                                   + rel * (np.abs(h) @ np.abs(w2[e]).T))
    return y, tol


# one token; tokens one by one; slots of up to four and up to sixteen rows, one workgroup
# that chooses for 16 tokens and above; more experts than pairs
ROUTED = [(1, 160, 96, 9, 4), (1, 64, 32, 3, 3), (3, 96, 64, 20, 2), (16, 128, 96, 5, 3),
          (17, 64, 64, 130, 4), (61, 96, 160, 12, 8), (128, 64, 96, 4, 4), (40, 1056, 288, 2, 1)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,E,k", ROUTED)
def test_layer_on_a_routing(T, H, I, E, k, out):
    x, w13, w2, xd, w13q, w2q = _layer(T, H, I, E, T + H)
    rng = np.random.default_rng(T)
    experts = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    shares = rng.standard_normal((T, k)).astype(np.float32)     # of any sign and sum
    y = mx4.mx4_moe_routed(xd, torch.from_numpy(experts).cuda(), torch.from_numpy(shares).cuda(),
                           w13q, w2q, TYPES[out])
    want, tol = _layer_ref(x, experts, shares, w13, w2)
    mx4_ref.assert_close(y.float().cpu().numpy(), want, tol, out, "routed layer")


@pytest.mark.parametrize("T,H,I,E,k", [(1, 96, 64, 6, 5), (4, 96, 64, 6, 5), (30, 96, 64, 6, 5),
                                       (100, 64, 32, 9, 4)])
def test_layer_skips_and_repeats_entries(T, H, I, E, k):
    """-1 anywhere, numbers far outside, one expert twice with both shares, a token with
    none; a NaN share reaches its token alone."""
    x, w13, w2, xd, w13q, w2q = _layer(T, H, I, E, 3 * T)
    rng = np.random.default_rng(T)
    experts = rng.integers(-1, E, (T, k)).astype(np.int32)
    experts[0, 0] = -1
    experts[-1, k - 1] = 2 ** 31 - 1
    experts[T // 2] = experts[T // 2, 1] if T > 1 else 3
    if T > 3:
        experts[2] = -1
        experts[3, :2] = (-2 ** 31, E)
    shares = rng.standard_normal((T, k)).astype(np.float32)
    if T > 3:
        experts[1, 1] = 0
        shares[1, 1] = np.nan
    shares[experts < 0] = np.nan                # counts for nothing
    y = mx4.mx4_moe_routed(xd, torch.from_numpy(experts).cuda(), torch.from_numpy(shares).cuda(),
                           w13q, w2q, torch.float32)
    want, tol = _layer_ref(x, experts, shares, w13, w2)
    mx4_ref.assert_close(y.cpu().numpy(), want, tol, "f32", "routed layer")
    if T > 3:
        assert bool((y[2] == 0).all()) and bool(y[1].isnan().all())


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 160, 96, 9, 4), (2, 64, 32, 70, 3), (16, 96, 64, 12, 5),
                                       (90, 64, 96, 5, 5)])
def test_layer_on_softmax_routing_is_the_layer_on_logits(T, H, I, E, k, renorm):
    """The same experts, and shares that the two differ in by fp32 roundings."""
    x, w13, w2, xd, w13q, w2q = _layer(T, H, I, E, T + E)
    l = _dev(_logits(T, E, T))
    a = mx4.mx4_moe(xd, l, w13q, w2q, k, renormalize=renorm, out_dtype=torch.float32)
    b = mx4.mx4_moe_routed(xd, *mx4.mx4_route(l, k, renormalize=renorm), w13q, w2q, torch.float32)
    e, s = (t.cpu().numpy() for t in mx4.mx4_route(l, k, renormalize=renorm))
    # of each share at most (16 + |l - top| + k) steps of 2^-23, twice
    rel = 2 * (16 + 12 + k) * 2.0 ** -23
    _, tol = _layer_ref(x, e, s, w13, w2)
    size = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            gu = x[t] @ w13[e[t, j]].T
            h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            size[t] += np.abs(s[t, j]) * (np.abs(h) @ np.abs(w2[e[t, j]]).T)
    d = (a - b).abs().cpu().numpy()
    assert np.all(d <= rel * size + 2 * tol)
