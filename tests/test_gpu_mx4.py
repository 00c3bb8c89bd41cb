"""MX4 operators on the GPU against the 64-bit reference (mx4_ref): the codec bit
for bit, products and the expert layer within the error of fp32 sums."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4, w12
from tests import mx4_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _values(shape, seed, sigma=1.0):
    """BF16-exact normal values in float64, rows of different sizes."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape) * sigma * np.exp(0.5 * rng.standard_normal(shape[:-1] + (1,)))
    return ref.bf16_to_f64(ref.f64_to_bf16_bits(v))


def _dev(v, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).cuda().to(dtype)


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check_container(q, code, e):
    if code.ndim == 2:
        code, e = code[None], e[None]
    codes, scales = ref.container(code, e)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales)


# ---- codec -------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 32), (1, 5120), (3, 96), (16, 128), (17, 160), (33, 512),
                                   (70, 544), (2, 5, 64), (3, 17, 1056)])
def test_codec(shape, dtype):
    v = _values(shape, sum(shape))
    v.flat[::37] = 0.0
    q = mx4.mx4_quantize(_dev(v, TYPES[dtype]))
    assert q.shape == shape
    assert q.codes.numel() == mx4.mx4_codes_bytes(q.batch or 1, q.R, q.K)
    assert q.scales.numel() == mx4.mx4_scales_bytes(q.batch or 1, q.R, q.K)
    code, e = ref.encode(v)
    _check_container(q, code, e)
    want = ref.decode(code, e)
    for out in ("bf16", "f32"):
        y = mx4.mx4_dequantize(q, out_dtype=TYPES[out])
        assert y.dtype == TYPES[out] and tuple(y.shape) == shape
        assert np.array_equal(_host(y), want)


def test_codec_every_bf16_value():
    """All 65536 patterns, each among neighbours of every size from its own up."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    rng = np.random.default_rng(5)
    rows = [bits, rng.permutation(bits), rng.permutation(bits)]
    # each value under a leader up to eight binades larger, finite blocks only
    lead = np.minimum((bits & 0x7F80).astype(int) + (rng.integers(0, 9, 65536) << 7), 0x7F00)
    for s in range(0, 65536, 2):
        bits_pair = bits[s:s + 2]
        if s == 0:
            blocks = []
        b = np.zeros(32, np.uint16)
        b[0], b[1:3] = lead[s], bits_pair
        blocks.append(b)
    rows.append(np.concatenate(blocks))
    for r in rows:
        x = r.reshape(-1, 512)
        code, e = ref.encode(ref.bf16_to_f64(x))
        q = mx4.mx4_quantize(torch.from_numpy(x.view(np.int16).copy()).cuda())
        _check_container(q, code, e)
        want = ref.decode(code, e)
        assert np.array_equal(_host(mx4.mx4_dequantize(q, torch.float32)), want, equal_nan=True)
        assert np.array_equal(_host(mx4.mx4_dequantize(q)), want, equal_nan=True)


def test_codec_fp32_patterns():
    """Random fp32 patterns (subnormals, infinities and NaN among them), values a
    last place beside every rounding edge, and negative zeros."""
    rng = np.random.default_rng(6)
    raw = rng.integers(0, 1 << 32, (64, 1024), dtype=np.uint64).astype(np.uint32)
    same = (rng.integers(0, 255, (64, 32, 1)).astype(np.uint32) << 23)
    near = (same + rng.integers(0, 1 << 23, (64, 32, 32)).astype(np.uint32)
            - (rng.integers(0, 4, (64, 32, 32)).astype(np.uint32) << 23)) & np.uint32(0x7FFFFFFF)
    near = np.where(near >= 0x7F800000, 0, near).astype(np.uint32).reshape(64, 1024)
    edges = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    e32 = np.concatenate([edges, np.nextafter(edges, np.float32(0)),
                          np.nextafter(edges, np.float32(9)), [np.float32(-0.0)]])
    blocks = np.zeros((64, 32, 32), np.float32)
    blocks[..., 0] = 4.5
    blocks[..., 1:1 + e32.size] = e32
    blocks *= np.ldexp(np.float32(1), rng.integers(-120, 120, (64, 32, 1))).astype(np.float32)
    sub = rng.integers(0, 1 << 24, (64, 1024)).astype(np.uint32)
    for u in (raw, near, blocks.reshape(64, 1024).view(np.uint32), sub):
        x = u.view(np.float32)
        with np.errstate(invalid="ignore"):
            code, e = ref.encode(x.astype(np.float64))
        q = mx4.mx4_quantize(torch.from_numpy(x.copy()).cuda())
        _check_container(q, code, e)
        assert np.array_equal(_host(mx4.mx4_dequantize(q, torch.float32)), ref.decode(code, e),
                              equal_nan=True)


def test_codec_strides_and_outputs():
    v = _values((3, 20, 640), 9)
    big = _dev(v)
    x = big[:, 1:18, 64:224]                       # matrix and row strides of its own
    q = mx4.mx4_quantize(x)
    code, e = ref.encode(v[:, 1:18, 64:224])
    _check_container(q, code, e)
    again = mx4.empty_mx4(17, 160, 3)
    assert mx4.mx4_quantize(x, out=again) is again and torch.equal(again.data, q.data)
    big.fill_(7.0)
    mx4.mx4_dequantize(q, out=x)
    want = np.full(v.shape, 7.0)
    want[:, 1:18, 64:224] = ref.decode(code, e)
    assert np.array_equal(_host(big), want)        # nothing beside the view is written
    assert mx4.mx4_quantize(torch.empty((0, 64), device="cuda")).data.numel() == 0


# ---- products -----------------------------------------------------------------------

GEMM_SHAPES = [(1, 16, 32), (1, 1, 32), (1, 7168, 512), (2, 33, 96), (5, 100, 160), (16, 256, 640),
               (17, 48, 128), (31, 130, 1056), (33, 5003, 544), (64, 640, 512), (100, 257, 2080),
               (128, 512, 1024), (129, 300, 416), (257, 513, 288), (300, 1040, 32),
               (520, 260, 1536), (1, 512, 17408), (40, 96, 9248)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("x_mx4", [False, True])
@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm(M, N, K, x_mx4, out):
    xv, wv = _values((M, K), M + K), _values((N, K), N + K, 0.02)
    wq = mx4.mx4_quantize(_dev(wv))
    x = _dev(xv)
    if x_mx4:
        x, xv = mx4.mx4_quantize(x), ref.rounded(xv)
    want, tol = ref.matmul(xv, ref.rounded(wv))
    guard = torch.full((M + 2, N + 5), 3.0, dtype=TYPES[out], device="cuda")
    y = guard[1:M + 1, 2:N + 2]
    assert mx4.mx4_gemm(x, wq, y=y) is y
    ref.assert_close(_host(y), want, tol, out, "gemm")
    inside = torch.zeros_like(guard, dtype=torch.bool)
    inside[1:M + 1, 2:N + 2] = True
    assert bool((guard[~inside] == 3.0).all())
    # a contiguous output, the same bits
    z = mx4.mx4_gemm(x, wq, out_dtype=TYPES[out])
    assert torch.equal(z, y)


# every kernel, tile, count of waves and cut of K that a product is given
GEMM_KERNELS = [(M, N, 416) for M in (3, 11, 27, 50)
                for N in (16390, 21390, 29390, 33390, 41390)] + [
    (2, 2600, 8224), (4, 40, 8736), (13, 2700, 8224), (16, 300, 8224), (40, 100, 17376),
    (70, 130, 8256), (150, 200, 8288), (200, 3000, 160), (250, 4200, 96), (700, 2000, 96),
    (96, 16400, 544), (129, 56330, 160), (450, 7170, 96), (300, 3000, 4128), (129, 28200, 160),
    (300, 1000, 8224), (1030, 3100, 8224)]


@pytest.mark.parametrize("M,N,K", GEMM_KERNELS)
def test_gemm_kernels(M, N, K):
    xv = _values((M, K), M + K)
    wq = mx4.mx4_quantize(torch.randn(N, K, device="cuda",
                                      generator=torch.Generator("cuda").manual_seed(N)))
    wv = _host(mx4.mx4_dequantize(wq, torch.float32))
    x = _dev(xv)
    for a, av in ((x, xv), (mx4.mx4_quantize(x), ref.rounded(xv))):
        want, tol = ref.matmul(av, wv)
        ref.assert_close(_host(mx4.mx4_gemm(a, wq)), want, tol, "f32", "gemm")
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        ref.assert_close(_host(mx4.mx4_gemm(a, wq, y=out)), want, tol, "bf16", "gemm")


@pytest.mark.parametrize("M,N", [(1, 70), (16, 70), (30, 70), (64, 70), (200, 70), (3, 16390),
                                 (11, 16390), (27, 16390), (50, 16390), (96, 16400), (200, 3000),
                                 (250, 4200), (450, 7170), (129, 28200), (129, 56330)])
def test_gemm_special_values(M, N):
    """NaN scales, infinities and NaN of x reach their own rows and columns only;
    rows behind x and columns behind K are never read into the sums."""
    K = 416
    xv, wv = _values((M, K), 1), _values((N, K), 2)
    wv[3, 40] = np.inf                             # one block of row 3 is NaN
    xv[0, 5] = np.inf
    if M > 1:
        xv[M - 1, 7] = np.nan
    wide = torch.full((M + 1, K + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:M, :K] = _dev(xv)
    wq = mx4.mx4_quantize(_dev(wv))
    wr = ref.rounded(wv)
    y = _host(mx4.mx4_gemm(wide[:M, :K], wq))
    with np.errstate(invalid="ignore"):
        want = xv @ wr.T
    keep = np.isfinite(want)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    assert np.array_equal(y[np.isinf(want)], want[np.isinf(want)])
    tol = ref.gamma(K) * (np.abs(np.where(np.isfinite(xv), xv, 0)) @ np.abs(np.nan_to_num(wr)).T)
    assert (np.abs(y[keep] - want[keep]) <= tol[keep] + 2.0 ** -24 * np.abs(want[keep])).all()
    q = mx4.mx4_quantize(wide[:M, :K])
    with np.errstate(invalid="ignore"):
        want = ref.rounded(xv) @ wr.T
    assert np.array_equal(np.isnan(_host(mx4.mx4_gemm(q, wq))), np.isnan(want))


def test_gemm_extreme_scales():
    """Weights and activations at both ends of the exponent range."""
    M, N, K = 4, 32, 256
    for sx, sw in ((1e30, 1e-30), (1e-36, 1e30), (2.0 ** 100, 2.0 ** -126), (1e18, 1e18)):
        xv, wv = _values((M, K), 1, sx), _values((N, K), 2, sw)
        wq = mx4.mx4_quantize(_dev(wv))
        for x_mx4 in (False, True):
            x = _dev(xv)
            if x_mx4:
                x = mx4.mx4_quantize(x)
            want, tol = ref.matmul(ref.rounded(xv) if x_mx4 else xv, ref.rounded(wv))
            ref.assert_close(_host(mx4.mx4_gemm(x, wq)), want, tol, "f32", "extreme")


@pytest.mark.parametrize("ldx", [(1 << 23) - 8, 1 << 23])
def test_gemm_wide_row_stride(ldx):
    """Rows of x 16 MB apart, on both sides of what a tile's 24-bit row offsets take."""
    M, N, K = 96, 16400, 64
    xv, wv = _values((M, K), 85), _values((N, K), 86)
    x = torch.empty_strided((M, K), (ldx, 1), dtype=torch.bfloat16, device="cuda")
    x.copy_(_dev(xv))
    want, tol = ref.matmul(xv, ref.rounded(wv))
    ref.assert_close(_host(mx4.mx4_gemm(x, mx4.mx4_quantize(_dev(wv)))), want, tol, "f32", "wide")


def test_offsets_past_32_bits():
    """A container of 4.4 GB that repeats one matrix (read again at stride 0): every
    repetition decodes to, and multiplies as, the first one, bit for bit."""
    B, R, K = 130, 1024, 65536
    w = _dev(_values((R, K), 90, 0.02))
    one = mx4.mx4_quantize(w)
    q = mx4.mx4_quantize(w.expand(B, R, K))
    assert q.codes.numel() > 1 << 32
    y = mx4.mx4_dequantize(q)
    first = mx4.mx4_dequantize(one)
    for b in (0, 64, 65, B - 1):
        assert torch.equal(y[b], first)
    del y
    whole = mx4.MX4Tensor(q.data, B * R, K)             # the same bytes as one [B R, K]
    for M in (1, 3, 40, 200):
        xv = _values((M, K), 91 + M)
        x = _dev(xv)
        for a, av in ((x, xv), (mx4.mx4_quantize(x), ref.rounded(xv))):
            y = mx4.mx4_gemm(a, whole).view(M, B, R)
            assert torch.equal(y, y[:, :1].expand(M, B, R))
            rows = _host(first[:64])
            want, tol = ref.matmul(av, rows)
            ref.assert_close(_host(y[:, B - 1, :64]), want, tol, "f32", "large")


# ---- expert layer -------------------------------------------------------------------

def _moe_case(T, H, I, E, seed):
    xv = _values((T, H), seed)
    w13, w2 = _values((E, 2 * I, H), seed + 1, 0.05), _values((E, H, I), seed + 2, 0.05)
    logits = np.random.default_rng(seed + 3).standard_normal((T, E)).astype(np.float32)
    q13, q2 = mx4.mx4_quantize(_dev(w13)), mx4.mx4_quantize(_dev(w2))
    return xv, logits, ref.rounded(w13), ref.rounded(w2), q13, q2


MOE_SHAPES = [(1, 64, 32, 1, 1), (1, 256, 96, 8, 2), (2, 160, 64, 5, 5), (7, 416, 160, 16, 3),
              (16, 512, 128, 64, 6), (33, 96, 544, 12, 4), (61, 288, 96, 127, 8),
              (128, 128, 64, 4, 2), (128, 96, 32, 300, 32), (3, 544, 1056, 70, 7),
              # few tokens that share most experts; few experts with a long I; many
              # workgroups of the down product; one token on every width of the choice
              (4, 512, 448, 8, 8), (9, 512, 256, 24, 12), (16, 288, 608, 70, 32),
              (6, 96, 4128, 4, 4), (40, 96, 4128, 4, 2), (40, 1056, 64, 64, 4),
              (24, 96, 64, 30, 2), (28, 96, 4128, 4, 2), (128, 160, 96, 3, 3),
              (70, 1056, 160, 2, 1), (1, 160, 96, 100, 3), (2, 96, 64, 250, 32),
              (1, 96, 64, 1024, 32)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,H,I,E,k", MOE_SHAPES)
def test_moe(T, H, I, E, k, renormalize, out):
    xv, logits, w13, w2, q13, q2 = _moe_case(T, H, I, E, T + H)
    want, tol = ref.moe(xv, logits, w13, w2, k, renormalize, 3 if out == "f32" else 2)
    guard = torch.full((T + 2, H + 5), 3.0, dtype=TYPES[out], device="cuda")
    y = guard[1:T + 1, 2:H + 2]
    wide = torch.full((T, H + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = _dev(xv)
    lw = torch.full((T, E + 3), float("inf"), device="cuda")
    lw[:, :E] = torch.from_numpy(logits).cuda()
    mx4.mx4_moe(wide[:, :H], lw[:, :E], q13, q2, k, renormalize=renormalize, y=y)
    ref.assert_close(_host(y), want, tol, out, "moe")
    inside = torch.zeros_like(guard, dtype=torch.bool)
    inside[1:T + 1, 2:H + 2] = True
    assert bool((guard[~inside] == 3.0).all())
    z = mx4.mx4_moe(_dev(xv), torch.from_numpy(logits).cuda(), q13, q2, k,
                    renormalize=renormalize, out_dtype=TYPES[out])
    assert torch.equal(z, y)


@pytest.mark.parametrize("T,E,H,I", [(9, 6, 128, 64), (9, 200, 128, 64), (9, 6, 512, 1024),
                                     (50, 6, 128, 64), (50, 200, 128, 64)])
def test_moe_routing_edges(T, E, H, I):
    """Ties (also of -0 and +0), masked experts, a token with fewer experts than
    top_k, one with none, and NaN and infinite logits."""
    k = 4
    xv, logits, w13, w2, q13, q2 = _moe_case(T, H, I, E, 40)
    logits[0] = 0.0
    logits[1] = np.where(np.arange(E) % 2, 0.0, -0.0)
    logits[2, 2:] = -np.inf
    logits[3] = -np.inf
    logits[4] = np.round(logits[4])
    logits[5, 3] = np.nan
    logits[6, 1] = np.inf
    logits[7, E - 1] = 100.0
    logits[8] = -1e30
    for renormalize in (True, False):
        rows = [0, 1, 2, 3, 4, 7, 8]
        want, tol = ref.moe(xv, np.where(np.isfinite(logits) | (logits == -np.inf), logits, 0.0),
                            w13, w2, k, renormalize, 3)
        y = _host(mx4.mx4_moe(_dev(xv), torch.from_numpy(logits).cuda(), q13, q2, k,
                              renormalize=renormalize, out_dtype=torch.float32))
        ref.assert_close(y[rows], want[rows], tol[rows], "f32", "routing")
        assert np.isnan(y[5]).all() and np.isnan(y[6]).all()
        assert (y[3] == 0).all()


def test_moe_bad_expert_stays_with_its_tokens():
    """A NaN block of one expert reaches the tokens that chose it and no others."""
    T, H, I, E, k = 12, 128, 64, 8, 2
    xv, logits, w13, w2, q13, q2 = _moe_case(T, H, I, E, 50)
    raw = _values((E, H, I), 52, 0.05)
    bad = int(np.argmax(logits[0]))
    raw[bad, 7, 3] = np.nan
    q2 = mx4.mx4_quantize(_dev(raw))
    y = _host(mx4.mx4_moe(_dev(xv), torch.from_numpy(logits).cuda(), q13, q2, k))
    chose = np.array([bad in np.argsort(-logits[t], kind="stable")[:k] for t in range(T)])
    assert chose.any() and not chose.all()
    assert np.array_equal(np.isnan(y).any(1), chose)
    assert np.array_equal(np.isnan(y[:, 7]), chose)


def test_moe_offsets_past_32_bits():
    """1024 times the same expert, 4.4 GB of gate and up weights: the last ones give
    what the first ones give, bit for bit."""
    H, I, E = 4096, 1056, 1024
    w13, w2 = _dev(_values((2 * I, H), 95, 0.02)), _dev(_values((H, I), 96, 0.02))
    q13 = mx4.mx4_quantize(w13.expand(E, 2 * I, H))
    q2 = mx4.mx4_quantize(w2.expand(E, H, I))
    assert q13.codes.numel() > 1 << 32
    for T in (1, 3, 40):
        x = _dev(_values((T, H), 97 + T))
        logits = torch.zeros((T, E), device="cuda")
        logits[:, 0], logits[:, 1] = 3.0, 2.5
        first = mx4.mx4_moe(x, logits, q13, q2, 2)
        last = mx4.mx4_moe(x, logits.roll(E - 2, 1), q13, q2, 2)
        assert first.abs().max() > 0 and torch.equal(first, last)


# ---- a run of them together ------------------------------------------------------------

def test_expert_block_with_its_router():
    """Router product on the lossless weights, expert layer, 4-bit projection of
    its output with both sides quantised: as a decode step chains them."""
    T, H, I, E, k, N = 5, 512, 128, 16, 4, 96
    xv, _, w13, w2, q13, q2 = _moe_case(T, H, I, E, 60)
    router, _ = w12.pack(_dev(_values((E, H), 61, 0.05)), exceptions=True)
    x = _dev(xv)
    logits = w12.w12_gemm(x, router)
    y = mx4.mx4_moe(x, logits, q13, q2, k)
    want, tol = ref.moe(xv, logits.cpu().numpy(), w13, w2, k, True, 2)
    ref.assert_close(_host(y), want, tol, "bf16", "chain: experts")
    wo = _values((N, H), 62, 0.05)
    out = mx4.mx4_gemm(mx4.mx4_quantize(y), mx4.mx4_quantize(_dev(wo)))
    want, tol = ref.matmul(ref.rounded(_host(y)), ref.rounded(wo))
    ref.assert_close(_host(out), want, tol, "f32", "chain: projection")


def test_graphs_and_streams():
    """Captured calls replayed with eager work between, two graphs in turn and on
    two streams at once: every result equals the eager one bit for bit."""
    T, H, I, E, k, N = 6, 256, 96, 12, 3, 4112
    xv, logits, _, _, q13, q2 = _moe_case(T, H, I, E, 70)
    wq = mx4.mx4_quantize(_dev(_values((N, H), 71)))
    xs = [_dev(xv), _dev(_values((T, H), 72))]
    big = [_dev(_values((40, H), 73)), _dev(_values((40, H), 74))]
    lg = torch.from_numpy(logits).cuda()
    lg40 = torch.from_numpy(np.random.default_rng(75).standard_normal((40, E))
                            .astype(np.float32)).cuda()

    def step(x, b):
        q = mx4.mx4_quantize(x)
        return (mx4.mx4_dequantize(q), mx4.mx4_gemm(x, wq), mx4.mx4_gemm(q, wq),
                mx4.mx4_gemm(b, wq), mx4.mx4_moe(x, lg, q13, q2, k),
                mx4.mx4_moe(b, lg40, q13, q2, k))

    want = [[t.clone() for t in step(x, b)] for x, b in zip(xs, big)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, b in zip(xs, big):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x, b))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = step(xs[rep % 2], big[rep % 2])
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in zip(outs[i], want[i]):
                assert torch.equal(a, b), (rep, i)
        for a, b in zip(eager, want[rep % 2]):
            assert torch.equal(a, b)


def test_same_data_in_both_places():
    """One container as both operands, one weight in two calls at once."""
    v = _values((40, 288), 80)
    q = mx4.mx4_quantize(_dev(v))
    r = ref.rounded(v)
    want, tol = ref.matmul(r, r)
    ref.assert_close(_host(mx4.mx4_gemm(q, q)), want, tol, "f32", "gram")
