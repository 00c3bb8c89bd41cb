"""The MX8 calls on the GPU against their 64-bit forms: the codec bit for bit, the
norm and the product within bounds that their roundings give."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4, mx8
from tests import mx4_ref, step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _bf16(v):
    return mx4_ref.bf16_to_f64(mx4_ref.f64_to_bf16_bits(v))


def _values(shape, seed, sigma=1.0):
    """BF16-exact normal values in float64."""
    return _bf16(np.random.default_rng(seed).standard_normal(shape) * sigma)


def _dev(v, dtype=torch.bfloat16):
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).cuda().to(dtype)


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _bytes(q):
    return q.values.view(torch.uint8).cpu().numpy(), q.scales.cpu().numpy()


def _same_codec(v, dtype):
    """v [R, K] float64, exact in dtype: bytes, scales, and the values read back."""
    q = mx8.mx8_quantize(_dev(v, TYPES[dtype]))
    code, e = ref.encode8(v)
    got_code, got_scales = _bytes(q)
    assert np.array_equal(got_code, code)
    assert np.array_equal(got_scales, ref.scale_rows(e))
    assert np.array_equal(q.block_scales.cpu().numpy(), e)
    want = ref.decode8(code, e)
    for out in ("bf16", "f32"):
        back = _host(mx8.mx8_dequantize(q, TYPES[out]))
        assert np.array_equal(back, want, equal_nan=True), out


def test_codec_every_bf16_value():
    """Every BF16 value beside each largest value of its block that changes the scale:
    each exponent from its own to twenty above."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    v = mx4_ref.bf16_to_f64(bits)
    for up in (0, 1, 3, 4, 8, 14, 20):
        rows = v[:65536 // 31 * 31].reshape(-1, 31)
        top = np.abs(np.where(np.isfinite(rows), rows, 0.0)).max(-1, keepdims=True)
        top = np.exp2(np.minimum(np.floor(np.log2(np.maximum(top, 2.0 ** -126))) + up, 127))
        _same_codec(np.concatenate((rows, top), 1), "bf16")
    _same_codec(np.repeat(v, 32).reshape(-1, 32), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 512), (3, 544), (17, 160), (64, 5120), (5, 17376)])
def test_codec(R, K, dtype):
    rng = np.random.default_rng(R + K)
    v = rng.standard_normal((R, K)) * np.exp2(rng.integers(-30, 30, (R, K // 32)).repeat(32, 1))
    v = _bf16(v) if dtype == "bf16" else v.astype(np.float32).astype(np.float64)
    v[:, 3] = 0.0
    v[0, 4] = -0.0
    _same_codec(v, dtype)


def test_codec_ties_and_edges_fp32():
    """Ties between neighbours, halves of the smallest, values around 448, subnormals,
    infinities and NaN."""
    grid = ref.TABLE[:127]
    mid = np.concatenate(((grid[:-1] + grid[1:]) / 2, np.arange(17) / 4 + 0.125))
    rows = []
    for s in (1.0, 2.0 ** -100, 2.0 ** 100):
        for t in (mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                  np.nextafter(mid.astype(np.float32), np.float32(1e9))):
            t = np.concatenate((t, -t)).astype(np.float64)
            t = np.resize(t, (len(t) + 30) // 31 * 31).reshape(-1, 31) * s
            rows.append(np.concatenate((t, np.full((len(t), 1), 256.0 * s)), 1))
    rows.append(np.array([[449.0, 463.9, 464.0, 465.0, 480.0, 511.9] + [0.0] * 26]))
    tiny = np.float64(np.float32(1e-45))
    rows.append(np.array([[tiny, -3 * tiny, 2.0 ** -126, 2.0 ** -127, 2.0 ** -140] + [0.0] * 27]))
    rows.append(np.array([[2.0 ** -119 * 1.9, 2.0 ** -136, 2.0 ** -137, tiny] + [0.0] * 28]))
    rows.append(np.array([[np.inf] + [1.0] * 31, [1.0] * 31 + [-np.inf], [np.nan] + [2.0] * 31,
                          [np.finfo(np.float32).max] * 32, [0.0] * 32]))
    _same_codec(np.concatenate(rows).astype(np.float32).astype(np.float64), "f32")


def test_codec_of_views():
    """Rows apart in memory, both ways; rows cut out; what lies beside them stays."""
    v = _values((9, 96), 3)
    full = _dev(np.pad(v, ((0, 0), (8, 24)), constant_values=5.0))
    out = mx8.MX8Tensor(torch.zeros(9, 128, dtype=torch.uint8, device="cuda").view(mx8.VALUES)[:, :96],
                        torch.full((9, 48), 9, dtype=torch.uint8, device="cuda")[:, 16:])
    q = mx8.mx8_quantize(full[:, 8:104], out)
    assert q is out
    code, e = ref.encode8(v)
    assert np.array_equal(q.values.view(torch.uint8).cpu().numpy(), code)
    assert np.array_equal(q.scales[:, :16].cpu().numpy(), ref.scale_rows(e))
    assert bool((q.scales[:, 16:] == 9).all())
    y = torch.full((9, 128), 7.0, device="cuda")
    mx8.mx8_dequantize(q[2:5], out=y[2:5, 16:112])
    want = np.full((9, 128), 7.0)
    want[2:5, 16:112] = ref.decode8(code, e)[2:5]
    assert np.array_equal(_host(y), want)


# ---- norm ------------------------------------------------------------------------------

# Everything before the last rounding is held in 64 bits: some steps of 2^-53 in the sum of
# up to 2^15 squares, its root and two products.  BF16 is rounded from fp32: half a step of
# fp32 more.
REL = 2.0 ** -36


def _assert_mx8_near(q, y):
    """Bytes and scales are those of some y (1 + d) with |d| <= REL."""
    got, scales = _bytes(q)
    K = y.shape[1]
    top = np.abs(y).reshape(len(y), -1, 32).max(-1)
    e = q.block_scales.cpu().numpy().astype(int)
    assert np.all((e == ref.exponent(top * (1 - REL))) | (e == ref.exponent(top * (1 + REL))))
    assert np.array_equal(scales, ref.scale_rows(e.astype(np.uint8)))
    t = np.abs(y) / np.ldexp(1.0, e - 127).repeat(32, 1)[:, :K]
    lo, hi = ref.nearest_e4m3(t * (1 - REL)), ref.nearest_e4m3(t * (1 + REL))
    assert np.all(((got & 127) >= lo) & ((got & 127) <= hi))
    assert np.array_equal(got >> 7, np.signbit(y).astype(np.uint8))
    back = _host(mx8.mx8_dequantize(q, torch.float32))
    assert np.array_equal(back, ref.decode8(got, e.astype(np.uint8)))


def _norm_case(M, K, x, res, w, out, seed=0):
    rng = np.random.default_rng(M * 7 + K + seed)
    spread = np.exp(rng.standard_normal((1, K)))
    exact = {"bf16": _bf16, "f32": lambda v: v.astype(np.float32).astype(np.float64)}
    xv = exact[x](rng.standard_normal((M, K)) * spread)
    rv = None if res == "none" else exact[res](3 * rng.standard_normal((M, K)) * spread)
    wv = exact[w](1 + 0.3 * rng.standard_normal(K))
    y, s = ref.norm(xv, rv, wv, 1e-6, res == "bf16")
    got = mx8.mx8_rms_norm(_dev(xv, TYPES[x]), _dev(wv, TYPES[w]), 1e-6,
                           residual=None if rv is None else _dev(rv, TYPES[res]),
                           out_dtype=mx8.VALUES if out == "mx8" else TYPES[out])
    if rv is not None:
        got, kept = got
        assert kept.dtype is TYPES[res] and np.array_equal(_host(kept), s)
    if out == "mx8":
        _assert_mx8_near(got, y)
    else:
        assert got.dtype is TYPES[out]
        mx4_ref.assert_close(_host(got), y, np.abs(y) * (REL + (2.0 ** -24 if out == "bf16" else 0.0)),
                             out, "norm")


@pytest.mark.parametrize("out", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("x,res,w", [("bf16", "none", "bf16"), ("f32", "none", "f32"),
                                     ("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"),
                                     ("bf16", "f32", "bf16"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 5120), (3, 160), (33, 1056)])
def test_norm_types(M, K, x, res, w, out):
    _norm_case(M, K, x, res, w, out)


# every width a row of threads holds, a value short of it and a block past it
@pytest.mark.parametrize("K", [64, 96, 128, 480, 512, 544, 1024, 2016, 2048, 2080, 4096, 4128,
                               8192, 8224, 16384, 16416, 32768])
@pytest.mark.parametrize("M", [1, 2, 37])
def test_norm_widths(M, K):
    _norm_case(M, K, "bf16", "bf16", "bf16", "mx8")
    _norm_case(M, K, "f32", "none", "f32", "f32")


@pytest.mark.parametrize("K", [128, 224, 256, 512, 544, 4096, 5120, 8192])
@pytest.mark.parametrize("M", [257, 1024, 1025, 2049])
def test_norm_many_rows(M, K):
    _norm_case(M, K, "bf16", "bf16", "bf16", "bf16")


def test_norm_of_extremes():
    """Rows of zeros, one value alone, squares past fp32's range, the smallest values, a
    NaN and an infinity: each row by itself."""
    K = 96
    v = np.zeros((8, K))
    v[1, 5] = 3.0
    v[2] = 2.0 ** 100
    v[3] = 2.0 ** -140
    v[4] = 1.0
    v[4, 7] = np.nan
    v[5] = 1.0
    v[5, 9] = np.inf
    v[6] = -1.0
    v[7] = 3.0e38
    w = np.ones(K)
    for eps in (1e-6, 0.0):
        got = _host(mx8.mx8_rms_norm(_dev(v, torch.float32), _dev(w), eps, out_dtype=torch.float32))
        with np.errstate(all="ignore"):
            x = v.astype(np.float32).astype(np.float64)
            want = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if eps == 0.0:
            want[0] = np.nan                    # 0 * (1 / 0)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fin = ~np.isnan(want)
        assert np.all(np.abs(got - want)[fin] <= np.abs(want[fin]) * 5 * 2.0 ** -24 + 2.0 ** -149)
    q = mx8.mx8_rms_norm(_dev(v, torch.float32), _dev(w), 1e-6)
    e = q.block_scales.cpu().numpy()
    assert np.all(e[4] == 255) and np.all(e[0] == 0) and np.all(e[6] == 118)
    assert list(e[5]) == [255, 0, 0]            # inf * 0, and 1 / inf = 0 beside it


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place(dtype):
    """The residual updated where it is, y written over x: bits of the call apart."""
    x, r = _dev(_values((19, 544), 1), TYPES[dtype]), _dev(_values((19, 544), 2), TYPES[dtype])
    w = _dev(_values(544, 3))
    y, s = mx8.mx8_rms_norm(x, w, residual=r, out_dtype=TYPES[dtype])
    y2, s2 = mx8.mx8_rms_norm(x, w, residual=r, residual_out=r, out=x)
    assert y2 is x and s2 is r
    assert torch.equal(y, x) and torch.equal(s, r)


def test_norm_of_more_rows_than_one_launch_axis_holds():
    """2^22 and some rows, a workgroup each: the grid's second axis."""
    M, K, P = (1 << 22) + 3 * 32, 4128, 32
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GiB of memory")
    rows = _dev(_values((P, K), 8))
    w = _dev(_values(K, 9))
    want = mx8.mx8_rms_norm(rows, w, out_dtype=torch.bfloat16)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.view(-1, P, K).copy_(rows)
    mx8.mx8_rms_norm(x, w, out=x)
    for first in (0, 1 << 20, (1 << 21) - P, 1 << 21, (1 << 22) - P, 1 << 22, M - P):
        assert torch.equal(x[first:first + P], want)
    del x
    torch.cuda.empty_cache()


def test_norm_of_views():
    full = _dev(_values((7, 160), 4))
    rfull = _dev(_values((7, 200), 5), torch.float32)
    w = _dev(_values(96, 6))
    x, r = full[::2, 32:128], rfull[:4, 8:104]
    y, s = mx8.mx8_rms_norm(x, w, residual=r, out_dtype=torch.bfloat16)
    y2, s2 = mx8.mx8_rms_norm(x.contiguous(), w, residual=r.contiguous(), out_dtype=torch.bfloat16)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    buf = torch.full((5, 112), 3.0, device="cuda", dtype=torch.bfloat16)
    mx8.mx8_rms_norm(x, w, residual=r, out=buf[:4, 8:104])
    assert torch.equal(buf[:4, 8:104], y)
    buf[:4, 8:104] = 3.0
    assert bool((buf == 3.0).all())


# ---- product -----------------------------------------------------------------------------

# few rows, tiles of 16, 32, 64, 128 rows and one past them; ragged N and K; a long K; then
# every kernel by its rule, whole and in slices: waves that split K over one tile (4, 8 of
# them) and two, 16 rows shared by 4 and 5 waves, by 2 x 2 and 4 x 2, 32 rows by 4 x 2, tiles
# of 32 x 128, 64 x 128, 64 x 160 and 64 x 256
GEMM_SHAPES = [(16, 5000, 544), (16, 7000, 6176), (13, 512, 6176), (129, 3000, 160),
               (5, 16400, 4128), (16, 23000, 4096), (160, 5120, 640), (256, 5000, 12320),
               (2050, 3333, 288), (60, 16500, 160), (1, 16, 32), (1, 7168, 5120), (2, 48, 160), (3, 1000, 2080), (16, 512, 544),
               (17, 100, 5120), (33, 5003, 1056), (40, 256, 17408), (64, 640, 1024),
               (65, 1040, 512), (128, 2048, 2560), (129, 300, 4128), (200, 5120, 640),
               (300, 96, 65536), (513, 1100, 288), (1024, 4096, 1024), (1, 20000, 96),
               (5, 34816, 256), (20, 17000, 544), (50, 20500, 320), (2000, 3000, 160),
               (64, 40900, 544), (127, 20001, 1056), (250, 1601, 12320),
               (17, 2414, 1120), (18, 71, 8992), (19, 4295, 1120), (19, 423, 9792), (17, 10090, 1568),
               (899, 64, 16768), (20, 64, 2272), (322, 9169, 544), (176, 11193, 1056),
               (1664, 129, 9056), (1665, 3912, 544), (70, 11072, 8800)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm_of_whole_numbers(M, N, K, out):
    """Every sum is one of whole numbers that fp32 holds: exact."""
    rng = np.random.default_rng(M + N + K)
    w = rng.choice([0.0, 1.0, 2.0, 3.0, -4.0, 6.0, -1.0], (N, K)).astype(np.float32)
    w[:, ::32] = 4.0                            # the scale of every block is 1
    x = rng.integers(-15, 16, (M, K)).astype(np.float32)
    wq = mx4.mx4_quantize(torch.from_numpy(w).cuda())
    xq = mx8.mx8_quantize(torch.from_numpy(x).cuda())
    # 15 is kept as 14 where it is its block's largest: 448 / 512 of the next power of two
    kept = ref.decode8(*ref.encode8(x.astype(np.float64)))
    assert np.array_equal(kept, np.where(np.abs(x) == 15, kept, x)) and np.abs(kept).max() <= 15
    assert np.array_equal(_host(mx8.mx8_dequantize(xq)), kept)
    x = kept.astype(np.float32)
    got = _host(mx8.mx8_gemm(xq, wq, TYPES[out]))
    want = (torch.from_numpy(x).cuda().double() @ torch.from_numpy(w).cuda().double().T)
    want = want.to(TYPES[out]).double().cpu().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 96, 1056), (7, 100, 5120), (16, 64, 96), (33, 530, 2080),
                                   (100, 200, 17408), (257, 260, 1024)])
def test_gemm_of_scaled_blocks(M, N, K, out):
    """Blocks whose scales differ by powers of two up to 2^24, on both sides."""
    rng = np.random.default_rng(M * N + K)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-12, 12, (M, K // 32)).repeat(32, 1))
    w = rng.standard_normal((N, K)) * np.exp2(rng.integers(-12, 12, (N, K // 32)).repeat(32, 1))
    x, w = _bf16(x), _bf16(w)
    got = _host(mx8.mx8_gemm(mx8.mx8_quantize(_dev(x)), mx4.mx4_quantize(_dev(w)), TYPES[out]))
    want, tol = mx4_ref.matmul(ref.decode8(*ref.encode8(x)), mx4_ref.rounded(w))
    mx4_ref.assert_close(got, want, tol, out, "gemm")


@pytest.mark.parametrize("M,N,K", [(1, 64, 96), (40, 64, 5120), (150, 130, 1056)])
def test_gemm_keeps_nan_in_its_row_and_column(M, N, K):
    x, w = _values((M, K), 1), _values((N, K), 2)
    x[M // 2, K - 1] = np.inf
    w[N // 3, 5] = np.nan
    y = _host(mx8.mx8_gemm(mx8.mx8_quantize(_dev(x)), mx4.mx4_quantize(_dev(w))))
    want = np.zeros((M, N), bool)
    want[M // 2] = True
    want[:, N // 3] = True
    assert np.array_equal(np.isnan(y), want)


@pytest.mark.parametrize("M,N,K", [(3, 50, 96), (33, 70, 544), (70, 1030, 17408), (300, 500, 512)])
def test_gemm_of_views(M, N, K):
    """Rows of x cut out of a larger one, with strides; a strided y whose neighbours stay."""
    v = _values((M + 4, K), 1)
    wq = mx4.mx4_quantize(_dev(_values((N, K), 2)))
    whole = mx8.mx8_quantize(_dev(v))
    n = whole.scales.shape[1]
    wide = mx8.MX8Tensor(
        torch.full((M + 4, K + 48), 255, dtype=torch.uint8, device="cuda").view(mx8.VALUES)[:, 16:16 + K],
        torch.full((M + 4, n + 32), 255, dtype=torch.uint8, device="cuda")[:, 16:16 + n])
    wide.values.view(torch.uint8)[:] = whole.values.view(torch.uint8)
    wide.scales[:] = whole.scales
    want = mx8.mx8_gemm(mx8.mx8_quantize(_dev(v[3:3 + M])), wq)
    y = torch.full((M, N + 5), 4.5, device="cuda")
    mx8.mx8_gemm(wide[3:3 + M], wq, y=y[:, 2:2 + N])
    assert torch.equal(y[:, 2:2 + N], want)
    y[:, 2:2 + N] = 4.5
    assert bool((y == 4.5).all())
    yb = torch.full((M, N + 3), 4.5, device="cuda", dtype=torch.bfloat16)
    mx8.mx8_gemm(wide[3:3 + M], wq, y=yb[:, 1:1 + N])
    assert torch.equal(yb[:, 1:1 + N], want.to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(1, 512, 17408), (33, 512, 17408), (200, 5120, 5120)])
def test_gemm_stays_within_its_workspace(M, N, K):
    need = mx8.mx8_gemm_workspace_bytes(M, N, K)
    xq, wq = mx8.mx8_quantize(_dev(_values((M, K), 1))), mx4.mx4_quantize(_dev(_values((N, K), 2)))
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    y = mx8.mx8_gemm(xq, wq, workspace=ws[:need])
    assert bool((ws[need:] == 255).all())
    assert torch.equal(y, mx8.mx8_gemm(xq, wq))
