"""Offsets past 32 bits and the largest sizes of the MX8 calls, the routing and the
verification: the same results as from compact rows."""
import pytest
import torch

from lossless_bit_weight_amd import draft, mx4, mx8
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

GIB = 1 << 30


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def _far(rows, ld, dtype):
    """rows (2-D) with ld elements from one to the next, in a buffer of their own."""
    R, K = rows.shape
    need = ((R - 1) * ld + K) * rows.element_size()
    if torch.cuda.mem_get_info()[0] < need + 8 * GIB:
        pytest.skip("%d GiB of memory" % (need >> 30))
    buf = torch.empty((R - 1) * ld + K, dtype=dtype, device="cuda")
    view = buf.as_strided((R, K), (ld, 1))
    view.copy_(rows)
    return view


def _bytes_of(q):
    return q.values.contiguous().view(torch.uint8), q.scales[:, :16 * ((q.shape[1] + 511) // 512)]


def _randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def test_norm_and_codec_of_rows_far_apart():
    x, r, w = _randn(3, 544), _randn(3, 544, seed=1), _randn(544, seed=2)
    want, s = mx8.mx8_rms_norm(x, w, residual=r)
    ld = 3 * GIB // 2 + 64                      # 3 GiB and some bytes from row to row
    fx = _far(x, ld, torch.bfloat16)
    got, fs = mx8.mx8_rms_norm(fx, w, residual=r, residual_out=fx)
    assert fs is fx and torch.equal(fx, s)
    for a, b in zip(_bytes_of(got), _bytes_of(want)):
        assert torch.equal(a, b)
    want = mx8.mx8_quantize(s)
    values = torch.empty(2 * ld + 544, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2 * ld + 32, dtype=torch.uint8, device="cuda")
    out = mx8.MX8Tensor(values.view(mx8.VALUES).as_strided((3, 544), (ld, 1)),
                        scales.as_strided((3, 32), (ld, 1)))
    mx8.mx8_quantize(fx, out)
    assert torch.equal(out.values.contiguous().view(torch.uint8), _bytes_of(want)[0])
    assert torch.equal(out.scales, _bytes_of(want)[1])
    fx.zero_()
    mx8.mx8_dequantize(out, out=fx)
    assert torch.equal(fx, mx8.mx8_dequantize(want))


# few rows, 16 and 32 of them in slices, tiles; on both sides of the distance (2^24) from
# which tiles give way to the few-row kernel
@pytest.mark.parametrize("M,N,K", [(9, 40, 544), (16, 512, 17408), (20, 512, 17408),
                                   (200, 4100, 1056), (130, 520, 17408)])
@pytest.mark.parametrize("ldv,lds", [((1 << 24) - 16, (1 << 24) - 16), (1 << 24, 1024),
                                     (17408, (1 << 24) + 16), ((1 << 26) + 16, 1024)])
def test_gemm_of_rows_far_apart(M, N, K, ldv, lds):
    q = mx8.mx8_quantize(_randn(M, K))
    w = mx4.mx4_quantize(_randn(N, K, seed=1))
    far = mx8.MX8Tensor(_far(q.values.view(torch.uint8), ldv, torch.uint8).view(mx8.VALUES),
                        _far(q.scales, lds, torch.uint8))
    want, got = mx8.mx8_gemm(q, w), mx8.mx8_gemm(far, w)
    # another kernel adds in another order: two sums of up to 137 instructions' results, each
    # addition off by half a step (2^-24) of a partial sum below 4 times the largest result
    assert float((got - want).abs().max()) <= 2 * 137 * 4 * 2.0 ** -24 * float(want.abs().max())


def test_gemm_into_rows_far_apart():
    q, w = mx8.mx8_quantize(_randn(200, 1056)), mx4.mx4_quantize(_randn(4100, 1056, seed=1))
    want = mx8.mx8_gemm(q, w, torch.bfloat16)
    y = _far(torch.zeros_like(want), (1 << 25) + 1, torch.bfloat16)
    mx8.mx8_gemm(q, w, y=y)
    assert torch.equal(y, want)


def test_route_of_rows_far_apart():
    l = _randn(3, 96)
    want = mx4.mx4_route(l, 5)
    got = mx4.mx4_route(_far(l, (1 << 31) + 1, torch.bfloat16), 5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_route_of_the_most_tokens():
    P = 1024
    T, l = 1 << 24, _randn(P, 4, dtype=torch.float32)
    e, s = mx4.mx4_route(l, 1)
    ee, ss = mx4.mx4_route(l.repeat(T // P, 1), 1)
    assert bool((ee.view(-1, P) == e.view(1, P)).all())
    assert bool((ss.view(-1, P) == s.view(1, P)).all())


@pytest.mark.parametrize("probs", [False, True])
def test_verify_of_rows_far_apart(probs):
    B, D, V, ld = 2, 2, 1003, (1 << 30) + 1
    l = _randn(B * (D + 1), V) * 2
    d = torch.randint(0, V, (B, D), device="cuda", dtype=torch.int32)
    d[:, 0] = l.view(B, D + 1, V)[:, 0].argmax(-1).to(torch.int32)
    u = torch.tensor([[0.0, 0.7, 0.3], [0.0, 0.2, 0.9]], device="cuda")
    q = torch.softmax(_randn(B * D, V, seed=3).float(), -1).to(torch.bfloat16) if probs else None
    want = draft.draft_verify(l.view(B, D + 1, V), d, u,
                              draft_probs=None if q is None else q.view(B, D, V))
    far = _far(l, ld, torch.bfloat16).as_strided((B, D + 1, V), ((D + 1) * ld, ld, 1))
    fq = None if q is None else \
        _far(q, ld, torch.bfloat16).as_strided((B, D, V), (D * ld, ld, 1))
    got = draft.draft_verify(far, d, u, draft_probs=fq)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int(want[1].min()) >= 1


def test_verify_of_the_most_words():
    """2^30 words, all masked but three of probabilities 1/8, 1/2, 3/8."""
    V = 1 << 30
    l = torch.full((1, 1, V), -torch.inf, dtype=torch.bfloat16, device="cuda")
    where = [5, (1 << 29) + 3, V - 1]
    l[0, 0, where] = torch.tensor([0.0, 2.0, 1.5849625], device="cuda").mul(0.6931472).bfloat16()
    none = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    for u, w in ((0.0, 0), (0.1, 0), (0.15, 1), (0.6, 1), (0.65, 2), (1.0, 2)):
        t, a = draft.draft_verify(l, none, torch.tensor([[u]], device="cuda"))
        assert t.tolist() == [[where[w]]] and a.tolist() == [0]
    t, _ = draft.draft_verify(l, none, torch.zeros(1, 1, device="cuda"),
                              temperature=torch.zeros(1, device="cuda"))
    assert t.tolist() == [[where[1]]]
