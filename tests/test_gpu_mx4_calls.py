"""Calls of the MX4 operators that the documentation allows: views as outputs, one
container in several calls at once."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4
from tests import mx4_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _values(shape, seed, sigma=1.0):
    """BF16-exact normal values in float64."""
    v = np.random.default_rng(seed).standard_normal(shape) * sigma
    return ref.bf16_to_f64(ref.f64_to_bf16_bits(v))


def _dev(v, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).cuda().to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,R,K", [(2, 1, 32), (3, 20, 160), (5, 33, 544), (1, 17, 64)])
def test_codec_interleaved_matrices(B, R, K, dtype):
    """Matrices whose rows lie between each other's: [R, B, K] memory seen as [B, R, K]."""
    v = _values((R, B, K + 8), B + R + K)
    rows = _dev(v, TYPES[dtype])
    x = rows[:, :, :K].transpose(0, 1)
    q = mx4.mx4_quantize(x)
    want = ref.rounded(v[:, :, :K])
    rows.fill_(7.0)
    assert mx4.mx4_dequantize(q, out=x) is x
    full = np.full(v.shape, 7.0)
    full[:, :, :K] = want
    assert np.array_equal(rows.float().cpu().numpy().astype(np.float64), full)


def _moe(T, H, I, E, seed):
    logits = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E))
                              .astype(np.float32)).cuda()
    return (_dev(_values((T, H), seed + 1)), logits,
            mx4.mx4_quantize(_dev(_values((E, 2 * I, H), seed + 2, 0.05))),
            mx4.mx4_quantize(_dev(_values((E, H, I), seed + 3, 0.05))))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 160, 96, 9, 4), (32, 64, 32, 20, 3), (40, 96, 64, 12, 5),
                                       (128, 64, 96, 5, 5)])
def test_moe_stays_within_its_workspace(T, H, I, E, k, out):
    x, logits, w13, w2 = _moe(T, H, I, E, 7)
    need = mx4.mx4_moe_workspace_bytes(T, H, I, E, k, TYPES[out])
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    y = mx4.mx4_moe(x, logits, w13, w2, k, out_dtype=TYPES[out], workspace=room[:need])
    assert bool((room[need:] == 0xA5).all())
    assert torch.equal(y, mx4.mx4_moe(x, logits, w13, w2, k, out_dtype=TYPES[out]))


@pytest.mark.parametrize("M,N,K", [(1, 1000, 512), (40, 300, 17408), (200, 3000, 160)])
def test_one_weight_in_two_products_at_once(M, N, K):
    """Two streams, one container, workspaces of their own: every result is the eager one."""
    wq = mx4.mx4_quantize(_dev(_values((N, K), 1, 0.02)))
    xs = [_dev(_values((M, K), 2 + i)) for i in range(2)]
    want = [(mx4.mx4_gemm(x, wq), mx4.mx4_gemm(mx4.mx4_quantize(x), wq)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((mx4.mx4_gemm(xs[i], wq),
                               mx4.mx4_gemm(mx4.mx4_quantize(xs[i]), wq)))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y[0], want[i][0]) and torch.equal(y[1], want[i][1])


@pytest.mark.parametrize("T,H,I,E,k", [(2, 160, 96, 9, 4), (40, 96, 1056, 12, 5)])
def test_one_expert_weight_in_two_layers_at_once(T, H, I, E, k):
    _, _, w13, w2 = _moe(T, H, I, E, 20)
    xs = [_moe(T, H, I, E, 30 + i)[:2] for i in range(2)]
    want = [mx4.mx4_moe(x, l, w13, w2, k) for x, l in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mx4.mx4_moe(*xs[i], w13, w2, k))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
