"""The calls of a verify step together, as a program makes them: norm and 8-bit
activations, products, routing, expert layer, the head's product and the
verification; the same on two streams and in a captured graph."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import draft, mx4, mx8, w12
from tests import mx4_ref, step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Step:
    """One layer and the head, on a block of D + 1 tokens for each of B sequences."""

    def __init__(self, B=2, D=3, H=256, I=96, E=12, k=3, V=1000, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)

        self.B, self.D, self.V, self.k = B, D, V, k
        M = B * (D + 1)
        self.x, self.stream = normal(M, H), normal(M, H)
        self.n1, self.n2, self.n3 = (1 + 0.1 * normal(H, sigma=1.0) for _ in range(3))
        self.wo = mx4.mx4_quantize(normal(H, H, sigma=0.06))
        self.router = w12.pack(normal(E, H, sigma=0.1), exceptions=True)[0]
        self.bias = 0.1 * torch.randn(E, generator=g, device="cuda")
        self.w13 = mx4.mx4_quantize(normal(E, 2 * I, H, sigma=0.06))
        self.w2 = mx4.mx4_quantize(normal(E, H, I, sigma=0.1))
        self.head = w12.pack(normal(V, H, sigma=0.15), exceptions=True)[0]
        self.drafts = torch.randint(0, V, (B, D), generator=g, device="cuda", dtype=torch.int32)
        self.uniforms = torch.rand((B, D + 1), generator=g, device="cuda")
        self.tau = torch.full((B,), 0.8, device="cuda")

    def run(self, keep=None):
        h, stream = mx8.mx8_rms_norm(self.x, self.n1, residual=self.stream)
        o = mx8.mx8_gemm(h, self.wo)                                    # fp32
        h2, stream = mx8.mx8_rms_norm(o, self.n2, residual=stream, out_dtype=torch.bfloat16)
        logits = w12.w12_gemm(h2, self.router)
        experts, shares = mx4.mx4_route(logits, self.k, scores="sigmoid", bias=self.bias, groups=4,
                                        kept_groups=2, group_terms=2, scale=1.5)
        y = mx4.mx4_moe_routed(h2, experts, shares, self.w13, self.w2)
        h3, stream = mx8.mx8_rms_norm(y, self.n3, residual=stream, out_dtype=torch.bfloat16)
        words = w12.w12_gemm(h3, self.head)
        out = draft.draft_verify(words.view(self.B, self.D + 1, self.V), self.drafts, self.uniforms,
                                 temperature=self.tau)
        if keep is not None:
            keep.update(h=h, o=o, h2=h2, logits=logits, experts=experts, shares=shares, y=y, h3=h3,
                        stream=stream, words=words)
        return out


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def test_step_against_64_bits():
    """Every call on what the one before gave it."""
    s = Step()
    kept = {}
    tokens, accepted = s.run(kept)
    y, _ = ref.norm(_host(s.x), _host(s.stream), _host(s.n1), 1e-6, True)
    h = _host(mx8.mx8_dequantize(kept["h"], torch.float32))
    # half a step of E4M3, or half the smallest step that is kept, 1/4
    unit = np.ldexp(1.0, kept["h"].block_scales.cpu().numpy().astype(int) - 127).repeat(32, 1)
    over = np.maximum(np.abs(y) - 448 * unit, 0)
    assert np.all(np.abs(h - y) <= np.abs(y) * (2.0 ** -4 + 1e-6) + unit * 2.0 ** -3 + over)
    w = _host(mx4.mx4_dequantize(s.wo, torch.float32))
    want, tol = mx4_ref.matmul(h, w)
    mx4_ref.assert_close(_host(kept["o"]), want, tol, "f32", "product")
    e, p = ref.route(_host(kept["logits"]), s.k, "sigmoid", _host(s.bias), 4, 2, 2, True, 1.5)
    assert np.array_equal(kept["experts"].cpu().numpy(), e)
    assert np.allclose(_host(kept["shares"]), p, rtol=2.0 ** -23, atol=0)
    want, n = ref.verify(_host(kept["words"]).reshape(s.B, s.D + 1, s.V), s.drafts.cpu().numpy(),
                         s.uniforms.cpu().numpy(), None, None, s.tau.cpu().numpy())
    assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(accepted.cpu().numpy(), n)


def test_step_twice_is_the_same_bits():
    s = Step(seed=1)
    a, b = {}, {}
    ta, tb = s.run(a), s.run(b)
    for name in a:
        if name == "h":
            assert torch.equal(a[name].values.view(torch.uint8), b[name].values.view(torch.uint8))
            assert torch.equal(a[name].scales, b[name].scales)
        else:
            assert torch.equal(a[name], b[name]), name
    assert torch.equal(ta[0], tb[0]) and torch.equal(ta[1], tb[1])


def test_steps_on_two_streams_at_once():
    steps = [Step(seed=2), Step(B=3, D=4, seed=3)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(steps):
            with torch.cuda.stream(streams[i]):
                got[i].append(s.run())
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o in outs:
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_step_in_a_graph():
    """Replayed over new inputs, with eager calls between."""
    s = Step(seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    kept = {}
    with torch.cuda.graph(graph):
        out = s.run(kept)
    for seed in range(5, 9):
        other = Step(seed=seed)
        s.x.copy_(other.x)
        s.uniforms.copy_(other.uniforms)
        s.drafts.copy_(other.drafts)
        graph.replay()
        torch.cuda.synchronize()
        again = {}
        want = s.run(again)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert torch.equal(kept["words"], again["words"]) and torch.equal(kept["y"], again["y"])


def test_single_token_step():
    s = Step(B=1, D=0, seed=9)
    tokens, accepted = s.run()
    assert tokens.shape == (1, 1) and 0 <= int(tokens) < s.V and int(accepted) == 0
