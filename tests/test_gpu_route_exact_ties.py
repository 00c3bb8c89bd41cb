"""Routing by sigmoid where scores are exactly 0, 1/2 and 1 and biases multiples of 1/8:
ranks of different experts are exactly alike, and the lowest goes first."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4
from tests import step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

SCORES = {0.0: 0.5, -0.0: 0.5, 60.0: 1.0, 1e30: 1.0, np.inf: 1.0, -800.0: 0.0, -1e30: 0.0}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _case(T, E, seed):
    rng = np.random.default_rng(seed)
    l = rng.choice(list(SCORES), (T, E)).astype(np.float32)
    return l, (rng.integers(-4, 5, E) / 8).astype(np.float32)


def _route(l, k, b, **kw):
    e, s = mx4.mx4_route(torch.from_numpy(l).cuda(), k, scores="sigmoid",
                         bias=None if b is None else torch.from_numpy(b).cuda(), **kw)
    return e.cpu().numpy(), s.cpu().numpy()


def test_two_experts():
    l = np.array([[0.0, 60.0], [60.0, 0.0]], np.float32)
    e, s = _route(l, 2, np.array([0.25, -0.25], np.float32), renormalize=False)
    assert e.tolist() == [[0, 1], [0, 1]] and s.tolist() == [[0.5, 1.0], [1.0, 0.5]]


@pytest.mark.parametrize("E,k", [(8, 8), (64, 6), (130, 32), (256, 8), (1000, 32)])
def test_ranks(E, k):
    l, b = _case(40, E, E)
    score = {float(np.float32(v)): s for v, s in SCORES.items()}
    s = np.vectorize(score.get)(l.astype(np.float64))
    want = np.argsort(-(s + b), axis=1, kind="stable")[:, :k]
    e, got = _route(l, k, b, renormalize=False)
    assert np.array_equal(e, want)
    assert np.array_equal(got, np.take_along_axis(s, want, 1).astype(np.float32))


@pytest.mark.parametrize("E,groups,kept,terms", [(64, 8, 3, 1), (64, 8, 3, 2), (256, 8, 4, 2),
                                                 (96, 3, 1, 2), (320, 64, 20, 2), (40, 20, 7, 2)])
@pytest.mark.parametrize("bias", [True, False])
def test_groups(E, groups, kept, terms, bias):
    l, b = _case(40, E, E + groups)
    b = b if bias else None
    e, s = _route(l, 6, b, groups=groups, kept_groups=kept, group_terms=terms)
    with np.errstate(over="ignore"):
        we, ws = ref.route(l.astype(np.float64), 6, "sigmoid", b, groups, kept, terms)
    # (ranks without a bias are logits: 60, 1e30 and inf are different ones)
    assert np.array_equal(e, we)
    assert np.all(np.abs(s - ws) <= np.abs(ws) * 2.0 ** -24 * (1 + 1e-6))
