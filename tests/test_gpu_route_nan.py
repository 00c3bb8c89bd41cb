"""What routing chooses where scores are NaN: the choice that include/mx4_route.h states,
and that of the 64-bit form."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4
from tests import step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _logits():
    l = np.random.default_rng(4).standard_normal((8, 40))
    l[0, 37] = NAN
    l[1, [12, 33]] = NAN
    l[2, 25] = INF
    l[3, [3, 30]] = INF, NAN
    l[4, 0:9] = -INF
    l[4, 20] = NAN
    l[5, 35] = -NAN
    l[6] = NAN
    return l.astype(np.float32).astype(np.float64)


def _dev(v):
    return torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).cuda()


def _route(l, k, **kw):
    e, s = mx4.mx4_route(_dev(l), k, **kw)
    return e.cpu().numpy(), s.cpu().numpy()


BIAS = np.linspace(-0.5, 0.5, 40).astype(np.float32)


@pytest.mark.parametrize("renorm", [True, False])
def test_softmax_with_a_bias_takes_the_lowest(renorm):
    e, s = _route(_logits(), 4, bias=_dev(BIAS), renormalize=renorm)
    for t in (0, 1, 2, 3, 5, 6):
        assert list(e[t]) == [0, 1, 2, 3] and np.isnan(s[t]).all(), t
    assert list(e[4]) == [9, 10, 11, 12] and np.isnan(s[4]).all()
    assert not np.isnan(s[7]).any()


@pytest.mark.parametrize("renorm", [True, False])
def test_softmax_groups_of_two_terms_take_the_lowest(renorm):
    """8 groups of 5, two of them kept: 0 and 1 (in row 4 the first that holds an expert,
    1 with its last, and 2); in them the order of the logits."""
    l = _logits()
    e, s = _route(l, 2, groups=8, kept_groups=2, group_terms=2, renormalize=renorm)
    for t in (0, 1, 2, 3, 5, 6):
        want = sorted(range(10), key=lambda i: (not np.isnan(l[t, i]), -l[t, i], i))[:2]
        assert list(e[t]) == want and np.isnan(s[t]).all(), t
    assert set(e[4]) <= {9, 10, 11, 12, 13, 14}


@pytest.mark.parametrize("kw", [dict(), dict(groups=8, kept_groups=3),
                                dict(scores="sigmoid"), dict(scores="sigmoid", groups=8, kept_groups=3),
                                dict(scores="sigmoid", groups=8, kept_groups=1, group_terms=2)])
def test_elsewhere_a_nan_logit_comes_first(kw):
    """Ranks are logits, or scores of each expert by itself."""
    l = _logits()
    for bias in (None, BIAS):
        if bias is not None and kw.get("scores") != "sigmoid":
            continue
        e, s = _route(l, 4, bias=None if bias is None else _dev(bias), renormalize=False, **kw)
        assert e[0, 0] == 37 and e[3, 0] == 30 and e[4, 0] == 20 and e[5, 0] == 35
        assert e[1, 0] == 12 and np.isnan(s[[0, 1, 3, 4, 5, 6], 0]).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bias", ["none", "plain", "nan"])
@pytest.mark.parametrize("groups,kept,terms", [(1, 1, 1), (8, 3, 1), (8, 3, 2), (4, 1, 2), (20, 7, 2)])
def test_as_the_64_bit_form(scores, renorm, bias, groups, kept, terms):
    l = _logits()
    b = None if bias == "none" else BIAS.copy()
    if bias == "nan":
        b[[17, 39]] = NAN
    e, s = _route(l, 6, scores=scores, bias=None if b is None else _dev(b), groups=groups,
                  kept_groups=kept, group_terms=terms, renormalize=renorm)
    we, ws = ref.route(l, 6, scores, b, groups, kept, terms, renorm)
    assert np.array_equal(e, we)
    assert np.array_equal(np.isnan(s), np.isnan(ws))
    fin = ~np.isnan(ws)
    assert np.all(np.abs(s - ws)[fin] <= np.abs(ws[fin]) * 2.0 ** -24 * (1 + 1e-6) + 2.0 ** -150)
