"""tests/mx8_cases.py's operands, without a GPU: their sums are exact in fp32, and would
not be if the matrix units dropped one bit more."""
import numpy as np
import pytest

from tests import mx4_ref, step_ref
from tests.mx8_cases import SHAPES, edges, summed_in_eights


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_edges_are_held_and_their_sums_too(M, N, K):
    x, w = edges(min(M, 24), min(N, 24), K)
    assert np.array_equal(step_ref.decode8(*step_ref.encode8(x)), x)
    assert np.array_equal(mx4_ref.rounded(w), w)
    assert np.array_equal(np.rint(4 * x), 4 * x) and np.array_equal(np.rint(2 * w), 2 * w)
    assert (np.abs(x) @ np.abs(w).T).max() < 2.0 ** 21      # sums in any order


@pytest.mark.parametrize("M,N,K", [(17, 19, 1056), (5, 40, 4128), (40, 40, 32)])
def test_one_bit_less_would_show(M, N, K):
    x, w = edges(M, N, K)
    want = x @ w.T
    assert np.array_equal(summed_in_eights(x, w, 13), want)
    off = (summed_in_eights(x, w, 12) != want).mean()
    assert off > (0.8 if K > 1000 else 0.1)
