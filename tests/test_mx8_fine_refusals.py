"""Which types take the flag of MX8's fine steps, without a GPU."""
import ctypes

import pytest

from lossless_bit_weight_amd import mx8

A = ctypes.c_void_p(4096)       # never dereferenced: every call here fails or has no rows
FINE = mx8.FINE_STEPS


@pytest.mark.parametrize("t,status", [(FINE, 0), (FINE | 1, 0), (FINE | 2, -4), (FINE | 3, -4),
                                      (2 * FINE, -4), (3 * FINE, -4), (-1, -4), (-FINE, -4)])
def test_quantize_types(t, status):
    assert mx8.lib().mx8_quantize(A, t, 0, 64, 64, A, 64, A, 16, None) == status


@pytest.mark.parametrize("t", [FINE, FINE | 1, FINE | 2])
def test_dequantize_has_no_steps(t):
    assert mx8.lib().mx8_dequantize(A, 64, A, 16, 0, 64, A, t, 64, None) == -4


@pytest.mark.parametrize("t,status", [(FINE | 2, 0), (FINE, -4), (FINE | 1, -4), (FINE | 3, -4),
                                      (2 * FINE | 2, -4), (-1, -4)])
def test_norm_types(t, status):
    assert mx8.lib().mx8_rms_norm(A, 0, 64, None, None, 0, 0, 0, A, 0, 1e-6, 0, 64, A, t, 64, A, 16,
                                  None) == status


@pytest.mark.parametrize("t", [FINE, FINE | 1])
def test_other_types_take_no_flag(t):
    args = [A, 0, 64, A, A, 0, 64, 64, A, 0, 1e-6, 0, 64, A, 2, 64, A, 16, None]
    for i in (1, 5, 9):
        bad = list(args)
        bad[i] = t
        assert mx8.lib().mx8_rms_norm(*bad) == -4
