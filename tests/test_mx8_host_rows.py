"""Rows of MX8 in host memory are refused as any host tensor is."""
import pytest
import torch

from lossless_bit_weight_amd import mx8


def _made():
    return mx8.empty_mx8(2, 64, device="cpu")


def _given():
    return mx8.MX8Tensor(torch.zeros(2, 64, dtype=torch.uint8).view(mx8.VALUES),
                         torch.zeros(2, 16, dtype=torch.uint8))


@pytest.mark.parametrize("rows", [_made, _given])
def test_host_rows_are_refused(rows):
    q = rows()
    assert q.shape == (2, 64) and q.values.shape == (2, 64) and q.scales.shape == (2, 16)
    with pytest.raises(ValueError, match="GPU"):
        q.parts("q")
    with pytest.raises(ValueError, match="GPU"):
        mx8.mx8_dequantize(q)
    with pytest.raises(ValueError, match="GPU"):
        mx8.mx8_dequantize(q[:1])
