"""A matrix without columns is refused by name (its dequantization divided by their number)."""
from __future__ import annotations

import pytest
import torch

from quantized_routed_expert_router_amd import mx


def _empty(device):
    return mx.MxMatrix(torch.zeros((4, 0), dtype=torch.uint8, device=device),
                       torch.zeros((4, 0), dtype=torch.uint8, device=device))


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_no_columns(device):
    m, x = _empty(device), torch.zeros((4, 0), device=device)
    for call in (lambda: mx.dequantize(m), lambda: mx.linear(x, m), lambda: mx.linear(m, m), lambda: mx.quantize(x)):
        with pytest.raises(ValueError, match="0 columns"):
            call()
