"""quantize_w4 on the CPU: its refusals."""
from __future__ import annotations

import pytest
import torch

import combine_get_dispatch_04_gb300 as ep


@pytest.mark.parametrize("shape,group", [((2, 8, 128), 0), ((2, 8, 128), -32), ((2, 8, 128), 16),
                                         ((2, 8, 100), 32), ((8, 128), 128)])
def test_refusals(shape, group):
    with pytest.raises(ep.EPError):
        ep.quantize_w4(torch.zeros(shape), group)
