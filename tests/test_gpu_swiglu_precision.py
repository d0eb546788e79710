"""The gradient of the top-k weights through the gated activation is a float32 output: strongly
negative gates cost it no more than a float32 exponential does."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# One channel of a row counts, so dw is a single product, in units of 2^-24: the exponential 4 (two units
# in the last place), 1 + e 1, its reciprocal 2 (one unit in the last place), e r 1, g s 1, times u 1, times
# dh 1; the zeros of the other channels add exactly.
UNITS = 11


@pytest.mark.parametrize("N", [8, 512, 2048])
@pytest.mark.parametrize("low,high", [(-85.0, -60.0), (-60.0, -20.0), (-20.0, 0.0), (0.0, 85.0)])
def test_weights_gradient_of_wide_gates(ep, N, low, high):
    T, K = 1024, 2
    gen = torch.Generator("cuda").manual_seed(N)
    rows = T * K
    slot = torch.randperm(rows, generator=gen, device="cuda").to(torch.int32).view(T, K)
    L = ep.LLLayout(slot, None, None, rows, 1, 1)
    g = low + (high - low) * torch.rand((rows, N), generator=gen, device="cuda")
    u = torch.randn((rows, N), generator=gen, device="cuda")
    gu = torch.cat((g, u), 1).to(BF16)
    dh = torch.zeros((rows, N), dtype=BF16, device="cuda")
    at = torch.randint(0, N, (rows,), generator=gen, device="cuda")
    dh[torch.arange(rows, device="cuda"), at] = torch.randn(rows, generator=gen, device="cuda").to(BF16)
    w = torch.rand((T, K), generator=gen, device="cuda")
    _, dw = ep.ll_swiglu_backward(dh, gu, L, w)
    _, want, _, mag = ref.swiglu_grad(dh, gu, torch.ones(rows, device="cuda"))
    off = (dw.to(ref.F) - want[slot.long()]).abs() / mag[slot.long()].clamp(min=1e-300)
    assert float(off.max()) <= UNITS * 2.0 ** -24, float(off.max()) * 2.0 ** 24
