"""The gradient of the norms between two blocks where the block's output holds infinities or
NaN: without a norm after the block, the gradient of that output does not depend on it."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref
from test_gpu_block_norm import BF16, F32, SUM, check, inputs, rand

pytestmark = pytest.mark.gpu


# 640 and 7168: the kernel of a vector a thread; 7176: the one of longer rows
@pytest.mark.parametrize("H", [640, 7168, 7176])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_dy_without_a_norm_after_the_block(ep, H, gate, pre, stream):
    T, scale = 7, 0.37
    s = inputs(T, H, gate, stream, F32, post=False, pre=pre, seed=11)
    dz = rand(s["gen"], T, H, dtype=stream)
    dh = rand(s["gen"], T, H, dtype=BF16) if pre else None
    want, mag = ref.block_norm_grad(dz, dh, s["x"], s["y"], s["gate"], None, s["pre"], scale, 1e-6)
    clean = ep.block_norm_backward(dz, dh, s["x"], s["y"], gate=s["gate"], pre_weight=s["pre"],
                                   scale=scale)
    y = s["y"].clone()
    y[0, 0] = float("inf")
    y[2, H - 1] = float("-inf")
    y[5, 3] = float("nan")
    r = ep.block_norm_backward(dz, dh, s["x"], y, gate=s["gate"], pre_weight=s["pre"], scale=scale)
    for name in ("dx", "dy"):
        got = getattr(r, name)
        # a row's factors: 4 SUM of the terms' magnitudes, and one rounding of the output
        check(got, want[name], 4 * SUM * mag[name] + ref.half_step(got.dtype) * want[name].abs() + 1e-38, name)
        assert torch.equal(got, getattr(clean, name)), name
    if pre:
        assert torch.equal(r.dpre_weight, clean.dpre_weight)
    if gate in ("token", "full"):  # which depends on y, in the token's row alone
        keep = [1, 3, 4, 6]
        assert torch.equal(r.dgate[keep], clean.dgate[keep])


@pytest.mark.parametrize("H", [640, 7176])
def test_a_block_output_that_nothing_needs(ep, H):
    """Neither gate nor norm: y may be given, and is not part of any gradient."""
    s = inputs(3, H, "none", BF16, F32, post=False, seed=12)
    dz, dh = rand(s["gen"], 3, H, dtype=BF16), rand(s["gen"], 3, H, dtype=BF16)
    y = torch.full((3, H), float("nan"), dtype=BF16, device="cuda")
    for kind in (dict(pre_weight=s["pre"]), dict()):
        d = dh if kind else None
        want = ep.block_norm_backward(dz, d, s["x"], None, scale=2.0, **kind)
        got = ep.block_norm_backward(dz, d, s["x"], y, scale=2.0, **kind)
        assert torch.equal(got.dx, want.dx) and torch.equal(got.dy, want.dy)
        assert not got.dy.isnan().any()
