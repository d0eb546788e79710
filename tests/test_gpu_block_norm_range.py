"""The norms between two blocks up to the magnitudes that include/ep.h allows: a row's sums of
squares and products stay below 2^128."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref
from test_gpu_block_norm import BF16, F32, check_backward, check_forward, inputs, rand

pytestmark = pytest.mark.gpu


def signs(gen, T, H):
    return (torch.randint(0, 2, (T, H), generator=gen, device="cuda") * 2 - 1).float()


@pytest.mark.parametrize("H", [8, 1024, 4104, 7168, 16384])
def test_rows_of_the_largest_magnitude(ep, H):
    s = inputs(3, H, "none", F32, F32, seed=31)
    top = 2.0 ** 63.9 / H ** 0.5
    x, y = signs(s["gen"], 3, H) * top, (signs(s["gen"], 3, H) * top * 0.99).to(BF16)
    r = ep.block_norm(x, pre_weight=s["pre"])
    check_forward(r, x, None, None, None, s["pre"], 1.0, 1e-6)
    kind = dict(post_weight=s["post"], pre_weight=s["pre"])
    r = ep.block_norm(s["x"], y, **kind)
    check_forward(r, s["x"], y, None, s["post"], s["pre"], 1.0, 1e-6)
    dz, dh = rand(s["gen"], 3, H), rand(s["gen"], 3, H, dtype=BF16)
    g = ep.block_norm_backward(dz, dh, x, s["y"], **kind)
    check_backward(g, dz, dh, x, s["y"], None, s["post"], s["pre"], 1.0, 1e-6)
    g = ep.block_norm_backward(dz, dh, s["x"], y, **kind)
    check_backward(g, dz, dh, s["x"], y, None, s["post"], s["pre"], 1.0, 1e-6)
