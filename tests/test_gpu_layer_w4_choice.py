"""The layer for a few tokens chooses as the router does where the keys differ in their last
bits only: softmax scores plus a bias, whose sum of exponentials has to be added up alike."""
from __future__ import annotations

import pytest
import torch

from test_gpu_layer_w4 import weights

pytestmark = pytest.mark.gpu


# sizes and groups of every tile of the router's choice in registers (two experts to sixteen a lane,
# two lanes to 32), and some that it makes in shared memory
@pytest.mark.parametrize("E,G", [(12, 1), (16, 2), (40, 1), (64, 1), (64, 4), (96, 1), (128, 1), (160, 1),
                                 (160, 32), (256, 1), (256, 8), (300, 1), (512, 1), (512, 32),
                                 (64, 32), (128, 32), (96, 8), (120, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_keys_that_differ_in_their_last_bits(ep, E, G, dtype, renormalize):
    gen = torch.Generator("cuda").manual_seed(E + G)
    K = min(8, E // 2)
    a = weights(ep, gen, E, 64, 32, 32, False)
    b = weights(ep, gen, E, 32, 32, 32, False)
    kind = dict(num_groups=G, topk_groups=max(1, G // 2 + 1) if G > 1 else 1, renormalize=renormalize)
    for _ in range(12):
        logits = (torch.randn((1, E), generator=gen, device="cuda") * 1.5).to(dtype)
        x = torch.randn((1, 32), generator=gen, device="cuda").to(torch.bfloat16)
        # a key is the score's own rounding error
        bias = -torch.softmax(logits.double(), 1)[0].float()
        idx, w = ep.route(logits, K, bias=bias, **kind)
        _, got, gw = ep.layer_w4(x, logits, a, b, K, bias=bias, **kind)
        assert torch.equal(idx, got)
        if renormalize:  # sums of K weights in another order: K roundings on either side
            assert torch.allclose(w, gw, rtol=4 * K * 2.0 ** -24, atol=0.0)
        else:
            assert torch.equal(w, gw)
