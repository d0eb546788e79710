"""GPU: the bounded waits of the experts' products with many rows."""
from __future__ import annotations

import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("step", [0, 2, 4])  # of the first item, and of the block's second one
def test_bounded_wait_reports_timeout_and_recovers(ep, fp8, step):
    """A step of x that block 0 never loads (test hook) makes its waits run out:
    the launch ends by itself with EP_ERRBIT_TIMEOUT, every other block's results
    are there, and the next launch is correct."""
    E, cap, I, N = 10, 40, 384, 4096  # three steps; 32 tiles an expert
    gen = torch.Generator("cuda").manual_seed(step)
    q = torch.randint(0, 256, (E, N, I // 2), dtype=torch.uint8, device="cuda", generator=gen)
    W = ep.W4Weights(q, torch.full((E, N, I // 128), 0.01, device="cuda").to(torch.bfloat16))
    x = torch.randn((E * cap, I), device="cuda", generator=gen)
    xs = torch.ones((E * cap, I // 128), device="cuda") if fp8 else None
    x = x.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(torch.bfloat16)
    L = ep.LLLayout(None, torch.full((E,), cap, dtype=torch.int32, device="cuda"), None, E, 1, cap)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = ep.ll_experts_w4(x, W, L, x_scales=xs, err=err)
    assert int(err.item()) == 0

    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    assert E * 32 > blocks
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    ep.lib().ep_debug_set_experts_stall(step)
    t0 = time.time()
    ep.ll_experts_w4(x, W, L, x_scales=xs, err=err, out=out)
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    assert int(err.item()) == ep.EP_ERRBIT_TIMEOUT
    assert 0.5 < elapsed < 10, elapsed
    got, right = out.reshape(E, cap, 32, 128), want.reshape(E, cap, 32, 128)
    for item in range(E * 32):
        e, tile = divmod(item, 32)
        same = torch.equal(got[e, :, tile], right[e, :, tile])
        assert same == (item % blocks != 0 or (step > 2 and item == 0)), item

    err.zero_()
    again = ep.ll_experts_w4(x, W, L, x_scales=xs, err=err)
    assert int(err.item()) == 0 and torch.equal(again, want)
