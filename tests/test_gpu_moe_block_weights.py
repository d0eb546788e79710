"""GPU: the gradients of the experts' weights that examples/moe_block.py makes, against automatic
differentiation in 64 bits."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref
from test_gpu_moe_block import BF16, F32, F64, example, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,stream", [(48, F32), (130, BF16), (3, BF16)])
def test_gradients_of_the_experts_weights(ep, example, tokens, stream):  # noqa: F811
    # what the allocator hands out again: a row that nothing wrote would show
    torch.full((1 << 26,), float("nan"), dtype=BF16, device="cuda")
    b = example.MoEBlock(512, 256, 8, 2, seed=3)
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((tokens, 512), generator=gen, device="cuda").to(stream)
    dz = torch.randn((tokens, 512), generator=gen, device="cuda").to(stream)
    dh = torch.randn((tokens, 512), generator=gen, device="cuda").to(BF16)
    _, _, saved = b.forward(x)
    _, grads, _ = b.backward(dz, dh, saved)
    idx = saved[3]

    w13, w2 = (v.to(F64).requires_grad_(True) for v in (b.w13, b.w2))

    def norm(v, weight):
        return v / ref.rms(v, 1e-6) * weight.to(F64)

    x64 = x.to(F64)
    h0 = norm(x64, b.before)
    w = torch.softmax((h0 @ b.router.to(F64).t()).gather(1, idx), 1)
    g, u = torch.einsum("tknh,th->tkn", w13[idx], h0).chunk(2, dim=2)
    a = g * torch.sigmoid(g) * u * w[..., None]
    y = torch.einsum("tkhn,tkn->th", w2[idx], a)
    z = x64 + b.scale * b.gate.to(F64) * norm(y, b.post)
    want = torch.autograd.grad((z * dz.to(F64)).sum() + (norm(z, b.after) * dh.to(F64)).sum(), [w13, w2])
    # bf16 roundings, half a step each: h, logits, gate_up, the activation, its product, y and z as they are
    # saved, dy, da, dgate_up and the weights' product; gate_up besides in E4M3, two roundings of 2^-4
    step = ref.half_step(BF16)
    near(grads["w2"], want[1], 11 * step, "w2")
    near(grads["w13"], want[0], 2 * 2.0 ** -4 + 11 * step, "w13")
    for e in range(8):
        if not (idx == e).any():
            assert not grads["w2"][e].any() and not grads["w13"][e].any()
