"""GPU: a whole block as examples/moe_block.py runs it, decoding and training,
against 64 bits and automatic differentiation."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
norm = torch.linalg.norm


@pytest.fixture(scope="module")
def example(ep):
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def near(got, want, bound, what):
    off = float(norm(got.to(F64) - want) / norm(want))
    assert off <= bound, f"{what}: {off}"


def rms_norm(v, weight):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * weight.to(F64)


@pytest.mark.parametrize("tokens,stream", [(1, BF16), (6, F32), (16, BF16)])
def test_decoding(ep, example, tokens, stream):
    blocks = [example.MoEBlock(512, 256, 16, 4, seed=i) for i in range(3)]
    for b in blocks:
        b.quantise()
    gen = torch.Generator("cuda").manual_seed(1)
    start = torch.randn((tokens, 512), generator=gen, device="cuda").to(stream)
    x = start.clone()
    h = ep.block_norm(x, pre_weight=blocks[0].before).h
    for b in blocks:
        # the block in 64 bits from its own inputs; the router's choice is the library's
        z0, h0 = x.to(F64), h.clone()
        out, idx, w = ep.layer_w4(h0, h0 @ b.router.t(), b.up4, b.down4, b.topk)
        y, _ = ref.layer(h0, idx, w, b.up4, b.down4)
        z = z0 + b.scale * b.gate.to(F64) * rms_norm(y, b.post)
        h = b.decode(x, h)
        # y rounded, z rounded (its own error relative to z), h rounded
        near(x, z, 2 * ref.half_step(BF16), "z")
        near(h, rms_norm(z, b.after), 3 * ref.half_step(BF16), "h")
    eager, eager_h = x.clone(), h.clone()

    def step():
        x.copy_(start)
        v = ep.block_norm(x, pre_weight=blocks[0].before).h
        for b in blocks:
            v = b.decode(x, v)
        return v

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, eager) and torch.equal(got, eager_h)


@pytest.mark.parametrize("tokens,stream", [(48, F32), (130, BF16)])
def test_training(ep, example, tokens, stream):
    b = example.MoEBlock(512, 256, 8, 2, seed=3)
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn((tokens, 512), generator=gen, device="cuda").to(stream)
    dz = torch.randn((tokens, 512), generator=gen, device="cuda").to(stream)
    dh = torch.randn((tokens, 512), generator=gen, device="cuda").to(BF16)
    z, h, saved = b.forward(x)
    dx, grads, _ = b.backward(dz, dh, saved)
    idx = saved[3]

    leaf = {n: getattr(b, n).to(F64).requires_grad_(True)
            for n in ("before", "post", "after", "gate", "router")}
    x64 = x.to(F64).requires_grad_(True)
    h0 = x64 / torch.sqrt(x64.square().mean(1, keepdim=True) + 1e-6) * leaf["before"]
    w = torch.softmax((h0 @ leaf["router"].t()).gather(1, idx), 1)  # renormalised
    p = torch.einsum("tknh,th->tkn", b.w13.to(F64)[idx], h0)
    g, u = p.chunk(2, dim=2)
    a = g * torch.sigmoid(g) * u * w[..., None]
    y = torch.einsum("tkhn,tkn->th", b.w2.to(F64)[idx], a)
    n = y / torch.sqrt(y.square().mean(1, keepdim=True) + 1e-6) * leaf["post"]
    z64 = x64 + b.scale * leaf["gate"] * n
    h64 = z64 / torch.sqrt(z64.square().mean(1, keepdim=True) + 1e-6) * leaf["after"]
    want = torch.autograd.grad((z64 * dz.to(F64)).sum() + (h64 * dh.to(F64)).sum(),
                               [x64] + list(leaf.values()))
    # bf16 roundings on the way, half a step each: h, logits, gate_up, a, y, z, h
    step = ref.half_step(BF16)
    near(z, z64.detach(), 7 * step, "z")
    near(h, h64.detach(), 7 * step, "h")
    # and back: two roundings to E4M3 (g and u; half a step is 2^-4), and of bf16 those of the saved
    # values above and of dy, its rows' product, dgate_up, its product, the combine and dx
    bound = 2 * 2.0 ** -4 + 14 * step
    near(dx, want[0], bound, "dx")
    for name, value in zip(leaf, want[1:]):
        near(grads[name], value, bound, name)
