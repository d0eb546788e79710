"""GPU: the router, the experts' products and the gradients together, as
examples/moe_layer.py runs them, and offsets beyond 32 bits.

Serving step: three bf16 roundings on the way (h, y, out), each 2^-9 of the
value, and as much again for everything in float32; the rows enter as the E4M3
codes that the dispatch made, so those are not an error here."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(ep):
    spec = importlib.util.spec_from_file_location(
        "moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def weights64(W):
    return ref.dequantize_w4(W.q.cpu().numpy(), W.scales.double().cpu().numpy(),
                             None if W.zeros is None else W.zeros.cpu().numpy())


def layer64(ep, layer, x):
    """The layer on the rows that the dispatch makes, from there on in 64 bits."""
    logits = torch.mm(x, layer.gate.t().to(x.dtype))
    idx, w = ep.route(logits, layer.topk, bias=layer.bias, **layer.route_args)
    cap = layer.capacity or x.shape[0]
    L = ep.ll_get_dispatch_layout(idx, layer.experts, 1, cap)
    d = ep.ll_dispatch(x, L, use_fp8=True)
    rows = (d.recv_x.view(torch.float8_e4m3fn).double().cpu().numpy()
            * np.repeat(d.recv_scales.double().cpu().numpy(), 128, 1))
    up, down = weights64(layer.up), weights64(layer.down)
    slot, ws = L.ll_slot.cpu().numpy(), w.double().cpu().numpy()
    out = np.zeros(tuple(x.shape))
    inter = down.shape[2]
    for t in range(slot.shape[0]):
        for k in range(slot.shape[1]):
            s = slot[t, k]
            if s >= 0:
                p = up[s // cap] @ rows[s]
                out[t] += ws[t, k] * (down[s // cap] @ (ref.silu(p[:inter]) * p[inter:]))
    return out


@pytest.mark.parametrize("tokens,experts,topk,groups", [(1, 8, 2, 1), (40, 16, 4, 4), (150, 4, 2, 1)])
def test_serving_step_eager_and_in_a_graph(ep, example, tokens, experts, topk, groups):
    """The graph's replays follow inputs that are written in place."""
    layer = example.MoELayer(256, 128, experts, topk, groups=groups,
                             topk_groups=max(1, groups // 2), seed=tokens)
    gen = torch.Generator("cuda").manual_seed(tokens)
    make = lambda: torch.randn((tokens, 256), generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x = make()
    out = layer(x)
    want = layer64(ep, layer, x)
    assert np.linalg.norm(out.double().cpu().numpy() - want) <= 4 * 2.0 ** -9 * np.linalg.norm(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = layer(x)
    for _ in range(3):
        x.copy_(make())
        graph.replay()
        assert torch.equal(captured, layer(x))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients_of_a_step(ep, example, score):
    """From the output's gradient to the logits, against automatic
    differentiation in 64 bits.  dweights are float32 sums of 256 products
    (2^-24 * 256 of their magnitude at most, some 2^-20 in norm), the router's
    gradient adds a few roundings: 2^-16.  dy is rounded to bf16 once."""
    T, H, E, K = 48, 256, 16, 4
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    dout = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    idx, w = ep.route(logits, K, score=score)
    L = ep.ll_get_dispatch_layout(idx, E, 1, T)
    rows = L.num_rows
    y = torch.randn((rows, H), generator=gen, device="cuda").to(torch.bfloat16)
    dy, dlogits = example.router_and_combine_gradients(logits, idx, w, y, L, dout, score=score)

    l64 = logits.double().requires_grad_()
    y64 = y.double().requires_grad_()
    s = torch.sigmoid(l64) if score == "sigmoid" else torch.softmax(l64, 1)
    u = s.gather(1, idx)
    u = u / u.sum(1, keepdim=True)
    out = (u[..., None] * y64[L.ll_slot.long()]).sum(1)
    out.backward(dout.double())
    got, want = dlogits.double(), l64.grad
    assert torch.linalg.norm(got - want) <= 2.0 ** -16 * torch.linalg.norm(want)
    assert torch.linalg.norm(dy.double() - y64.grad) <= 2.0 ** -9 * torch.linalg.norm(y64.grad)
    # the gradient of the dispatch is the combine without weights
    dx = ep.ll_combine(dy, None, L).double()
    want = dy.double()[L.ll_slot.long()].sum(1)
    assert torch.linalg.norm(dx - want) <= 2.0 ** -8 * torch.linalg.norm(want)


# E, capacity, rows of the last expert: its rows of x and of y, or its codes,
# start beyond 2^31 elements
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("E,cap,rows", [(8, 40000, 5), (8, 40000, 200), (72, 16, 3), (72, 16, 12)])
def test_experts_beyond_32_bits(ep, E, cap, rows, fp8):
    I = N = 8192
    gen = torch.Generator("cuda").manual_seed(E + rows)
    e = E - 1
    assert e * cap * I > 2 ** 31 or e * N * I // 2 > 2 ** 31
    q = torch.randint(0, 256, (E, N, I // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = (torch.rand((E, N, I // 128), device="cuda", generator=gen) + 0.5).to(torch.bfloat16)
    count = torch.zeros(E, dtype=torch.int32, device="cuda")
    count[e] = rows
    live = torch.randn((rows, I), device="cuda", generator=gen)
    out = torch.full((E * cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
    if fp8:
        x = torch.zeros((E * cap, I), dtype=torch.uint8, device="cuda")
        x[e * cap:e * cap + rows] = live.to(torch.float8_e4m3fn).view(torch.uint8)
        xs = torch.ones((E * cap, I // 128), device="cuda")
        x64 = live.to(torch.float8_e4m3fn).double()
    else:
        x = torch.zeros((E * cap, I), dtype=torch.bfloat16, device="cuda")
        x[e * cap:e * cap + rows] = live.to(torch.bfloat16)
        xs, x64 = None, live.to(torch.bfloat16).double()
    ep.ll_experts_w4(x, ep.W4Weights(q, scales), ep.LLLayout(None, count, None, E, 1, cap),
                     x_scales=xs, out=out)
    codes = torch.stack((q[e] & 15, q[e] >> 4), -1).reshape(N, I).double() - 8
    want = x64 @ (codes * scales[e].double().repeat_interleave(128, 1)).t()
    got = out[e * cap:e * cap + rows].double()
    assert torch.linalg.norm(got - want) <= 2.0 ** -8 * torch.linalg.norm(want)
    assert bool((out[:e * cap] == 7).all()) and bool((out[e * cap + rows:] == 7).all())


def test_gradients_beyond_32_bits(ep):
    """Rows of y beyond 2^31 elements, and logits beyond 2^31 elements."""
    H, rows, T, K = 8192, 280000, 3, 2
    gen = torch.Generator("cuda").manual_seed(9)
    y = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([[rows - 1, 0], [rows - 2, rows - 3], [-1, 270000]], dtype=torch.int32,
                        device="cuda")
    named = slot[slot >= 0].long()
    y[named] = torch.randn((len(named), H), device="cuda", generator=gen).to(torch.bfloat16)
    dout = torch.randn((T, H), device="cuda", generator=gen).to(torch.bfloat16)
    w = torch.rand((T, K), device="cuda", generator=gen)
    L = ep.LLLayout(slot, torch.zeros(1, dtype=torch.int32, device="cuda"), None, 1, 1, rows)
    dy, dw = ep.ll_combine_backward(dout, y, w, L)
    for t in range(T):
        for k in range(K):
            s = int(slot[t, k])
            if s < 0:
                assert dw[t, k] == 0
                continue
            assert torch.equal(dy[s], (w[t, k] * dout[t].float()).to(torch.bfloat16))
            want = (dout[t].double() * y[s].double()).sum()
            size = (dout[t].double() * y[s].double()).abs().sum()
            assert abs(dw[t, k].double() - want) <= 2.0 ** -16 * size
    del y, dy

    T, E, K = 2 ** 22 + 5, 520, 4
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    logits[-3:] = torch.randn((3, E), device="cuda", generator=gen).to(torch.bfloat16)
    idx, w = ep.route(logits, K)
    last = logits[-3:].float().cpu().numpy()
    want = ref.choose(ref.route_keys(last, "softmax"), K)
    assert np.array_equal(idx[-3:].cpu().numpy(), want)
    assert torch.equal(idx[0].cpu(), torch.arange(K))
    dl = ep.route_backward(torch.ones_like(w) * w, logits, idx)
    want = ref.route_grad(w[-3:].double().cpu().numpy(), last, want, "softmax", True, 1.0)
    got = dl[-3:].double().cpu().numpy()
    assert np.abs(got - want).max() <= 2.0 ** -8 * np.abs(want).max()
