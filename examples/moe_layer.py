"""One mixture-of-experts layer out of the library's calls, run on one GPU.

Serving: logits -> route -> expert-major layout -> dispatch (FP8 rows) ->
gate and up projections with SwiGLU -> down projection (4-bit weights) ->
combine, the whole step also captured in a CUDA graph.  Training: the gradients
of the router and of the combine, which with the combine itself (the gradient
of the dispatch) carry a layer's gradient from its output back to the logits
and to the dispatched rows.

    python examples/moe_layer.py [--tokens 64] [--experts 32] [--topk 4] ...
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_get_dispatch_04_gb300 as ep  # noqa: E402


class MoELayer:
    """4-bit experts behind a sigmoid router with a balance bias."""

    def __init__(self, hidden, inter, experts, topk, groups=1, topk_groups=1, capacity=0,
                 group_size=128, device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=gen, device=device)  # noqa: E731
        self.experts, self.topk, self.capacity = experts, topk, capacity
        self.route_args = dict(score="sigmoid", num_groups=groups, topk_groups=topk_groups,
                               scale=1.0)
        self.gate = rand(experts, hidden) / hidden ** 0.5
        self.bias = rand(experts) * 0.01
        self.up = ep.quantize_w4(rand(experts, 2 * inter, hidden) / hidden ** 0.5, group_size)
        self.down = ep.quantize_w4(rand(experts, hidden, inter) / inter ** 0.5, group_size,
                                   zero_points=True)

    def __call__(self, x):
        """[T, H] bfloat16 -> [T, H] bfloat16; enqueued on the current stream."""
        logits = torch.mm(x, self.gate.t().to(x.dtype))
        idx, w = ep.route(logits, self.topk, bias=self.bias, **self.route_args)
        L = ep.ll_get_dispatch_layout(idx, self.experts, 1, self.capacity or x.shape[0])
        rows = ep.ll_dispatch(x, L, use_fp8=True)
        h = ep.ll_experts_w4(rows.recv_x, self.up, L, x_scales=rows.recv_scales, act="swiglu")
        y = ep.ll_experts_w4(h, self.down, L)
        return ep.ll_combine(y, w, L)


def router_and_combine_gradients(logits, idx, w, y, layout, dout, *, score="sigmoid"):
    """From the gradient of the layer's output to those of the experts' outputs
    (dy, row for row of y) and of the router's logits."""
    dy, dw = ep.ll_combine_backward(dout, y, w, layout)
    return dy, ep.route_backward(dw, logits, idx, score=score)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 64), ("hidden", 2048), ("inter", 1024), ("experts", 32),
                        ("topk", 4), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = MoELayer(a.hidden, a.inter, a.experts, a.topk)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    out = layer(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = layer(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, captured)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        graph.replay()
    stop.record()
    torch.cuda.synchronize()
    print(f"serving step, {a.tokens} tokens: {start.elapsed_time(stop) / a.steps * 1e3:.1f} us "
          "(CUDA-graph replay)")

    logits = torch.randn(a.tokens, a.experts, device="cuda")
    idx, w = ep.route(logits, a.topk, score="sigmoid")
    L = ep.ll_get_dispatch_layout(idx, a.experts, 1, a.tokens)
    y = ep.ll_dispatch(x, L).recv_x  # experts that hand their rows back
    dy, dlogits = router_and_combine_gradients(logits, idx, w, y, L, torch.ones_like(x))
    dx = ep.ll_combine(dy, None, L)  # the gradient of the dispatch
    torch.cuda.synchronize()
    print("gradients:", tuple(dy.shape), tuple(dlogits.shape), tuple(dx.shape))


if __name__ == "__main__":
    main()
