"""A mixture-of-experts block with its norms and residual stream, out of the
library's calls, run on one GPU.

Decoding: norm -> router logits -> the whole layer for a few tokens (4-bit
weights) -> norm after the block, gate, residual scale, addition and the next
block's norm: four launches a block, captured in a CUDA graph.
Training: the same block with bf16 weights, forward and backward.  What the
activation's gradient needs is kept in 8 bits, half of what bf16 takes; the top-k
weights are applied to the activation, so the combine takes none, and the gradient goes
back through the norms, the combine, the experts and the router to the stream and to
every weight.  For those of the experts' weights the activation is kept in bf16 and the
experts' input rows are dispatched again; in both, rows that no token fills are zeros.

    python examples/moe_block.py [--tokens 4] [--train-tokens 512] [--hidden 2048] ...
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_get_dispatch_04_gb300 as ep  # noqa: E402


class MoEBlock:
    """z = x + scale * gate * norm(experts(norm(x))); its next norm is `after`."""

    def __init__(self, hidden, inter, experts, topk, scale=0.5, device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=gen, device=device)  # noqa: E731
        bf16 = torch.bfloat16
        self.experts, self.topk, self.scale = experts, topk, scale
        self.router = (rand(experts, hidden) / hidden ** 0.5).to(bf16)
        self.w13 = (rand(experts, 2 * inter, hidden) / hidden ** 0.5).to(bf16)
        self.w2 = (rand(experts, hidden, inter) / inter ** 0.5).to(bf16)
        self.before, self.post, self.after = (1 + 0.1 * rand(hidden) for _ in range(3))
        self.gate = torch.sigmoid(rand(hidden))

    def quantise(self):
        self.up4, self.down4 = ep.quantize_w4(self.w13), ep.quantize_w4(self.w2)

    # --- decoding -------------------------------------------------------------------
    def decode(self, x, h):
        """x [T, H], the stream, is updated in place; h = norm(x).  Returns the next block's h."""
        logits = h @ self.router.t()
        y, _, _ = ep.layer_w4(h, logits, self.up4, self.down4, self.topk)
        return ep.block_norm(x, y, gate=self.gate, post_weight=self.post, pre_weight=self.after,
                             scale=self.scale, out=x).h

    # --- training -------------------------------------------------------------------
    def rows(self, x, L):
        """The experts' rows of x [T, H], zeros where no token goes."""
        out = ep.LLDispatched(x.new_zeros(L.num_rows, x.shape[1]), None,
                              torch.empty(L.num_rows, dtype=torch.int32, device=x.device), False)
        return ep.ll_dispatch(x, L, out=out).recv_x.view(self.experts, L.expert_capacity, -1)

    def forward(self, x):
        """x [T, H], the stream (bf16 or float32).  Returns z, h and what backward needs."""
        h = ep.block_norm(x, pre_weight=self.before).h
        logits = (h @ self.router.t()).float()
        idx, w = ep.route(logits, self.topk)
        L = ep.ll_get_dispatch_layout(idx, self.experts, 1)
        gate_up = torch.bmm(self.rows(h, L), self.w13.transpose(1, 2)).flatten(0, 1)
        kept = ep.alloc_checkpoint8(L.num_rows, gate_up.shape[1], x.device)
        a = ep.ll_swiglu(gate_up, L, w, checkpoint=kept,
                         out=gate_up.new_zeros(L.num_rows, gate_up.shape[1] // 2))
        a = a.view(self.experts, L.expert_capacity, -1)
        y = torch.bmm(a, self.w2.transpose(1, 2)).flatten(0, 1)
        r = ep.ll_combine_norm(y, None, L, x, gate=self.gate, post_weight=self.post,
                               pre_weight=self.after, scale=self.scale, save=True)
        return r.z, r.h, (x, h, logits, idx, w, L, kept, r.z, r.y, a)

    def backward(self, dz, dh, saved):
        """Gradients of x, of the weights and of the experts' rows (gate_up, y), from those of z
        and of the next block's h."""
        x, h, logits, idx, w, L, kept, z, y, a = saved
        g = ep.block_norm_backward(dz, dh, z, y, gate=self.gate, post_weight=self.post,
                                   pre_weight=self.after, scale=self.scale)
        # of a combine without weights: every row gets its token's gradient
        dy = self.rows(g.dy, L)
        da = torch.bmm(dy, self.w2).flatten(0, 1)
        d13, dw = ep.ll_swiglu_backward(da, kept, L, w)
        d13 = d13.view(self.experts, L.expert_capacity, -1)
        drows = torch.bmm(d13, self.w13).flatten(0, 1)
        dlogits = ep.route_backward(dw, logits, idx)
        dh = ep.ll_combine(drows, None, L) + dlogits.to(h.dtype) @ self.router
        first = ep.block_norm_backward(g.dx, dh, x, pre_weight=self.before)
        grads = dict(before=first.dpre_weight, after=g.dpre_weight, post=g.dpost_weight, gate=g.dgate,
                     router=dlogits.t() @ h.float(), w13=torch.bmm(d13.transpose(1, 2), self.rows(h, L)),
                     w2=torch.bmm(dy.transpose(1, 2), a))
        return first.dx, grads, (d13, dy)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 4), ("train-tokens", 512), ("hidden", 2048), ("inter", 1024),
                        ("experts", 32), ("topk", 4), ("blocks", 4), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    blocks = [MoEBlock(a.hidden, a.inter, a.experts, a.topk, seed=i) for i in range(a.blocks)]
    for b in blocks:
        b.quantise()
    start = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    x = start.clone()

    def step():
        x.copy_(start)
        h = ep.block_norm(x, pre_weight=blocks[0].before).h
        for b in blocks:
            h = b.decode(x, h)
        return h

    want = step().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"decoding step, {a.tokens} tokens, {a.blocks} blocks: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us (CUDA-graph replay)")

    x = torch.randn(a.train_tokens, a.hidden, device="cuda")
    z, h, saved = blocks[0].forward(x)
    dx, grads, _ = blocks[0].backward(torch.randn_like(z), torch.randn_like(h), saved)
    torch.cuda.synchronize()
    print("training:", tuple(z.shape), tuple(dx.shape), {k: tuple(v.shape) for k, v in grads.items()})


if __name__ == "__main__":
    main()
