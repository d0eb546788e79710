"""The norms between two blocks and their gradient with many tokens a block: kernels whose blocks
stay go round their loops, rings and lists several times."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref
from test_gpu_block_norm import BF16, F32, GRADS, SUM, check, check_backward, check_forward, inputs, rand

pytestmark = pytest.mark.gpu


# out of the experts' rows; a GPU holds at most 32 blocks an SM for rows of one vector a thread (64), 3
# for 7168, 1 for 16384.  Slots are masked at random, so that lists differ in length from token to token, and
# runs of tokens have no row at all.
@pytest.mark.parametrize("T,H,E,K", [(4099, 7168, 16, 8), (1300, 16384, 8, 4), (20001, 64, 40, 32),
                                     (30011, 1032, 4, 1), (2500, 4104, 16, 6)])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_combine_norm(ep, T, H, E, K, stream):
    s = inputs(T, H, "channel", stream, F32, seed=21)
    idx = torch.rand((T, E), generator=s["gen"], device="cuda").topk(K).indices
    idx[torch.rand((T, K), generator=s["gen"], device="cuda") < 0.3] = -1
    idx[torch.rand(T, generator=s["gen"], device="cuda") < 0.1] = -1
    idx[T // 2:T // 2 + 700] = -1  # several in a row of most blocks
    L = ep.ll_get_dispatch_layout(idx, E, 1, int(torch.bincount(idx[idx >= 0], minlength=E).max()))
    rows = rand(s["gen"], L.num_rows, H, dtype=BF16)
    w = torch.softmax(rand(s["gen"], T, K), 1)
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"], scale=0.5)
    r = ep.ll_combine_norm(rows, w, L, s["x"], save=True, **kind)
    again = ep.ll_combine_norm(rows, w, L, s["x"], save=True, **kind)
    for a, b in ((r.z, again.z), (r.h, again.h), (r.y, again.y)):
        assert torch.equal(a, b)
    slot = L.ll_slot.long()
    for t0 in range(0, T, 512):
        part = slice(t0, min(t0 + 512, T))
        each = (rows[slot[part].clamp(min=0)].to(ref.F)
                * torch.where(slot[part] >= 0, w[part], 0.0).to(ref.F)[..., None])
        y, ym = each.sum(1), each.abs().sum(1)
        check(r.y[part], y, ref.half_step(BF16) * y.abs() + K * 2.0 ** -24 * ym + 1e-40, "y")
        z, h, mag = ref.block_norm(s["x"][part], y, s["gate"], s["post"], s["pre"], 0.5, 1e-6)
        # K roundings of the combine's sum, relative to its magnitudes, and those of the mean square
        f = s["gate"].to(ref.F) * 0.5 * s["post"].to(ref.F).abs() / ref.rms(y, 1e-6)
        off = K * 2.0 ** -24 * f * (ym + y.abs() * (ym.square().mean(1, keepdim=True).sqrt()
                                                   / ref.rms(y, 1e-6)))
        check(r.z[part], z, ref.half_step(stream) * z.abs() + SUM * mag + off + 1e-40, "z")
        f = (s["pre"].to(ref.F) / ref.rms(z, 1e-6)).abs()
        spread = off.square().mean(1, keepdim=True).sqrt() / ref.rms(z, 1e-6)
        check(r.h[part], h, ref.half_step(BF16) * h.abs() + f * (2 * SUM * mag + off + z.abs() * spread)
              + 1e-38, "h")


@pytest.mark.parametrize("T,H", [(20003, 1024), (5003, 7168)])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_forward(ep, T, H, stream):
    s = inputs(T, H, "full", stream, BF16, seed=22)
    r = ep.block_norm(s["x"], s["y"], gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"], scale=0.37)
    check_forward(r, s["x"], s["y"], s["gate"], s["post"], s["pre"], 0.37, 1e-6)


# one vector a thread, three rows in shared memory (640, 6144), of float32 rows two from 6152 on; and
# the kernel of longer rows
@pytest.mark.parametrize("T,H", [(3001, 640), (1003, 6144), (1003, 6152), (701, 7168), (701, 7176)])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_backward(ep, T, H, post, pre, gate, stream):
    s = inputs(T, H, gate, stream, F32, post, pre, seed=23)
    dz = rand(s["gen"], T, H, dtype=stream)
    dh = rand(s["gen"], T, H, dtype=BF16) if pre else None
    y = s["y"] if post or gate != "none" else None
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"], scale=2.0)
    r = ep.block_norm_backward(dz, dh, s["x"], y, **kind)
    check_backward(r, dz, dh, s["x"], y, s["gate"], s["post"], s["pre"], 2.0, 1e-6)
    again = ep.block_norm_backward(dz, dh, s["x"], y, **kind)
    for name in GRADS:
        a, b = getattr(r, name), getattr(again, name)
        assert a is b is None or torch.equal(a, b), name


@pytest.mark.parametrize("T,H", [(2003, 640), (703, 7168), (703, 7176)])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_backward_without_dz(ep, T, H, stream):
    s = inputs(T, H, "token", stream, F32, seed=24)
    dh = rand(s["gen"], T, H, dtype=BF16)
    r = ep.block_norm_backward(None, dh, s["x"], s["y"], gate=s["gate"], post_weight=s["post"],
                               pre_weight=s["pre"])
    check_backward(r, None, dh, s["x"], s["y"], s["gate"], s["post"], s["pre"], 1.0, 1e-6)
