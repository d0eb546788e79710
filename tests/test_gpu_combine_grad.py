"""GPU: the gradient of the combine against the plain 64-bit form.

dy is one float32 sum of weights (k ascending), one multiply and one rounding
to bf16: compared bit for bit with the same steps in numpy.  dweights is a
float32 sum of H products, in chains of at most H / 128 terms per thread and
a few more to join them: (H / 128 + 16) * 2^-23 of the sum of magnitudes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import workloads
from ep_testlib import bf16_from_bits, bits_of, device_inputs, small_configs
from workloads import Config, make_case

pytestmark = pytest.mark.gpu
POISON = 0xFFFF


def bf16_bits(f32: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(f32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def reference(dout_bits, y_bits, rows, w):
    """rows [T, K]: the row of each slot (-1: none)."""
    d = oracle.bf16_to_double(dout_bits)
    T, K = rows.shape
    dw, mag = np.zeros((T, K)), np.zeros((T, K))
    weight = {}
    for t in range(T):
        for k in range(K):
            r = int(rows[t, k])
            if r < 0:
                continue
            y = oracle.bf16_to_double(y_bits[r:r + 1])[0]
            dw[t, k], mag[t, k] = (d[t] * y).sum(), np.abs(d[t] * y).sum()
            prev = weight.get(r, (t, np.float32(0)))[1]
            weight[r] = (t, np.float32(prev + np.float32(w[t, k])))
    dy = np.full_like(y_bits, POISON)
    d32 = d.astype(np.float32)
    for r, (t, s) in weight.items():
        dy[r] = bf16_bits(s * d32[t])
    return dy, dw, mag


def slots_of(idx, slot, E, R):
    dest = np.where((idx >= 0) & (idx < E), idx // (E // R), -1)
    return np.where(dest >= 0, np.take_along_axis(slot, np.maximum(dest, 0), 1), -1)


def check(ep, call, dout_bits, y_bits, rows, w, hidden):
    dy_want, dw_want, mag = reference(dout_bits, y_bits, rows, w)
    out = bf16_from_bits(np.full_like(y_bits, POISON))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dy, dw = call(out, err)
    torch.cuda.synchronize()
    assert dy is out
    assert np.array_equal(bits_of(dy), dy_want)
    lim = (hidden / 128 + 16) * 2.0 ** -23 * mag
    assert (np.abs(dw.cpu().numpy() - dw_want) <= lim).all()
    return int(err.item())


@pytest.mark.parametrize("cfg", small_configs()[1:], ids=lambda c: c.name)
def test_rank_major(ep, cfg):
    if cfg.num_tokens > 1000:
        cfg = cfg.scaled(60)
    c = make_case(cfg, with_hidden=False)
    idx, w, _ = device_inputs(c)
    E, R, H = cfg.num_experts, cfg.num_ranks, cfg.hidden
    L = ep.get_dispatch_layout(idx, E, R)
    P = ep.total_rows(L)
    rng = np.random.default_rng(cfg.seed)
    y_bits = workloads.expert_outputs(P + 3, H, cfg.seed + 1)  # three rows that no slot names
    dout_bits = workloads.expert_outputs(cfg.num_tokens, H, cfg.seed + 2)
    wn = rng.standard_normal(c.topk_idx.shape).astype(np.float32)
    rows = slots_of(c.topk_idx, L.slot.cpu().numpy(), E, R)
    d, y, wd = bf16_from_bits(dout_bits), bf16_from_bits(y_bits), torch.from_numpy(wn).cuda()
    e = check(ep, lambda out, err: ep.combine_backward(d, y, idx, wd, L, out=out, err=err),
              dout_bits, y_bits, rows, wn, H)
    assert e == 0


@pytest.mark.parametrize("T,H,E,K,R,cap,mask", [
    (1, 8, 4, 1, 1, 1, 0.0), (24, 264, 8, 3, 4, 24, 0.2), (64, 1032, 16, 4, 4, 9, 0.0),
    (16, 7168, 32, 8, 8, 16, 0.1), (6, 8200, 4, 2, 2, 6, 0.0), (3, 65528, 4, 2, 1, 3, 0.0),
    (40, 4096, 64, 32, 2, 40, 1.0)])
def test_expert_major(ep, T, H, E, K, R, cap, mask):
    cfg = Config("x", R, T // R if T % R == 0 else T, H, E, K, mask_prob=mask, seed=T + H)
    c = make_case(cfg, with_hidden=False)
    T = cfg.num_tokens
    idx, _, _ = device_inputs(c)
    L = ep.ll_get_dispatch_layout(idx, E, R, cap)
    y_bits = workloads.expert_outputs(E * cap, H, 3)
    dout_bits = workloads.expert_outputs(T, H, 4)
    wn = np.random.default_rng(1).standard_normal((T, K)).astype(np.float32)
    d, y, wd = bf16_from_bits(dout_bits), bf16_from_bits(y_bits), torch.from_numpy(wn).cuda()
    e = check(ep, lambda out, err: ep.ll_combine_backward(d, y, wd, L, out=out, err=err),
              dout_bits, y_bits, L.ll_slot.cpu().numpy(), wn, H)
    assert e == 0


def test_bad_ids_and_rows_beyond_the_buffer(ep):
    T, H, E, R = 12, 128, 8, 4
    idx_np = np.random.default_rng(0).integers(0, E, (T, 3)).astype(np.int64)
    idx_np[2, 1], idx_np[5, 0] = E, -7
    idx = torch.from_numpy(idx_np).cuda()
    L = ep.get_dispatch_layout(idx, E, R)
    P = ep.total_rows(L)
    y_bits, dout_bits = workloads.expert_outputs(P - 2, H, 1), workloads.expert_outputs(T, H, 2)
    wn = np.random.default_rng(1).random((T, 3)).astype(np.float32)
    rows = slots_of(idx_np, L.slot.cpu().numpy(), E, R)
    rows = np.where(rows >= P - 2, -1, rows)
    d, y, wd = bf16_from_bits(dout_bits), bf16_from_bits(y_bits), torch.from_numpy(wn).cuda()
    e = check(ep, lambda out, err: ep.combine_backward(d, y, idx, wd, L, out=out, err=err),
              dout_bits, y_bits, rows, wn, H)
    assert e == ep.EP_ERRBIT_BAD_EXPERT | ep.EP_ERRBIT_CAPACITY


def test_special_values_stay_in_their_rows(ep):
    """Infinities and NaN of a row that no slot names, or of one token, reach
    nothing else."""
    T, H, E, R = 8, 256, 8, 4
    c = make_case(Config("x", R, T // R, H, E, 2, seed=9), with_hidden=False)
    idx, w, _ = device_inputs(c)
    L = ep.get_dispatch_layout(idx, E, R)
    P = ep.total_rows(L)
    y = torch.randn((P + 4, H), device="cuda").to(torch.bfloat16)
    d = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    dy0, dw0 = ep.combine_backward(d, y, idx, w, L)
    y[P:] = float("nan")
    d[3] = float("inf")
    dy1, dw1 = ep.combine_backward(d, y, idx, w, L)
    rows = L.slot[3][L.slot[3] >= 0].long()
    keep = torch.ones(P + 4, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(dy0[keep], dy1[keep])
    assert (dy1[P:] == 0).all()
    others = [t for t in range(T) if t != 3]
    assert torch.equal(dw0[others], dw1[others])


def test_gradient_against_differences(ep):
    """<dout, combine(y + h v)> - <dout, combine(y - h v)> over 2 h, with the
    combine in 64 bits, against <dy, v>, and the same for the weights."""
    rng = np.random.default_rng(2)
    T, H, E, R, K = 16, 64, 8, 4, 3
    c = make_case(Config("x", R, T // R, H, E, K, seed=4, mask_prob=0.1), with_hidden=False)
    idx, w, _ = device_inputs(c)
    L = ep.get_dispatch_layout(idx, E, R)
    P = ep.total_rows(L)
    y_bits, dout_bits = workloads.expert_outputs(P, H, 5), workloads.expert_outputs(T, H, 6)
    dy, dw = ep.combine_backward(bf16_from_bits(dout_bits), bf16_from_bits(y_bits), idx, w, L)
    y, d = oracle.bf16_to_double(y_bits), oracle.bf16_to_double(dout_bits)
    wn = c.topk_weights.astype(np.float64)
    rows = slots_of(c.topk_idx, L.slot.cpu().numpy(), E, R)

    def loss(y, w):
        picked = np.where((rows >= 0)[..., None], y[np.maximum(rows, 0)], 0.0)
        return (d * (w[..., None] * picked).sum(1)).sum()

    v, u = rng.standard_normal(y.shape), rng.standard_normal(wn.shape)
    dyn = dy.float().cpu().numpy().astype(np.float64)
    num = (loss(y + v, wn) - loss(y - v, wn)) / 2  # the combine is linear: no truncation error
    assert abs((dyn * v).sum() - num) <= 2.0 ** -8 * np.abs(dyn * v).sum()
    num = (loss(y, wn + u) - loss(y, wn - u)) / 2
    dwn = dw.cpu().numpy().astype(np.float64)
    assert abs((dwn * u).sum() - num) <= 1e-4 * np.abs(dwn * u).sum()


def test_empty_and_refusals(ep):
    L = ep.get_dispatch_layout(torch.empty((0, 2), dtype=torch.int64, device="cuda"), 8, 4)
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.ones((5, 64), dtype=torch.bfloat16, device="cuda")
    dy, dw = ep.combine_backward(z, y, torch.empty((0, 2), dtype=torch.int64, device="cuda"),
                                 torch.empty((0, 2), device="cuda"), L)
    assert (dy == 0).all() and dw.shape == (0, 2)
    idx = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    L = ep.get_dispatch_layout(idx, 8, 4)
    d, w = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((4, 2), device="cuda")
    with pytest.raises(ep.EPError):
        ep.combine_backward(d[:, :32], y, idx, w, L)
    with pytest.raises(ep.EPError):
        ep.combine_backward(d.float(), y, idx, w, L)
    with pytest.raises(ep.EPError):
        ep.combine_backward(d, y, idx, w[:, :1], L)
    with pytest.raises(ep.EPError):
        ep.combine_backward(d[:, :60].contiguous(), y[:, :60].contiguous(), idx, w, L)  # H % 8
    with pytest.raises(ep.EPError):
        ep.combine_backward(d, y, idx, w, L, out=torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"))
