"""GPU: the experts' products with 4-bit weights against the plain 64-bit form.

Per product p = sum w x: the float32 sum of I terms is off by at most
I * 2^-23 * sum |w x| (each addition of the tensor cores rounds or truncates
once).  The bounds below also leave room for a form that rounds each weight to
bf16 once (2^-9 of sum |w x|; over a row these are independent, so the error
of all outputs together is held to 2^-9 of their norm).  The result is rounded
to bf16 once (2^-9 |y|, 2^-8 here).  silu has a slope of at most 1.1."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu


def make(ep, E, cap, I, N, group, act, fp8, zeros, counts, seed):
    rng = np.random.default_rng(seed)
    rows = 2 * N if act == "swiglu" else N
    q = rng.integers(0, 256, (E, rows, I // 2)).astype(np.uint8)
    scales = torch.from_numpy((rng.random((E, rows, I // group)) * 0.5 + 0.75).astype(np.float32)
                              / (4.6 * np.sqrt(I))).to(torch.bfloat16)
    z = rng.integers(0, 16, (E, rows, I // group)).astype(np.uint8) if zeros else None
    x = torch.from_numpy(rng.standard_normal((E * cap, I)).astype(np.float32))
    if fp8:
        sc = torch.from_numpy((rng.random((E * cap, I // 128)) + 0.1).astype(np.float32) / 100)
        codes = (x * 100).to(torch.float8_e4m3fn)
        xd, xs = codes.view(torch.uint8).cuda(), sc.cuda()
        x64 = codes.double().numpy() * np.repeat(sc.double().numpy(), 128, 1)
    else:
        xb = x.to(torch.bfloat16)
        xd, xs, x64 = xb.cuda(), None, xb.double().numpy()
    W = ep.W4Weights(torch.from_numpy(q).cuda(), scales.cuda(),
                     None if z is None else torch.from_numpy(z).cuda())
    count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    L = ep.LLLayout(None, count, None, E, 1, cap)
    return W, L, xd, xs, x64, ref.dequantize_w4(q, scales.double().numpy(), z)


def check(got, x64, w64, counts, cap, N, act, rounded_weights):
    num = den = 0.0
    I = x64.shape[1]
    for e, c in enumerate(counts):
        n = min(c, cap)
        x = x64[e * cap:e * cap + n]
        p, mag = x @ w64[e].T, np.abs(x) @ np.abs(w64[e]).T
        tol = (I * 2.0 ** -23 + (2.0 ** -9 if rounded_weights else 0.0)) * mag
        if act == "swiglu":
            g, u = p[:, :N], p[:, N:]
            want = ref.silu(g) * u
            tol = 1.1 * (np.abs(u) + tol[:, N:]) * tol[:, :N] + (np.abs(ref.silu(g))) * tol[:, N:] \
                + 1e-6 * np.abs(want)
        else:
            want = p
        y = got[e * cap:e * cap + n]
        # a row with an E4M3 NaN code (a value beyond 448 in the test's rows) is NaN in both
        fine = np.isfinite(want)
        assert np.array_equal(np.isfinite(y), fine)
        y, want, tol = y[fine], want[fine], tol[fine]
        assert (np.abs(y - want) <= tol + 2.0 ** -8 * np.abs(want) + 1e-30).all()
        num += ((y - want) ** 2).sum()
        den += (want ** 2).sum()
        rest = got[e * cap + n:(e + 1) * cap]
        assert (rest == -7.0).all()  # rows beyond the count are not touched
    if den:
        assert np.sqrt(num / den) <= (2.0 if act == "none" else 3.0) * 2.0 ** -9


def run(ep, E, cap, I, N, group, act, fp8, zeros, counts, seed=0):
    W, L, xd, xs, x64, w64 = make(ep, E, cap, I, N, group, act, fp8, zeros, counts, seed)
    # rows beyond the count hold NaN: they must not reach the others
    for e, c in enumerate(counts):
        if fp8:
            xd[e * cap + min(c, cap):(e + 1) * cap] = 0x7F
        else:
            xd[e * cap + min(c, cap):(e + 1) * cap] = float("nan")
    out = torch.full((E * cap, N), -7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ep.ll_experts_w4(xd, W, L, x_scales=xs, act=act, out=out, err=err)
    torch.cuda.synchronize()
    assert y is out and int(err.item()) == 0
    check(y.float().cpu().numpy().astype(np.float64), x64, w64, counts, cap, N, act, True)
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
def test_forms(ep, group, act, fp8, zeros):
    run(ep, 3, 12, 384, 72, group, act, fp8, zeros, [5, 0, 12], seed=group)


@pytest.mark.parametrize("E,cap,I,N,counts", [
    (1, 1, 128, 8, [1]),                    # one row, one step, eight channels
    (2, 1, 1024, 264, [1, 0]),
    (4, 8, 2048, 40, [8, 7, 1, 0]),
    (3, 16, 256, 1000, [16, 9, 3]),         # a ragged last tile
    (2, 32, 640, 136, [31, 32]),
    (2, 40, 896, 128, [40, 33]),            # more rows than one pass takes
    (2, 70, 512, 200, [65, 70]),
    (5, 130, 256, 128, [129, 64, 0, 17, 130]),
    (2, 300, 768, 328, [257, 300]),
    (1, 700, 512, 264, [643]),
    (3, 6, 256, 16, [9, 6, 2]),             # a count above the capacity
    (2, 3, 256, 16, [0, 0]),                # nothing to do
    (300, 2, 128, 16, [i % 3 for i in range(300)]),
])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_shapes(ep, E, cap, I, N, counts, act):
    run(ep, E, cap, I, N, 128, act, False, True, counts, seed=E * I + N)


@pytest.mark.parametrize("I,group", [(32, 32), (96, 32), (160, 32), (64, 64), (192, 64), (7168, 128)])
@pytest.mark.parametrize("rows", [3, 50, 140])
def test_channels(ep, I, group, rows):
    run(ep, 2, rows, I, 72, group, "none", False, False, [rows, rows - 1], seed=I)


@pytest.mark.parametrize("I", [128, 384, 2048])
@pytest.mark.parametrize("rows", [1, 33, 100, 260])
@pytest.mark.parametrize("group", [32, 128])
def test_fp8_rows(ep, I, rows, group):
    run(ep, 3, rows, I, 136, group, "swiglu", True, True, [rows, 0, (rows + 1) // 2], seed=I + rows)


def test_one_nonfinite_row_stays_alone(ep):
    for rows in (4, 40, 150):
        W, L, xd, xs, x64, w64 = make(ep, 1, rows, 256, 64, 128, "none", False, False, [rows], 3)
        a = ep.ll_experts_w4(xd, W, L)
        xd[2] = float("inf")
        b = ep.ll_experts_w4(xd, W, L)
        keep = [r for r in range(rows) if r != 2]
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(b[2].float()).any()


def test_repeats_bit_for_bit_and_on_another_stream(ep):
    for rows in (3, 60, 200):
        W, L, xd, xs, *_ = make(ep, 4, rows, 1024, 256, 64, "swiglu", False, True,
                                [rows, rows // 2, 1, 0], 5)
        outs = [torch.zeros((4 * rows, 256), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for o in outs[:3]:
            ep.ll_experts_w4(xd, W, L, act="swiglu", out=o)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ep.ll_experts_w4(xd, W, L, act="swiglu", out=outs[3])
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert torch.equal(o, outs[0])


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("group", [32, 128])
def test_quantize_round_trip(ep, group, zero_points):
    """Quantised weights stay within half a step (of the bf16 scale), plus the
    clipping that the scale's own rounding can cause (7 or 15 steps of 2^-8)."""
    w = torch.randn((2, 24, 256), device="cuda")
    W = ep.quantize_w4(w, group, zero_points=zero_points)
    s = W.scales.double().cpu().numpy()
    back = ref.dequantize_w4(W.q.cpu().numpy(), s, None if W.zeros is None else W.zeros.cpu().numpy())
    step = np.repeat(s, group, -1)
    assert (np.abs(back - w.double().cpu().numpy()) <= (1.0 if zero_points else 0.5 + 7 / 256) * step * 1.001).all()


def test_whole_step_matches_the_pieces(ep):
    """route -> layout -> dispatch -> products -> combine on the expert-major
    layout, with the experts in 64 bits."""
    T, H, I, E, K, R = 64, 256, 128, 16, 4, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16)
    idx, w = ep.route(torch.randn((T, E), device="cuda", generator=g), K)
    w13 = ep.quantize_w4(torch.randn((E, 2 * I, H), device="cuda", generator=g) / 16)
    w2 = ep.quantize_w4(torch.randn((E, H, I), device="cuda", generator=g) / 11)
    L = ep.ll_get_dispatch_layout(idx, E, R)
    d = ep.ll_dispatch(x, L)
    h = ep.ll_experts_w4(d.recv_x, w13, L, act="swiglu")
    y = ep.ll_experts_w4(h, w2, L)
    out = ep.ll_combine(y, w, L).double().cpu().numpy()
    a = ref.dequantize_w4(w13.q.cpu().numpy(), w13.scales.double().cpu().numpy(), None)
    b = ref.dequantize_w4(w2.q.cpu().numpy(), w2.scales.double().cpu().numpy(), None)
    xs, ids, ws = x.double().cpu().numpy(), idx.cpu().numpy(), w.double().cpu().numpy()
    want = np.zeros((T, H))
    for t in range(T):
        for k in range(K):
            p = a[ids[t, k]] @ xs[t]
            want[t] += ws[t, k] * (b[ids[t, k]] @ (ref.silu(p[:I]) * p[I:]))
    # three bf16 roundings on the way (h, y, out), each 2^-9, and one of the weights' slack
    assert np.linalg.norm(out - want) <= 4 * 2.0 ** -9 * np.linalg.norm(want)


def test_refusals(ep):
    W, L, xd, xs, *_ = make(ep, 2, 4, 256, 16, 128, "none", False, False, [4, 4], 1)
    with pytest.raises(ep.EPError):
        ep.ll_experts_w4(xd[:, :128].contiguous(), W, L)
    with pytest.raises(ep.EPError):
        ep.ll_experts_w4(xd.float(), W, L)
    with pytest.raises(ep.EPError):
        ep.ll_experts_w4(xd, W, L, act="gelu")
    with pytest.raises(ep.EPError):  # E4M3 rows without scales are not bfloat16
        ep.ll_experts_w4(xd.view(torch.uint8)[:, :256].contiguous(), W, L)
    with pytest.raises(ep.EPError):  # 16 channels a group
        ep.ll_experts_w4(xd, ep.W4Weights(W.q, torch.ones((2, 16, 16), dtype=torch.bfloat16, device="cuda")), L)
    with pytest.raises(ep.EPError):  # N % 8
        ep.ll_experts_w4(xd, ep.W4Weights(W.q[:, :12].contiguous(), W.scales[:, :12].contiguous()), L)
    with pytest.raises(ep.EPError):
        ep.ll_experts_w4(xd, ep.W4Weights(W.q, W.scales, W.scales), L)
    with pytest.raises(ep.EPError):
        ep.quantize_w4(torch.randn((2, 8, 100), device="cuda"), 64)
