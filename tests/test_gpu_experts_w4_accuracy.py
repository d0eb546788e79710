"""GPU: the accuracy that the experts' products with 4-bit weights promise, and
launches whose blocks and warps take several items each.

Both kernels add (q - zero) * x of one group in float32 and then the scaled
sums of the groups, so a product is off by at most one unit (2^-23: the tensor
cores may truncate) of the sum of magnitudes for each addition on the way: one
for every channel of a group, one for every group, and 16 for the joins of
parts, the scaling and the row's scale.  The magnitudes are |q - zero| * scale
* |x|, except for E4M3 rows of experts with many rows, where codes and zero
points are multiplied one after the other: (q + zero) * scale * |x|, and twice
as many additions.  The result is rounded to bf16 once: it has to lie between
the roundings of the bound's two ends.  The gate's slope is at most 1.1, its
exponential good to 1e-6 here."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
FEW_ROWS = 8  # most rows that the kernel for few rows takes


def make(ep, E, cap, I, N, group, act, fp8, zeros, counts, seed, mean=0.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    rows = 2 * N if act == "swiglu" else N
    q = torch.randint(0, 256, (E, rows, I // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = ((torch.rand((E, rows, I // group), device="cuda", generator=gen) * 0.5 + 0.75)
              / (4.6 * math.sqrt(I))).to(torch.bfloat16)
    z = torch.randint(0, 16, (E, rows, I // group), dtype=torch.uint8, device="cuda",
                      generator=gen) if zeros else None
    x = torch.randn((E * cap, I), device="cuda", generator=gen) + mean
    xs = None
    if fp8:
        xs = torch.rand((E * cap, I // 128), device="cuda", generator=gen) + 0.1
        x = (x * 40).to(torch.float8_e4m3fn).view(torch.uint8)
        xs /= 40
    else:
        x = x.to(torch.bfloat16)
    count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    for e, c in enumerate(counts):  # rows beyond the count hold NaN
        x[e * cap + min(c, cap):(e + 1) * cap] = 0x7F if fp8 else float("nan")
    return x, xs, ep.W4Weights(q, scales, z), ep.LLLayout(None, count, None, E, 1, cap)


def product64(W, e, x, xs):
    """(p, magnitudes |q - zero|, magnitudes q + zero) of expert e's rows in 64 bits."""
    q = torch.stack((W.q[e] & 15, W.q[e] >> 4), -1).flatten(1).double()
    group = q.shape[1] // W.scales.shape[2]
    z = 8.0 if W.zeros is None else W.zeros[e].double().repeat_interleave(group, 1)
    s = W.scales[e].double().repeat_interleave(group, 1)
    if xs is None:
        x = x.double()
    else:
        x = x.view(torch.float8_e4m3fn).double() * xs.double().repeat_interleave(128, 1)
    return (x @ ((q - z) * s).t(), x.abs() @ ((q - z).abs() * s.abs()).t(),
            x.abs() @ ((q + z) * s.abs()).t())


def between(got, want, tol):
    """got is the rounding of a number within tol of want (rounding is monotonic)."""
    lo, hi = (v.float().to(torch.bfloat16).double() for v in (want - tol, want + tol))
    return bool(((got >= lo) & (got <= hi)).all())


def check(got, W, L, x, xs, counts, act):
    E, cap = L.num_experts, L.expert_capacity
    N, groups = got.shape[1], W.scales.shape[2]
    group = 2 * W.q.shape[2] // groups
    got = got.double()
    for e, c in enumerate(counts):
        n = min(c, cap)
        rows = slice(e * cap, e * cap + n)
        assert bool((got[e * cap + n:(e + 1) * cap] == -7.0).all())  # not touched
        if n == 0:
            continue
        split = xs is not None and n > FEW_ROWS
        p, mag, apart = product64(W, e, x[rows], None if xs is None else xs[rows])
        tol = ((2 if split else 1) * group + groups + 16) * 2.0 ** -23 * (apart if split else mag)
        want = p
        if act == "swiglu":
            g, u = p[:, :N], p[:, N:]
            want = g * torch.sigmoid(g) * u
            tol = 1.1 * (u.abs() + tol[:, N:]) * tol[:, :N] + (g * torch.sigmoid(g)).abs() * tol[:, N:] \
                + 1e-6 * want.abs()
        assert between(got[rows], want, tol), (e, n, float(((got[rows] - want).abs() - tol).max()))


def run(ep, E, cap, I, N, group, act, fp8, zeros, counts, seed=0, mean=0.0):
    x, xs, W, L = make(ep, E, cap, I, N, group, act, fp8, zeros, counts, seed, mean)
    out = torch.full((E * cap, N), -7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ll_experts_w4(x, W, L, x_scales=xs, act=act, out=out, err=err)
    assert int(err.item()) == 0
    check(out, W, L, x, xs, counts, act)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
def test_accuracy(ep, group, zeros, act, fp8):
    run(ep, 4, 24, 1024, 72, group, act, fp8, zeros, [5, 1, 24, 9], seed=group)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 8, 9, 200])
def test_accuracy_of_long_rows_with_a_mean(ep, rows, fp8):
    run(ep, 1, rows, 7168, 136, 128, "none", fp8, True, [rows], seed=rows, mean=1.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [3, 40])
def test_large_channel_at_its_zero_point(ep, rows, fp8):
    """A channel whose codes are the zero points adds nothing, however large:
    the other channels' sum keeps its accuracy.  (E4M3: 448 is the largest;
    with many rows its code and its zero point are separate products.)"""
    I, N = 512, 64
    x, xs, W, L = make(ep, 1, rows, I, N, 128, "none", fp8, False, [rows], 1)
    W.q[:, :, 10] = 8 | 8 << 4
    x[:, 20:22] = 0x7E if fp8 else 2.0 ** 20
    out = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    ep.ll_experts_w4(x, W, L, x_scales=xs, out=out)
    check(out, W, L, x, xs, [rows], "none")


@pytest.mark.parametrize("rows", [3, 40])
def test_large_finite_rows_stay_finite(ep, rows):
    """(q - zero) * x is at most 8 * 2^122 here, far from float32's limit."""
    I, N = 256, 64
    x, xs, W, L = make(ep, 1, rows, I, N, 128, "none", False, False, [rows], 2)
    x[:, 5] = 2.0 ** 122
    out = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    ep.ll_experts_w4(x, W, L, out=out)
    check(out, W, L, x, xs, [rows], "none")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [3, 12])
def test_swiglu_of_very_negative_gates(ep, rows, fp8):
    """exp(gate) down to 1e-40 (a subnormal, good to 2^-149 / 1e-40 < 2e-5)
    times an up projection of 2^115: results that bf16 holds."""
    gates = [60.0, 87.0, 87.5, 88.0, 88.5, 89.0, 90.0, 91.0]
    N = len(gates)
    q = torch.full((1, 2 * N, 64), 0x88, dtype=torch.uint8, device="cuda")
    q[0, :N, 0], q[0, N:, 0] = 0x87, 0x89  # channel 0: -1 for the gate, +1 for up
    scales = torch.tensor(gates + [2.0 ** 115] * N, device="cuda").to(torch.bfloat16).reshape(1, 2 * N, 1)
    L = ep.LLLayout(None, torch.tensor([rows], dtype=torch.int32, device="cuda"), None, 1, 1, rows)
    xs = None
    if fp8:
        x, xs = torch.full((rows, 128), 0x38, dtype=torch.uint8, device="cuda"), torch.ones((rows, 1), device="cuda")
    else:
        x = torch.ones((rows, 128), dtype=torch.bfloat16, device="cuda")
    got = ep.ll_experts_w4(x, ep.W4Weights(q, scales), L, x_scales=xs, act="swiglu").double()
    g = -scales[0, :N, 0].double()
    want = g * torch.sigmoid(g) * 2.0 ** 115
    assert between(got, want, 1e-4 * want.abs()), (got[0], want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [3, 12])
def test_zero_points_count_by_their_low_four_bits(ep, rows, fp8):
    x, xs, W, L = make(ep, 2, rows, 384, 40, 128, "none", fp8, True, [rows, 1], 3)
    a = torch.zeros((2 * rows, 40), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros_like(a)
    ep.ll_experts_w4(x, W, L, x_scales=xs, out=a)
    W.zeros |= 0xF0
    ep.ll_experts_w4(x, W, L, x_scales=xs, out=b)
    assert torch.equal(a, b)


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("I,group,zeros,act", [
    (128, 128, False, "none"), (128, 32, True, "swiglu"), (384, 32, True, "none"),
    (384, 128, True, "swiglu"), (640, 64, False, "swiglu"), (640, 128, False, "none"),
    (896, 64, True, "none"), (1152, 128, True, "none")])
@pytest.mark.parametrize("fp8", [False, True])
def test_many_rows_several_items_a_block(ep, fp8, I, group, zeros, act):
    """Items of experts with many rows in every block, between experts of the
    other kernel and empty ones, of one to nine steps and every height of a
    block's rows."""
    E, cap, N = 64, 200, 1000
    heights = [40, 0, 9, 3, 33, 16, 64, 65, 1, 97, 128, 8, 160, 161, 200, 192]
    counts = [heights[(5 * e + e // 16) % 16] for e in range(E)]
    most = 160 if fp8 else 192
    tiles = -(-N // (64 if act == "swiglu" else 128))
    items = sum(-(-c // most) * tiles for c in counts if c > FEW_ROWS)
    assert items > 2 * sm_count()
    run(ep, E, cap, I, N, group, act, fp8, zeros, counts, seed=I + group)


def test_many_rows_ragged_channels_several_items_a_block(ep):
    """bf16 rows whose last step is part filled, item after item."""
    for I, group in ((160, 32), (96, 32), (320, 64)):
        run(ep, 64, 24, I, 1000, group, "none", False, True, [(7 * e) % 25 for e in range(64)], seed=I)


def few_rows_plan(items, steps):
    """The launch's warps, and how many of them share a tile."""
    warps = sm_count() * 2 * 8
    best, share = -(-items // warps) * steps, 1
    for k in (2, 4, 8):
        if k <= steps and -(-items * k // warps) * -(-steps // k) < best:
            best, share = -(-items * k // warps) * -(-steps // k), k
    return warps, share


@pytest.mark.parametrize("E,I,N,act,shared", [
    (256, 256, 1000, "none", False), (256, 128, 1000, "swiglu", False), (300, 640, 1000, "none", False),
    (188, 1024, 1000, "none", True), (94, 1024, 1000, "swiglu", True), (100, 1536, 1000, "none", True)])
@pytest.mark.parametrize("fp8,group,zeros", [(False, 32, True), (False, 128, False), (True, 64, True),
                                             (True, 128, False)])
def test_few_rows_several_items_a_warp(ep, fp8, group, zeros, E, I, N, act, shared):
    counts = [1 + (3 * e + e // 8) % 8 for e in range(E)]
    items = E * -(-N // (32 if act == "swiglu" else 64))
    warps, share = few_rows_plan(items, I // 128)
    assert (share > 1) == shared and items * share > warps
    run(ep, E, 8, I, N, group, act, fp8, zeros, counts, seed=E + I)
