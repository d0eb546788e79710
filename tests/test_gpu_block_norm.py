"""The norms between two blocks (block_norm, ll_combine_norm) and their gradient
against the 64-bit definitions, at shapes, types and inputs where they can go wrong."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# A row's sum of squares is added up by threads (at most 32 values each), lanes and
# warps: 32 + 5 + 5 roundings; the factor made of it takes half of that, two units for the
# reciprocal root, and at most 6 products follow: below 64 roundings of 2^-24.
SUM = 64 * 2.0 ** -24


def rand(gen, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def inputs(T, H, gate, stream, weights, post=True, pre=True, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    return dict(x=rand(gen, T, H, dtype=stream, scale=2.0), y=rand(gen, T, H, dtype=BF16, scale=1.5),
                gate=None if shape is None else torch.sigmoid(rand(gen, *shape)).to(weights),
                post=(1 + 0.2 * rand(gen, H)).to(weights) if post else None,
                pre=(1 + 0.2 * rand(gen, H)).to(weights) if pre else None, gen=gen)


def check(got, want, bound, what):
    off = (got.to(ref.F) - want).abs()
    worst = (off - bound).max()
    assert off.numel() == 0 or float(worst) <= 0.0, \
        f"{what}: {float((off / bound.clamp(min=1e-300)).max())} times the bound"


def check_forward(r, x, y, gate, post, pre, scale, eps):
    z, h, mag = ref.block_norm(x, y, gate, post, pre, scale, eps)
    if y is not None:
        check(r.z, z, ref.half_step(x.dtype) * z.abs() + SUM * mag + 1e-40, "z")
    if pre is not None:
        f = (pre.to(ref.F) / ref.rms(z, eps)).abs()
        check(r.h, h, ref.half_step(BF16) * h.abs() + 2 * SUM * f * mag + 1e-38, "h")


@pytest.mark.parametrize("T,H", [(1, 8), (3, 256), (7, 520), (2, 2056), (5, 7168), (2, 16384),
                                 (700, 264), (33, 4104)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_forward(ep, T, H, gate, stream):
    s = inputs(T, H, gate, stream, F32 if H % 16 else BF16)
    r = ep.block_norm(s["x"], s["y"], gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"],
                      scale=0.37, eps=1e-5)
    check_forward(r, s["x"], s["y"], s["gate"], s["post"], s["pre"], 0.37, 1e-5)


@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_forward_parts(ep, post, pre, gate):
    s = inputs(9, 512, gate, BF16, F32, post, pre)
    r = ep.block_norm(s["x"], s["y"], gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"],
                      scale=-1.5)
    assert (r.h is None) == (not pre)
    check_forward(r, s["x"], s["y"], s["gate"], s["post"], s["pre"], -1.5, 1e-6)


def test_norm_alone_and_in_place(ep):
    s = inputs(6, 776, "channel", F32, F32)
    r = ep.block_norm(s["x"], pre_weight=s["pre"])
    assert r.z is None
    check_forward(r, s["x"], None, None, None, s["pre"], 1.0, 1e-6)
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"])
    want = ep.block_norm(s["x"], s["y"], **kind)
    got = ep.block_norm(s["x"], s["y"], out=s["x"], **kind)
    assert got.z.data_ptr() == s["x"].data_ptr()
    assert torch.equal(got.z, want.z) and torch.equal(got.h, want.h)


def test_rows_of_zeros_infinity_and_nan_stay_alone(ep):
    s = inputs(6, 1024, "none", BF16, F32)
    clean = ep.block_norm(s["x"], s["y"], post_weight=s["post"], pre_weight=s["pre"])
    s["y"][1] = 0.0
    s["x"][1] = 0.0
    s["y"][2, 5] = float("inf")
    s["x"][3, 1023] = float("nan")
    r = ep.block_norm(s["x"], s["y"], post_weight=s["post"], pre_weight=s["pre"])
    assert (r.z[1] == 0).all() and (r.h[1] == 0).all()
    assert r.z[2].isnan().any() and r.h[3].isnan().all()
    for t in (0, 4, 5):
        assert torch.equal(r.z[t], clean.z[t]) and torch.equal(r.h[t], clean.h[t])


@pytest.mark.parametrize("T,H,E,K", [(1, 64, 4, 1), (50, 264, 16, 4), (300, 2048, 64, 6),
                                     (17, 7168, 256, 8), (9, 1032, 64, 32)])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_combine_norm(ep, T, H, E, K, weighted, stream):
    s = inputs(T, H, "token", stream, F32, seed=3)
    idx = torch.rand((T, E), generator=s["gen"], device="cuda").topk(K).indices
    idx[torch.rand((T, K), generator=s["gen"], device="cuda") < 0.1] = -1
    if T > 5:
        idx[5] = -1  # a token without any row
    L = ep.ll_get_dispatch_layout(idx, E, 1)
    rows = rand(s["gen"], L.num_rows, H, dtype=BF16)
    w = torch.softmax(rand(s["gen"], T, K), 1) if weighted else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = ep.ll_combine_norm(rows, w, L, s["x"], gate=s["gate"], post_weight=s["post"],
                           pre_weight=s["pre"], scale=0.5, save=True, err=err)
    slot = L.ll_slot.long()
    each = (rows[slot.clamp(min=0)].to(ref.F)
            * torch.where(slot >= 0, 1.0 if w is None else w, 0.0).to(ref.F)[..., None])
    y, ym = each.sum(1), each.abs().sum(1)
    check(r.y, y, ref.half_step(BF16) * y.abs() + K * 2.0 ** -24 * ym + 1e-40, "y")
    z, h, mag = ref.block_norm(s["x"], y, s["gate"], s["post"], s["pre"], 0.5, 1e-6)
    # K roundings of the combine's sum, relative to its magnitudes; the mean square sees
    # them averaged, and the factor of the norm is below 1 / sqrt(eps) = 1000
    f = s["gate"].to(ref.F) * 0.5 * s["post"].to(ref.F).abs() / ref.rms(y, 1e-6)
    part = K * 2.0 ** -24 * f * (ym + y.abs() * (ym.square().mean(1, keepdim=True).sqrt()
                                                / ref.rms(y, 1e-6)))
    check(r.z, z, ref.half_step(stream) * z.abs() + SUM * mag + part + 1e-40, "z")
    f = (s["pre"].to(ref.F) / ref.rms(z, 1e-6)).abs()
    spread = part.square().mean(1, keepdim=True).sqrt() / ref.rms(z, 1e-6)
    check(r.h, h, ref.half_step(BF16) * h.abs() + f * (2 * SUM * mag + part + z.abs() * spread) + 1e-38, "h")
    assert int(err) == 0


def test_float32_streams_on_16_byte_boundaries(ep):
    """Buffers that are 16-byte but not 32-byte aligned give what aligned ones give."""
    T, H = 7, 1032
    s = inputs(T, H, "full", F32, F32, seed=4)
    dz, dh = rand(s["gen"], T, H), rand(s["gen"], T, H, dtype=BF16)
    kind = dict(post_weight=s["post"], pre_weight=s["pre"])

    def off(t):
        flat = torch.empty(t.numel() + 4, dtype=t.dtype, device="cuda")[4:]
        assert flat.data_ptr() % 32 == 16
        return flat.view(t.shape).copy_(t)

    want = ep.block_norm(s["x"], s["y"], gate=s["gate"], **kind)
    got = ep.block_norm(off(s["x"]), s["y"], gate=off(s["gate"]), out=off(s["x"]), **kind)
    assert torch.equal(want.z, got.z) and torch.equal(want.h, got.h)
    want = ep.block_norm_backward(dz, dh, s["x"], s["y"], gate=s["gate"], **kind)
    got = ep.block_norm_backward(off(dz), dh, off(s["x"]), s["y"], gate=off(s["gate"]), **kind)
    for name in GRADS:
        assert torch.equal(getattr(want, name), getattr(got, name)), name


def test_offsets_beyond_32_bits(ep):
    """More than 2^31 elements: the last tokens and rows are those of a small call."""
    H, T = 7168, 300_100
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    y = torch.zeros((T, H), dtype=BF16, device="cuda")
    s = inputs(5, H, "channel", BF16, F32, seed=5)
    x[-5:], y[-5:] = s["x"], s["y"]
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"])
    want, got = ep.block_norm(s["x"], s["y"], **kind), ep.block_norm(x, y, **kind)
    assert torch.equal(want.z, got.z[-5:]) and torch.equal(want.h, got.h[-5:])
    assert not got.z[:100].any() and not got.h[:100].any()
    dz, dh = torch.zeros_like(x), torch.zeros_like(x)
    dz[-5:], dh[-5:] = rand(s["gen"], 5, H, dtype=BF16), rand(s["gen"], 5, H, dtype=BF16)
    want = ep.block_norm_backward(dz[-5:].clone(), dh[-5:].clone(), s["x"], s["y"], **kind)
    got = ep.block_norm_backward(dz, dh, x, y, **kind)
    assert torch.equal(want.dx, got.dx[-5:]) and torch.equal(want.dy, got.dy[-5:])
    del dz, dh, got
    slot = torch.tensor([[T - 5, T - 1], [T - 2, -1]], dtype=torch.int32, device="cuda")
    L = ep.LLLayout(slot, None, None, T, 1, 1)
    got = ep.ll_combine_norm(y, None, L, s["x"][:2].contiguous(), save=True, **kind)
    small = ep.LLLayout(slot - torch.where(slot < 0, 0, T - 5).to(torch.int32), None, None, 5, 1, 1)
    want = ep.ll_combine_norm(s["y"], None, small, s["x"][:2].contiguous(), save=True, **kind)
    assert torch.equal(want.y, got.y) and torch.equal(want.z, got.z) and torch.equal(want.h, got.h)


def test_combine_norm_rows_beyond_the_buffer_are_left_out(ep):
    T, H = 4, 64
    x = torch.zeros((T, H), device="cuda")
    rows = torch.ones((3, H), dtype=BF16, device="cuda")
    slot = torch.tensor([[0, 3], [2, 1], [-1, -1], [2_000_000_000, 0]], dtype=torch.int32, device="cuda")
    L = ep.LLLayout(slot, None, None, 3, 1, 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = ep.ll_combine_norm(rows, None, L, x, err=err)
    assert r.z[:, 0].tolist() == [1.0, 2.0, 0.0, 1.0] and int(err) == ep.EP_ERRBIT_CAPACITY


GRADS = ("dx", "dy", "dgate", "dpost_weight", "dpre_weight")


def check_backward(r, dz, dh, z, y, gate, post, pre, scale, eps):
    want, mag = ref.block_norm_grad(dz, dh, z, y, gate, post, pre, scale, eps)
    T = z.shape[0]
    for name in GRADS:
        got = getattr(r, name)
        if name not in want:
            assert got is None, name
            continue
        # a row's factors (two norms, six sums): 4 SUM of the terms' magnitudes; sums over
        # tokens add at most T roundings more; outputs are rounded once
        bound = (4 * SUM + (T * 2.0 ** -24 if got.dim() == 1 else 0.0)) * mag[name]
        check(got, want[name], bound + ref.half_step(got.dtype) * want[name].abs() + 1e-38, name)


# rows of a few vectors; as long as one vector a thread allows (7168) and longer; float32 rows
# of which three (4688) or two (4696) are kept at once; one, three and many tokens a block
@pytest.mark.parametrize("T,H", [(1, 8), (3, 256), (5, 520), (700, 264), (37, 2056), (5, 7168),
                                 (2, 16384), (400, 1024), (640, 4688), (310, 4696), (3, 7176),
                                 (1300, 8192), (20000, 32)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_backward(ep, T, H, gate, stream):
    weights = BF16 if H % 16 == 0 else F32
    s = inputs(T, H, gate, stream, weights, seed=1)
    dz, dh = rand(s["gen"], T, H, dtype=stream), rand(s["gen"], T, H, dtype=BF16)
    r = ep.block_norm_backward(dz, dh, s["x"], s["y"], gate=s["gate"], post_weight=s["post"],
                               pre_weight=s["pre"], scale=0.37, eps=1e-5)
    check_backward(r, dz, dh, s["x"], s["y"], s["gate"], s["post"], s["pre"], 0.37, 1e-5)
    again = ep.block_norm_backward(dz, dh, s["x"], s["y"], gate=s["gate"], post_weight=s["post"],
                                   pre_weight=s["pre"], scale=0.37, eps=1e-5)
    for name in GRADS:
        a, b = getattr(r, name), getattr(again, name)
        assert a is b is None or torch.equal(a, b), name


@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("use_dz", [True, False])
def test_backward_parts(ep, post, pre, gate, use_dz):
    if not pre and not use_dz:
        pytest.skip("no gradient comes in")
    s = inputs(11, 640, gate, BF16, F32, post, pre, seed=2)
    dz = rand(s["gen"], 11, 640, dtype=BF16) if use_dz else None
    dh = rand(s["gen"], 11, 640, dtype=BF16) if pre else None
    y = s["y"] if post or gate != "none" else None
    r = ep.block_norm_backward(dz, dh, s["x"], y, gate=s["gate"], post_weight=s["post"],
                               pre_weight=s["pre"], scale=2.0)
    check_backward(r, dz, dh, s["x"], y, s["gate"], s["post"], s["pre"], 2.0, 1e-6)


def test_backward_rows_of_zeros_and_no_tokens(ep):
    s = inputs(4, 256, "channel", BF16, F32)
    s["x"][1] = 0.0
    s["y"][1] = 0.0
    dz, dh = rand(s["gen"], 4, 256, dtype=BF16), rand(s["gen"], 4, 256, dtype=BF16)
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"])
    r = ep.block_norm_backward(dz, dh, s["x"], s["y"], **kind)
    check_backward(r, dz, dh, s["x"], s["y"], s["gate"], s["post"], s["pre"], 1.0, 1e-6)
    r = ep.block_norm_backward(dz[:0], dh[:0], s["x"][:0], s["y"][:0], **kind)
    torch.cuda.synchronize()
    assert r.dx.shape == (0, 256) and not r.dgate.any() and not r.dpost_weight.any()
    assert not r.dpre_weight.any()
    r = ep.block_norm(s["x"][:0], s["y"][:0], post_weight=s["post"], pre_weight=s["pre"])
    assert r.z.shape == r.h.shape == (0, 256)


@pytest.mark.parametrize("H", [512, 7176])
@pytest.mark.parametrize("zs,ys,use_dz", [(1e15, 1e15, True), (1e15, 1.0, False), (1e12, 1e12, False),
                                          (1e-14, 1.0, True), (1.0, 1e-14, True)])
def test_backward_of_large_and_small_rows(ep, H, zs, ys, use_dz):
    """Rows whose 1 / rms cubed is not a 32-bit number have the same relative bounds."""
    s = inputs(7, H, "token", F32, F32, seed=6)
    z, y = s["x"] * zs, (s["y"].float() * ys).to(BF16)
    dz = rand(s["gen"], 7, H) if use_dz else None
    dh = rand(s["gen"], 7, H, dtype=BF16)
    r = ep.block_norm_backward(dz, dh, z, y, gate=s["gate"], post_weight=s["post"],
                               pre_weight=s["pre"], eps=1e-30)
    check_backward(r, dz, dh, z, y, s["gate"], s["post"], s["pre"], 1.0, 1e-30)


def test_formula_agrees_with_differences():
    """The 64-bit gradient against central differences (error h^2 / 6 of a third
    derivative, and 1e-16 / h of the values)."""
    gen = torch.Generator().manual_seed(0)
    T, H, step = 3, 8, 1e-5
    r = lambda *shape: torch.randn(shape, generator=gen, dtype=torch.float64)  # noqa: E731
    x, y, gate, post, pre, cz, ch = r(T, H), r(T, H), r(H), r(H), r(H), r(T, H), r(T, H)

    def loss(x, y, gate, post, pre):
        z, h, _ = ref.block_norm(x, y, gate, post, pre, 0.7, 1e-3)
        return float((cz * z).sum() + (ch * h).sum())

    leaves = [x, y, gate, post, pre]
    z, _, _ = ref.block_norm(*leaves, 0.7, 1e-3)
    want, _ = ref.block_norm_grad(cz, ch, z, y, gate, post, pre, 0.7, 1e-3)
    for i, name in enumerate(GRADS):
        for at in range(0, leaves[i].numel(), 3):
            d = torch.zeros_like(leaves[i]).flatten()
            d[at] = step
            d = d.reshape(leaves[i].shape)
            plus, minus = ([v + (k * d if j == i else 0.0) for j, v in enumerate(leaves)] for k in (1, -1))
            num = (loss(*plus) - loss(*minus)) / (2 * step)
            assert abs(num - float(want[name].flatten()[at])) < 1e-7, (name, at)


def test_arguments(ep):
    s = inputs(4, 64, "channel", BF16, F32)
    x, y, kind = s["x"], s["y"], dict(post_weight=s["post"], pre_weight=s["pre"])
    dz, dh = torch.ones_like(x), torch.ones_like(y)
    bad = [lambda: ep.block_norm(x), lambda: ep.block_norm(x, gate=s["gate"], pre_weight=s["pre"]),
           lambda: ep.block_norm(x, y[:3], **kind), lambda: ep.block_norm(x, y.float(), **kind),
           lambda: ep.block_norm(x.half(), y, **kind), lambda: ep.block_norm(x, y, eps=0.0, **kind),
           lambda: ep.block_norm(x, y, eps=float("nan"), **kind),
           lambda: ep.block_norm(x, y, gate=s["gate"].to(BF16), **kind),
           lambda: ep.block_norm(x, y, gate=s["gate"][:32], **kind),
           lambda: ep.block_norm(x, y, out=y, **kind),
           lambda: ep.block_norm(x, y, out=x.float(), **kind),
           lambda: ep.block_norm(x[:, :60].contiguous(), y[:, :60].contiguous()),
           lambda: ep.block_norm(x.t(), y.t()), lambda: ep.block_norm(x.cpu(), y.cpu()),
           lambda: ep.block_norm(x, y, post_weight=s["post"].cpu()),
           lambda: ep.block_norm_backward(None, None, x, y, **kind),
           lambda: ep.block_norm_backward(dz, None, x, y, **kind),
           lambda: ep.block_norm_backward(dz, dh, x, None, **kind),
           lambda: ep.block_norm_backward(dz.float(), dh, x, y, **kind),
           lambda: ep.block_norm_backward(dz, dh[:3], x, y, **kind)]
    for i, call in enumerate(bad):
        with pytest.raises(ep.EPError):
            call()
            print(i)
    flat = torch.zeros(4 * 64 * 2, dtype=BF16, device="cuda")
    with pytest.raises(ep.EPError):  # z would overlap y by half a row
        ep.block_norm(x, flat[:256].view(4, 64), out=flat[32:288].view(4, 64))
    with pytest.raises(ep.EPError):  # not on a 16-byte boundary
        ep.block_norm(x, flat[4:260].view(4, 64))


def test_captured_and_on_two_streams(ep):
    s = inputs(64, 1024, "channel", F32, F32)
    dz, dh = rand(s["gen"], 64, 1024), rand(s["gen"], 64, 1024, dtype=BF16)
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"])

    def step():
        r = ep.block_norm(s["x"], s["y"], **kind)
        g = ep.block_norm_backward(dz, dh, r.z, s["y"], **kind)
        return [r.z, r.h, g.dx, g.dy, g.dgate, g.dpost_weight, g.dpre_weight]

    want = step()
    torch.cuda.synchronize()
    streams, graphs, got = [torch.cuda.Stream() for _ in range(2)], [], []
    for st in streams:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            got.append(step())
        graphs.append(graph)
    for _ in range(10):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for out in got:
        for a, b in zip(want, out):
            assert torch.equal(a, b)
