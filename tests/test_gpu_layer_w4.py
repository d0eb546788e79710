"""The layer for a few tokens against the 64-bit definition and the single
operators."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def weights(ep, gen, E, rows, inner, group, zeros):
    q = torch.randint(0, 256, (E, rows, inner // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (0.75 + 0.5 * torch.rand((E, rows, inner // group), generator=gen, device="cuda"))
    s = (s / (4.6 * inner ** 0.5)).to(BF16)
    z = None
    if zeros:  # the upper four bits do not count
        z = torch.randint(0, 256, s.shape, dtype=torch.uint8, device="cuda", generator=gen)
    return ep.W4Weights(q, s, z)


def case(ep, T, H, N, E, groups=(128, 128), zeros=(False, False), seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF16)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    return (x, logits, weights(ep, gen, E, 2 * N, H, groups[0], zeros[0]),
            weights(ep, gen, E, H, N, groups[1], zeros[1]))


def check(ep, got, x, logits, gate_up, down, K, **kind):
    out, idx, w = got
    want_idx, want_w = ep.route(logits, K, **kind)
    assert torch.equal(idx, want_idx)
    # the same float32 formula, its sums (of at most 512 exponentials: 16 in a lane, then 5
    # joins, so 21 roundings on either side, and a few) in another order
    assert torch.allclose(w, want_w, rtol=96 * 2.0 ** -24, atol=0.0)
    want, off = ref.layer(x, idx, w, gate_up, down)
    bound = off + ref.half_step(BF16) * (want.abs() + off) + 1e-38
    diff = (out.to(ref.F) - want).abs()
    assert bool((diff <= bound).all()), f"{float((diff / bound).max())} times the bound"


@pytest.mark.parametrize("T", [1, 2, 4, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("E,K", [(2, 1), (16, 4), (64, 6)])
def test_tokens(ep, T, E, K):
    x, logits, a, b = case(ep, T, 512, 256, E, seed=T)
    check(ep, ep.layer_w4(x, logits, a, b, K), x, logits, a, b, K)


@pytest.mark.parametrize("H,N,groups", [(128, 128, (128, 128)), (32, 32, (32, 32)),
                                        (160, 96, (32, 32)), (192, 320, (64, 64)),
                                        (576, 64, (64, 32)), (384, 640, (128, 64)),
                                        (1152, 1408, (32, 128)), (4096, 1024, (64, 128)),
                                        (7168, 2048, (128, 128))])
@pytest.mark.parametrize("zeros", [(False, False), (True, True), (True, False)])
@pytest.mark.parametrize("T", [1, 7, 16])
def test_shapes(ep, H, N, groups, zeros, T):
    x, logits, a, b = case(ep, T, H, N, 12, groups, zeros, seed=H + T)
    check(ep, ep.layer_w4(x, logits, a, b, 3), x, logits, a, b, 3)


@pytest.mark.parametrize("kind", [dict(score="sigmoid", num_groups=4, topk_groups=2, scale=2.5),
                                  dict(score="sigmoid", renormalize=False),
                                  dict(score="softmax", renormalize=False, scale=0.5),
                                  dict(score="softmax", num_groups=8, topk_groups=3)])
@pytest.mark.parametrize("E", [64, 96, 256, 320, 512])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_router_options(ep, kind, E, dtype):
    x, logits, a, b = case(ep, 6, 128, 64, E, (128, 64), seed=E)
    logits = logits.to(dtype)
    if kind["score"] == "sigmoid":
        gen = torch.Generator("cuda").manual_seed(1)
        kind = dict(kind, bias=torch.randn(E, generator=gen, device="cuda") * 0.1)
    check(ep, ep.layer_w4(x, logits, a, b, 6, **kind), x, logits, a, b, 6, **kind)


@pytest.mark.parametrize("K", [1, 32])
def test_most_experts_a_token(ep, K):
    x, logits, a, b = case(ep, 16, 128, 32, 40, (128, 32), seed=K)
    check(ep, ep.layer_w4(x, logits, a, b, K), x, logits, a, b, K)


def test_strided_logits_and_experts_switched_off(ep):
    x, logits, a, b = case(ep, 9, 256, 128, 16, seed=5)
    wide = torch.full((9, 37), 50.0, device="cuda")
    wide[:, :16] = logits
    wide[2, :14] = float("-inf")   # two experts are left of four
    wide[4, :16] = float("nan")    # none is left
    view = wide[:, :16]
    got = ep.layer_w4(x, view, a, b, 4)
    check(ep, got, x, view, a, b, 4)
    out, idx, w = got
    assert (idx[4] == -1).all() and (w[4] == 0).all() and (out[4] == 0).all()
    assert (idx[2] >= 0).sum() == 2
    wide[:, :16] = float("-inf")   # no token has any
    out, idx, w = ep.layer_w4(x, view, a, b, 4)
    assert (out == 0).all() and (idx == -1).all() and (w == 0).all()


def test_infinity_and_nan_stay_in_their_token(ep):
    for T in (5, 12):
        x, logits, a, b = case(ep, T, 256, 128, 4, seed=6)
        clean = ep.layer_w4(x, logits, a, b, 2)[0]
        x[1, 7] = float("inf")
        x[3, 200] = float("nan")
        out = ep.layer_w4(x, logits, a, b, 2)[0]
        assert not out[1].isfinite().any() and out[3].isnan().all()
        keep = [t for t in range(T) if t not in (1, 3)]
        assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("power", [-60, -40, 40, 100])
def test_magnitudes(ep, power):
    """Rows of any magnitude: products and sums scale by powers of two exactly as long
    as nothing leaves the range of the types (the gate's exponential does not scale, so
    only u does: its rows' scales)."""
    x, logits, a, b = case(ep, 3, 256, 128, 4, seed=8)
    big = ep.W4Weights(a.q, a.scales.clone(), None)
    big.scales[:, 128:] *= 2.0 ** power
    small = ep.W4Weights(b.q, b.scales * 2.0 ** -(power // 2), None)
    out = ep.layer_w4(x, logits, a, b, 2)[0]
    got = ep.layer_w4(x, logits, big, small, 2)[0]
    assert torch.equal(got, out * 2.0 ** (power - power // 2))


def test_in_place_repeated_and_agrees_with_the_single_calls(ep):
    x, logits, a, b = case(ep, 11, 1024, 512, 32, zeros=(True, False), seed=7)
    out, idx, w = ep.layer_w4(x, logits, a, b, 4)
    for _ in range(3):
        again = ep.layer_w4(x, logits, a, b, 4)
        assert torch.equal(again[0], out) and torch.equal(again[2], w)
    L = ep.ll_get_dispatch_layout(idx, 32, 1)
    rows = ep.ll_dispatch(x, L).recv_x
    chain = ep.ll_combine(ep.ll_experts_w4(ep.ll_experts_w4(rows, a, L, act="swiglu"), b, L), w, L)
    # the chain rounds h and the experts' outputs to bf16 (half a step each), both round the result
    norm = torch.linalg.norm
    assert float(norm(out.double() - chain.double()) / norm(out.double())) < 4 * 2.0 ** -8
    got = ep.layer_w4(x, logits, a, b, 4, out=x)
    assert got[0].data_ptr() == x.data_ptr() and torch.equal(x, out)


def test_captured_on_two_streams(ep):
    cases = [case(ep, T, 512, 256, 16, seed=T) for T in (3, 16)]
    want = [ep.layer_w4(*c, 4) for c in cases]
    torch.cuda.synchronize()
    streams, graphs, got = [torch.cuda.Stream() for _ in cases], [], []
    for st, c in zip(streams, cases):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            ep.layer_w4(*c, 4)
            got.append(ep.layer_w4(*c, 4))
        graphs.append(graph)
    for _ in range(20):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        ep.layer_w4(*cases[0], 4)  # beside an eager call on another stream
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_many_replays_see_new_inputs(ep):
    x, logits, a, b = case(ep, 2, 256, 128, 8, seed=9)
    ep.layer_w4(x, logits, a, b, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, idx, w = ep.layer_w4(x, logits, a, b, 2)
    for seed in range(20, 24):
        new = case(ep, 2, 256, 128, 8, seed=seed)
        x.copy_(new[0])
        logits.copy_(new[1])
        graph.replay()
        check(ep, (out, idx, w), x, logits, a, b, 2)


def test_experts_beyond_32_bits(ep):
    """Weights of more than 2^31 bytes: the last experts' are read at their place."""
    E, H, N = 512, 4096, 1152  # 4.8 and 2.4 GB
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((3, H), generator=gen, device="cuda").to(BF16)
    logits = torch.zeros((3, E), device="cuda")
    logits[:, -4:] = torch.randn((3, 4), generator=gen, device="cuda") + 10
    a, b = weights(ep, gen, E, 2 * N, H, 128, True), weights(ep, gen, E, H, N, 128, True)
    check(ep, ep.layer_w4(x, logits, a, b, 3), x, logits, a, b, 3)


def test_no_tokens_and_arguments(ep):
    x, logits, a, b = case(ep, 4, 256, 128, 8)
    out, idx, w = ep.layer_w4(x[:0], logits[:0], a, b, 2)
    assert out.shape == (0, 256) and idx.shape == w.shape == (0, 2)
    many = torch.zeros((17, 256), dtype=BF16, device="cuda")
    bad = [lambda: ep.layer_w4(many, torch.zeros((17, 8), device="cuda"), a, b, 2),
           lambda: ep.layer_w4(x[:3], logits, a, b, 2), lambda: ep.layer_w4(x.float(), logits, a, b, 2),
           lambda: ep.layer_w4(x, logits, b, a, 2), lambda: ep.layer_w4(x, logits, a, a, 2),
           lambda: ep.layer_w4(x, logits[:, :7], a, b, 2), lambda: ep.layer_w4(x, logits, a, b, 9),
           lambda: ep.layer_w4(x, logits, a, b, 0), lambda: ep.layer_w4(x, logits, a, b, 2, score="tanh"),
           lambda: ep.layer_w4(x, logits, a, b, 2, num_groups=3),
           lambda: ep.layer_w4(x, logits, a, b, 2, bias=torch.zeros(7, device="cuda")),
           lambda: ep.layer_w4(x.cpu(), logits, a, b, 2), lambda: ep.layer_w4(x, logits.cpu(), a, b, 2),
           lambda: ep.layer_w4(x, logits, ep.W4Weights(a.q.cpu(), a.scales, None), b, 2),
           lambda: ep.layer_w4(x, logits, ep.W4Weights(a.q, a.scales[:, :, :1].repeat(1, 1, 16).contiguous(), None), b, 2),
           lambda: ep.layer_w4(x, logits, a, b, 2, out=x[:3]),
           lambda: ep.layer_w4(x, logits, a, b, 2, out=logits.view(BF16)[:, :8])]
    for i, call in enumerate(bad):
        with pytest.raises(ep.EPError):
            call()
            print(i)
