"""The gated activation with its 8-bit checkpoint and its gradient against the
64-bit definitions."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HALF = ref.half_step(BF16)


def case(ep, T, E, K, N, seed=0, masked=0.1, capacity=None):
    gen = torch.Generator("cuda").manual_seed(seed)
    idx = torch.rand((T, E), generator=gen, device="cuda").topk(K).indices
    idx[torch.rand((T, K), generator=gen, device="cuda") < masked] = -1
    L = ep.ll_get_dispatch_layout(idx, E, 1, capacity)
    gu = (torch.randn((L.num_rows, 2 * N), generator=gen, device="cuda") * 2).to(BF16)
    dh = torch.randn((L.num_rows, N), generator=gen, device="cuda").to(BF16)
    w = torch.softmax(torch.randn((T, K), generator=gen, device="cuda"), 1)
    return L, gu, dh, w


def named(L, w=None):
    """The rows that slots name and the weight of each."""
    slot = L.ll_slot.long()
    live = slot >= 0
    return slot[live], (torch.ones_like(slot, dtype=torch.float32) if w is None else w)[live], live


def sigmoid_off(gate_up):
    """What a sigmoid, and the few products made of it, may be off, relative: the exponential by
    2 + 1.173 |g| units in the last place (2^-23), the reciprocal and six products by
    eight of 2^-24."""
    g = gate_up.to(ref.F).chunk(2, dim=1)[0].abs()
    return (2 * (2 + 1.173 * g) + 8) * 2.0 ** -24


def check(got, want, bound, what):
    off = (got.to(ref.F) - want).abs()
    assert off.numel() == 0 or bool((off <= bound).all()), \
        f"{what}: {float((off / bound.clamp(min=1e-300)).max())} times the bound"


# few and many slots, and rows of few and many vectors, on either side of the rule that gives a
# row a warp or a block
SHAPES = [(1, 4, 1, 128), (30, 8, 2, 256), (64, 16, 4, 640), (9, 256, 8, 2048), (200, 64, 6, 384),
          (3, 4, 3, 4096), (1300, 16, 4, 640), (900, 8, 6, 1152)]


@pytest.mark.parametrize("T,E,K,N", SHAPES + [(5, 4, 2, 8), (40, 8, 2, 136), (7, 16, 4, 5000)])
@pytest.mark.parametrize("weighted", [True, False])
def test_forward(ep, T, E, K, N, weighted):
    L, gu, _, w = case(ep, T, E, K, N)
    w = w if weighted else None
    out = torch.full((L.num_rows, N), 7.0, dtype=BF16, device="cuda")
    kept = None
    if N % 128 == 0:
        kept = ep.Checkpoint8(torch.full((L.num_rows, 2 * N), 0x55, dtype=torch.uint8, device="cuda"),
                              torch.full((L.num_rows, 2 * N // 128), 7.0, device="cuda"))
    h = ep.ll_swiglu(gu, L, w, checkpoint=kept, out=out)
    rows, wr, _ = named(L, w)
    want = ref.swiglu(gu[rows], wr)
    check(h[rows], want, (HALF + sigmoid_off(gu[rows])) * want.abs() + 1e-38, "h")
    other = torch.ones(L.num_rows, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert (h[other] == 7.0).all()
    if kept is not None:
        codes, scales = ref.to_8_bits(gu[rows])
        assert torch.equal(kept.codes[rows], codes) and torch.equal(kept.scales[rows], scales)
        assert (kept.codes[other] == 0x55).all() and (kept.scales[other] == 7.0).all()
        assert torch.equal(h, ep.ll_swiglu(gu, L, w, out=out.clone()))


def check_backward(ep, d, dw, dh, gu, L, w):
    rows, wr, live = named(L, w)
    want, ww, mag, wm = ref.swiglu_grad(dh[rows], gu[rows], wr)
    off = sigmoid_off(gu[rows])
    check(d[rows], want, HALF * want.abs() + torch.cat((off, off), 1) * mag + 1e-38, "dgate_up")
    if w is None:
        assert dw is None
        return
    N = dh.shape[1]
    assert (dw[~live] == 0).all()
    # each lane adds N / 32 values in a row at most, then lanes and warps
    check(dw[live], ww, (24 + N / 32 + 16) * 2.0 ** -24 * wm + 1e-38, "dweights")


@pytest.mark.parametrize("T,E,K,N", SHAPES)
@pytest.mark.parametrize("weighted", [True, False])
def test_backward_from_the_checkpoint(ep, T, E, K, N, weighted):
    L, gu, dh, w = case(ep, T, E, K, N, seed=1)
    w = w if weighted else None
    kept = ep.alloc_checkpoint8(L.num_rows, 2 * N, gu.device)
    ep.ll_swiglu(gu, L, w, checkpoint=kept)
    d, dw = ep.ll_swiglu_backward(dh, kept, L, w)
    rows, _, _ = named(L)
    other = torch.ones(L.num_rows, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert not d[other].any()
    stored = torch.zeros((L.num_rows, 2 * N), device="cuda")
    stored[rows] = ref.from_8_bits(kept.codes[rows], kept.scales[rows])
    check_backward(ep, d, dw, dh, stored, L, w)
    # what 8 bits cost: a rounding of each of g and u
    if rows.numel():
        full = ref.swiglu_grad(dh[rows], gu[rows], named(L, w)[1])[0]
        assert float(torch.linalg.norm(d[rows].to(ref.F) - full) / torch.linalg.norm(full)) < 2.0 ** -3


@pytest.mark.parametrize("T,E,K,N", SHAPES + [(5, 4, 2, 8), (40, 8, 2, 136), (7, 16, 4, 5000)])
@pytest.mark.parametrize("weighted", [True, False])
def test_backward_from_the_input(ep, T, E, K, N, weighted):
    L, gu, dh, w = case(ep, T, E, K, N, seed=2)
    w = w if weighted else None
    out = torch.full((L.num_rows, 2 * N), 3.0, dtype=BF16, device="cuda")
    d, dw = ep.ll_swiglu_backward(dh, gu, L, w, out=out)
    check_backward(ep, d, dw, dh, gu, L, w)
    rows, _, _ = named(L)
    other = torch.ones(L.num_rows, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert (d[other] == 3.0).all()


def test_wide_gates(ep):
    """Gates from the smallest to where the exponential under- and overflows."""
    L, gu, dh, w = case(ep, 8, 4, 2, 128, masked=0.0)
    g = torch.linspace(-120, 120, L.num_rows * 128, device="cuda").reshape(-1, 128)
    gu[:, :128] = g.to(BF16)
    gu[0, :4] = torch.tensor([1e-30, -1e-30, 3e38, -3e38], device="cuda").to(BF16)
    rows, wr, _ = named(L, w)
    h = ep.ll_swiglu(gu, L, w)
    want = ref.swiglu(gu[rows], wr)
    fine = want.abs() < 3e38
    # exponentials below the smallest normal number count as 0: below 1e-35 absolutely
    off = (h[rows].to(ref.F) - want).abs()
    assert bool((off <= (HALF + sigmoid_off(gu[rows])) * want.abs() + 1e-35)[fine].all())
    d, dw = ep.ll_swiglu_backward(dh, gu, L, w)
    assert not d[rows].isnan().any() and not dw.isnan().any()


def test_infinity_and_nan_stay_in_their_block(ep):
    L, gu, dh, w = case(ep, 6, 4, 2, 256, masked=0.0)
    rows, _, _ = named(L)
    gu[rows[3], 130] = float("inf")   # the second block of g
    gu[rows[7], 256 + 5] = float("nan")  # the first block of u
    kept = ep.alloc_checkpoint8(L.num_rows, 512, gu.device)
    ep.ll_swiglu(gu, L, w, checkpoint=kept)
    read = ref.from_8_bits(kept.codes, kept.scales).isnan()
    for row, block in ((rows[3], 1), (rows[7], 2)):
        assert read[row, block * 128:(block + 1) * 128].all()
        read[row, block * 128:(block + 1) * 128] = False
    assert not read[rows].any()
    d, dw = ep.ll_swiglu_backward(dh, kept, L, w)
    assert int(d[rows].isnan().any(1).sum()) == 2 and int(dw.isnan().sum()) == 2


def test_rows_beyond_the_buffer_are_skipped(ep):
    slot = torch.tensor([[0, 4], [3, 2_000_000_000]], dtype=torch.int32, device="cuda")
    L = ep.LLLayout(slot, None, None, 4, 1, 1)
    gu = torch.ones((4, 256), dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros((4, 128), dtype=BF16, device="cuda")
    ep.ll_swiglu(gu, L, err=err, out=out)
    assert int(err) == ep.EP_ERRBIT_CAPACITY
    assert out[:, 0].ne(0).tolist() == [True, False, False, True]
    err.zero_()
    w = torch.ones((2, 2), device="cuda")
    d, dw = ep.ll_swiglu_backward(out, gu, L, w, err=err)
    assert int(err) == ep.EP_ERRBIT_CAPACITY
    assert dw.ne(0).tolist() == [[True, False], [True, False]]


def test_offsets_beyond_32_bits(ep):
    """Rows that begin beyond 2^31 elements give what a small call gives."""
    rows, N = 600_000, 2048
    gen = torch.Generator("cuda").manual_seed(4)
    small = torch.randn((4, 2 * N), generator=gen, device="cuda").to(BF16)
    dh = torch.randn((4, N), generator=gen, device="cuda").to(BF16)
    w = torch.rand((2, 2), generator=gen, device="cuda")
    slot = torch.tensor([[0, 3], [2, 1]], dtype=torch.int32, device="cuda")
    S = ep.LLLayout(slot, None, None, 4, 1, 1)
    B = ep.LLLayout(slot + (rows - 4), None, None, rows, 1, 1)
    big, bigdh = torch.zeros((rows, 2 * N), dtype=BF16, device="cuda"), torch.zeros((rows, N), dtype=BF16, device="cuda")
    big[-4:], bigdh[-4:] = small, dh
    k, K = ep.alloc_checkpoint8(4, 2 * N, w.device), ep.alloc_checkpoint8(rows, 2 * N, w.device)
    assert torch.equal(ep.ll_swiglu(small, S, w, checkpoint=k), ep.ll_swiglu(big, B, w, checkpoint=K)[-4:])
    assert torch.equal(k.codes, K.codes[-4:]) and torch.equal(k.scales, K.scales[-4:])
    for kept, KEPT in ((k, K), (small, big)):
        d, dw = ep.ll_swiglu_backward(dh, kept, S, w)
        D, DW = ep.ll_swiglu_backward(bigdh, KEPT, B, w)
        assert torch.equal(d, D[-4:]) and torch.equal(dw, DW)


def test_repeats_and_two_captured_streams(ep):
    L, gu, dh, w = case(ep, 300, 16, 4, 512, seed=7)

    def step():
        kept = ep.alloc_checkpoint8(L.num_rows, 1024, gu.device)
        kept.codes.zero_()
        kept.scales.zero_()
        h = ep.ll_swiglu(gu, L, w, checkpoint=kept, out=torch.zeros_like(dh))
        return [h, kept.codes, kept.scales, *ep.ll_swiglu_backward(dh, kept, L, w)]

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
        step()
    torch.cuda.synchronize()
    for out in got:
        for a, b in zip(want, out):
            assert torch.equal(a, b)


def test_no_tokens_and_arguments(ep):
    L, gu, dh, w = case(ep, 4, 4, 2, 128)
    empty = ep.LLLayout(L.ll_slot[:0], None, None, 4, 1, 4)
    out = torch.full((L.num_rows, 128), 2.0, dtype=BF16, device="cuda")
    assert (ep.ll_swiglu(gu, empty, out=out) == 2.0).all()
    d, dw = ep.ll_swiglu_backward(dh, gu, empty, w[:0])
    assert not d.any() and dw.shape == (0, 2)
    kept = ep.alloc_checkpoint8(L.num_rows, 256, gu.device)
    short = ep.Checkpoint8(kept.codes[:-1], kept.scales[:-1])
    bad = [lambda: ep.ll_swiglu(gu.float(), L), lambda: ep.ll_swiglu(gu[:, :248].contiguous(), L, checkpoint=kept),
           lambda: ep.ll_swiglu(gu, L, w[:, :1]), lambda: ep.ll_swiglu(gu, L, checkpoint=short),
           lambda: ep.ll_swiglu(gu, L, out=dh[:-1]), lambda: ep.ll_swiglu(gu[:, :4], L),
           lambda: ep.ll_swiglu(gu, L, out=gu.view(-1)[:dh.numel()].view(dh.shape)),
           lambda: ep.ll_swiglu(gu.cpu(), L), lambda: ep.alloc_checkpoint8(4, 100, gu.device),
           lambda: ep.ll_swiglu_backward(dh, gu, L, out=gu), lambda: ep.ll_swiglu_backward(dh, short, L),
           lambda: ep.ll_swiglu_backward(dh, gu[:-1], L), lambda: ep.ll_swiglu_backward(gu, gu, L),
           lambda: ep.ll_swiglu_backward(dh, kept, L, w.double()),
           lambda: ep.ll_swiglu(gu[:-1], L), lambda: ep.ll_swiglu_backward(dh[:-1], gu[:-1], L)]
    for i, call in enumerate(bad):
        with pytest.raises(ep.EPError):
            call()
            print(i)


def test_formula_agrees_with_differences():
    gen = torch.Generator().manual_seed(0)
    step = 1e-5
    gu = torch.randn((3, 12), generator=gen, dtype=torch.float64) * 2
    dh, w = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((3, 6), (3,)))
    grad, dw, _, _ = ref.swiglu_grad(dh, gu, w)
    for at in range(12):
        d = torch.zeros_like(gu)
        d[:, at] = step
        num = ((ref.swiglu(gu + d, w) - ref.swiglu(gu - d, w)) * dh).sum(1) / (2 * step)
        assert (num - grad[:, at]).abs().max() < 1e-8
    num = ((ref.swiglu(gu, w + step) - ref.swiglu(gu, w - step)) * dh).sum(1) / (2 * step)
    assert (num - dw).abs().max() < 1e-8
