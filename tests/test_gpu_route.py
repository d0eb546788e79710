"""GPU: the router and its gradient against the plain 64-bit forms.

Weights are float32 results of an exponential (2 ulp), its argument's rounding
(|l - max| * 2^-24 relative), a sum of at most 32 terms and two divisions or
multiplications: 4e-6 relative covers them for |l - max| <= 40.  A gradient is
a difference of such terms, each at most scale * max|dw|: 1e-5 of that bound,
plus one rounding for bfloat16 results (2^-8 relative).  Keys are compared
within 1e-6, and ties exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu


def run_route(ep, logits, K, **kw):
    idx, w = ep.route(logits, K, **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def check_route(logits, bias, idx, w, K, score, groups, keep, renorm, scale):
    """The choice by its keys (near ties may go either way), then the weights
    of the choice that was made."""
    T, E = logits.shape
    key = ref.route_keys(logits, score, bias)
    full = key
    if groups > 1:
        key, g = ref.keep_groups(full, score, groups, keep)
        # tokens whose group cut is a near tie: check only that the experts are allowed
        s = np.sort(g, axis=1)[:, ::-1]
        with np.errstate(invalid="ignore"):
            sure = ~(np.abs(s[:, keep - 1] - s[:, min(keep, groups - 1)]) < 1e-6) if keep < groups \
                else np.ones(T, bool)
    else:
        sure = np.ones(T, bool)
    best = -np.sort(-key, axis=1)[:, :K]
    got = np.where(idx >= 0, np.take_along_axis(key, np.maximum(idx, 0), 1), -np.inf)
    assert ((idx >= -1) & (idx < E)).all()
    fin = np.isfinite(best)
    assert np.array_equal(fin[sure], np.isfinite(got)[sure])
    d = np.abs(np.where(fin, best, 0) - np.where(fin, got, 0))[sure]
    assert (d <= 1e-6 * (1 + np.abs(np.where(fin, best, 0)[sure]))).all()
    for t in range(T):
        live = idx[t][idx[t] >= 0]
        assert len(set(live.tolist())) == len(live)
    want = ref.route_weights(logits, idx, score, renorm, scale)
    assert np.all(np.abs(w - want) <= 4e-6 * np.abs(want) + 1e-30)


SHAPES = [  # T, E, K, groups, kept groups
    (1, 1, 1, 1, 1), (3, 8, 2, 1, 1), (37, 16, 4, 4, 2), (130, 60, 4, 1, 1), (9, 60, 6, 5, 2),
    (65, 64, 6, 8, 3), (50, 96, 8, 3, 2), (33, 128, 8, 4, 1), (64, 160, 6, 8, 3), (5, 160, 6, 4, 2),
    (131, 256, 8, 8, 4), (7, 256, 32, 16, 16), (12, 257, 5, 1, 1), (6, 512, 10, 64, 7),
    (5, 1000, 16, 1, 1), (4, 1030, 8, 10, 3), (3, 4096, 32, 64, 9), (2, 24, 24, 1, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,G,keep", SHAPES)
def test_route_shapes(ep, T, E, K, G, keep, score, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    for with_bias in (False, True):
        for renorm in (False, True):
            logits = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).cuda().to(dtype)
            logits[torch.rand((T, E), device="cuda") < 0.05] = float("-inf")
            bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * 0.2).cuda() \
                if with_bias else None
            idx, w = run_route(ep, logits, K, score=score, bias=bias, num_groups=G, topk_groups=keep,
                               renormalize=renorm, scale=2.5)
            check_route(logits.float().cpu().numpy(), None if bias is None else bias.cpu().numpy(),
                        idx, w, K, score, G, keep, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,G,keep", [(16, 16, 1, 1), (64, 6, 8, 3), (60, 7, 6, 2), (256, 8, 1, 1),
                                        (1024, 9, 1, 1), (513, 9, 3, 2)])
def test_route_ties_go_to_the_lowest_index(ep, E, K, G, keep, score):
    rng = np.random.default_rng(E + K)
    logits = rng.integers(-1, 2, (200, E)).astype(np.float32)
    logits[0] = 0.0
    logits[1, ::2] = -0.0  # equal to +0
    logits[1, 1::2] = 0.0
    idx, _ = run_route(ep, torch.from_numpy(logits).cuda(), K, score=score, num_groups=G,
                       topk_groups=keep)
    key = ref.route_keys(logits, score)
    if score == "sigmoid":  # equal logits have equal float32 scores: compare in float32
        key = key.astype(np.float32).astype(np.float64)
    if G > 1:
        key, _ = ref.keep_groups(key, score, G, keep)
    assert np.array_equal(idx, ref.choose(key, K))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,G,keep", [(16, 1, 1), (16, 4, 2), (15, 3, 2), (600, 1, 1)])
def test_route_special_rows(ep, E, G, keep, score, renorm):
    """Rows that a mask empties, in part or whole, and rows of extremes."""
    lowest = float(np.finfo(np.float32).min)
    rng = np.random.default_rng(E)
    x = rng.standard_normal((12, E)).astype(np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, E // 2] = 0.5          # one expert left
    x[3, ::2] = np.nan
    x[4] = lowest               # finite, so it may be chosen
    x[5] = lowest
    x[5, E - 1] = 1.0
    x[6, 1] = np.inf
    x[7, 1] = x[7, 3] = np.inf
    x[8] = np.inf
    x[9, :] = -np.inf
    x[9, [0, E - 1]] = [lowest, -np.inf]
    x[10, 0] = -200.0
    idx, w = run_route(ep, torch.from_numpy(x).cuda(), 4, score=score, num_groups=G,
                       topk_groups=keep, renormalize=renorm)
    assert np.isfinite(w).all()
    assert (idx[0] == -1).all() and (idx[1] == -1).all() and (w[:2] == 0).all()
    assert idx[2, 0] == E // 2 and (idx[2, 1:] == -1).all()
    assert not np.isin(idx[3], np.arange(0, E, 2)).any()
    key = ref.route_keys(x, score)
    if G > 1:
        key = ref.keep_groups(key, score, G, keep)[0]
    exact = [0, 1, 2, 4, 5, 9] + ([6, 7, 8] if score == "softmax" else [])
    assert np.array_equal(idx[exact], ref.choose(key, 4)[exact])
    want = ref.route_weights(x, idx, score, renorm, 1.0)
    assert np.all(np.abs(w - want) <= 4e-6 * np.abs(want) + 1e-30)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("E,K", [(1, 1), (7, 3), (8, 8), (32, 8), (33, 5), (64, 6), (100, 8), (256, 8),
                                 (257, 8), (1000, 7), (1024, 8), (1025, 8), (256, 9)])
def test_route_bf16_keys(ep, E, K, offset, renorm):
    """Ties, zeros of both signs, NaN of both signs, infinities, the largest
    and the smallest numbers, in rows aligned or not (offset)."""
    rng = np.random.default_rng(E + K)
    x = rng.integers(-2, 3, (70, E)).astype(np.float32)
    x[x == 0] *= rng.choice([-1.0, 1.0], (x == 0).sum())
    x[1] = -np.inf
    x[2] = np.nan
    x[3] = np.copysign(np.nan, -1)
    x[4, ::2] = -np.inf
    x[5, ::3] = np.nan
    x[6, ::3] = np.copysign(np.nan, -1)
    x[7, -1] = np.inf
    x[8] = 2.0 ** -133 * rng.integers(-3, 4, E)  # subnormal
    x[9] = np.where(rng.random(E) < 0.5, -3.3895314e38, 3.3895314e38)
    x[10] = rng.standard_normal(E)
    buf = torch.full((70, E + 8 - E % 8 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    logits = buf[:, offset:offset + E]
    logits.copy_(torch.from_numpy(x))
    idx, w = run_route(ep, logits, K, renormalize=renorm, scale=0.5)
    back = logits.float().cpu().numpy()
    assert np.array_equal(idx, ref.choose(ref.route_keys(back, "softmax"), K))
    want = ref.route_weights(back, idx, "softmax", renorm, 0.5)
    assert np.all(np.abs(w - want) <= 4e-6 * np.abs(want) + 1e-30)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep", [(16, 1, 1), (16, 4, 2), (600, 1, 1), (600, 4, 2)])
def test_route_bias_that_rules_experts_out(ep, E, G, keep, score):
    rng = np.random.default_rng(E + G)
    x = rng.standard_normal((40, E)).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    bias[::2] = -np.inf
    bias[1] = np.nan
    bias[E // 2:] = -np.inf  # with groups: some have no expert left
    idx, w = run_route(ep, torch.from_numpy(x).cuda(), 4, score=score, num_groups=G,
                       topk_groups=keep, bias=torch.from_numpy(bias).cuda())
    live = idx[idx >= 0]
    assert np.isfinite(bias[live]).all() and np.isfinite(w).all() and (w[idx < 0] == 0).all()
    left = np.isfinite(bias).reshape(G, -1).sum(1)
    assert ((idx >= 0).sum(1) <= min(4, left.sum())).all()
    if G == 1:
        assert ((idx >= 0).sum(1) == min(4, left.sum())).all()
    want = ref.route_weights(x, idx, score, True, 1.0)
    assert np.all(np.abs(w - want) <= 4e-6 * np.abs(want) + 1e-30)


def test_route_strided_and_unaligned_logits(ep):
    base = torch.randn((41, 300), device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        wide = base.to(dtype)
        for start in (0, 1, 3):
            view = wide[:, start:start + 256]
            assert not view.is_contiguous()
            a = ep.route(view, 8, score="sigmoid", num_groups=8, topk_groups=4)
            b = ep.route(view.contiguous(), 8, score="sigmoid", num_groups=8, topk_groups=4)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            dw = torch.randn((41, 8), device="cuda")
            for kw in (dict(score="sigmoid"), dict(score="softmax", renormalize=False)):
                assert torch.equal(ep.route_backward(dw, view, a[0], **kw),
                                   ep.route_backward(dw, view.contiguous(), a[0], **kw))


def test_route_empty_and_outputs_given(ep):
    idx, w = ep.route(torch.empty((0, 16), device="cuda"), 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    assert ep.route_backward(w, torch.empty((0, 16), device="cuda"), idx).shape == (0, 16)
    logits = torch.randn((5, 16), device="cuda")
    out = (torch.full((5, 4), 99, dtype=torch.int64, device="cuda"), torch.empty((5, 4), device="cuda"))
    got = ep.route(logits, 4, out=out)
    assert got[0] is out[0] and (out[0] < 16).all()


def test_route_on_another_stream(ep):
    logits = torch.randn((4096, 256), device="cuda")
    want = ep.route(logits, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = ep.route(logits, 8)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def grad_close(got, want, dw, scale, bf16):
    bound = 1e-5 * scale * np.abs(np.where(np.isfinite(dw), dw, 0)).max(1, keepdims=True) * dw.shape[1]
    lim = bound + (2.0 ** -8 * np.abs(want) if bf16 else 0.0)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= lim).all(), np.abs(got - want).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (5, 8, 2), (130, 60, 4), (65, 64, 6), (33, 256, 8),
                                   (9, 257, 5), (4, 1000, 32), (3, 4096, 8), (6, 63, 3)])
def test_route_backward(ep, T, E, K, score, renorm, dtype):
    rng = np.random.default_rng(T + E)
    logits = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).cuda().to(dtype)
    idx, _ = ep.route(logits, K, score=score)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    ids = idx.cpu().numpy()
    if K > 1:
        ids[::3, 1] = -1                # masked slots
        if T > 4:
            ids[4] = -1                 # a row with nothing left
    got = ep.route_backward(torch.from_numpy(dw).cuda(), logits, torch.from_numpy(ids).cuda(),
                            score=score, renormalize=renorm, scale=1.5)
    want = ref.route_grad(dw, logits.float().cpu().numpy(), ids, score, renorm, 1.5)
    assert got.dtype == dtype
    grad_close(got.float().cpu().numpy(), want, dw, 1.5, dtype == torch.bfloat16)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_duplicates_bad_ids_and_masked_logits(ep, score, renorm):
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((40, 16)).astype(np.float32)
    logits[3, 2] = -np.inf
    logits[4, 5] = np.nan
    logits[5] = -np.inf
    ids = rng.integers(0, 16, (40, 6)).astype(np.int64)
    ids[0] = 7
    ids[3, 0], ids[4, 0] = 2, 5
    ids[6, 1], ids[7, 2] = 16, -5
    dw = rng.standard_normal((40, 6)).astype(np.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ep.route_backward(torch.from_numpy(dw).cuda(), torch.from_numpy(logits).cuda(),
                            torch.from_numpy(ids).cuda(), score=score, renormalize=renorm, err=err)
    assert int(err.item()) == ep.EP_ERRBIT_BAD_EXPERT
    # a slot at -inf or NaN is taken as masked
    off = ~(np.take_along_axis(logits, np.clip(ids, 0, 15), 1) > -np.inf)
    clean = np.where((ids < 0) | (ids > 15) | off, -1, ids)
    want = ref.route_grad(dw, logits, clean, score, renorm, 1.0)
    grad_close(got.cpu().numpy(), want, dw, 1.0, False)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_against_differences(ep, score, renorm):
    """Central differences of the 64-bit weights at a fixed choice: the
    truncation error is h^2 / 6 times a third derivative of order one."""
    rng = np.random.default_rng(11)
    T, E, K, h = 7, 12, 4, 1e-4
    logits = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    lg = torch.from_numpy(logits).cuda()
    idx, _ = ep.route(lg, K, score=score)
    got = ep.route_backward(torch.from_numpy(dw).cuda(), lg, idx, score=score, renormalize=renorm,
                            scale=2.0).cpu().numpy()
    ids, diff = idx.cpu().numpy(), np.zeros((T, E))
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        up = ref.route_weights(logits.astype(np.float64) + d, ids, score, renorm, 2.0)
        dn = ref.route_weights(logits.astype(np.float64) - d, ids, score, renorm, 2.0)
        diff[:, e] = ((up - dn) * dw).sum(1) / (2 * h)
    assert np.abs(got - diff).max() <= 1e-5 * 2.0 * np.abs(dw).max() * K


def test_route_refusals(ep):
    lg = torch.randn((4, 16), device="cuda")
    with pytest.raises(ep.EPError):
        ep.route(lg, 17)                                   # more slots than experts
    with pytest.raises(ep.EPError):
        ep.route(lg, 0)
    with pytest.raises(ep.EPError):
        ep.route(lg, 4, score="none")
    with pytest.raises(ep.EPError):
        ep.route(lg, 4, num_groups=3)                      # does not divide the experts
    with pytest.raises(ep.EPError):
        ep.route(lg, 4, num_groups=4, topk_groups=5)
    with pytest.raises(ep.EPError):
        ep.route(lg.half(), 4)
    with pytest.raises(ep.EPError):
        ep.route(lg.t(), 2)                                # strided along the experts
    with pytest.raises(ep.EPError):
        ep.route(lg[:1].expand(4, 16), 4)                  # rows overlap
    with pytest.raises(ep.EPError):
        ep.route(lg, 4, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ep.EPError):
        ep.route(lg.cpu(), 4)
    idx, w = ep.route(lg, 4)
    with pytest.raises(ep.EPError):
        ep.route_backward(w[:, :3], lg, idx)
    with pytest.raises(ep.EPError):
        ep.route_backward(w, lg, idx.int())
