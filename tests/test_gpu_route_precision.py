"""GPU: the router's gradient where float32 is tight: confident sigmoid scores,
and scores near the smallest that float32 holds.

Without renormalisation a gradient is scale * dw * s * (1 - s): two exponentials
(2 ulp each), two sums, two reciprocals and three products, 16 roundings of
2^-24 at most, so 1e-6 relative.  Below 2^-126 a factor is good to 2^-149."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def sigmoid64(l):
    return np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,K", [(16, 8), (600, 12)])
def test_gradient_of_confident_sigmoid_scores(ep, E, K, dtype):
    rng = np.random.default_rng(E)
    T = 64
    logits = (rng.uniform(8.0, 90.0, (T, E)) * rng.choice([-1.0, 1.0], (T, E))).astype(np.float32)
    logits[0] = 12.0
    logits[1] = 17.0
    lg = torch.from_numpy(logits).cuda().to(dtype)
    l64 = lg.double().cpu().numpy()
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int64)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = ep.route_backward(torch.from_numpy(dw).cuda(), lg, torch.from_numpy(ids).cuda(),
                            score="sigmoid", renormalize=False, scale=2.5).double().cpu().numpy()
    at = np.take_along_axis(l64, ids, 1)
    want = np.zeros((T, E))
    np.put_along_axis(want, ids, 2.5 * dw * sigmoid64(at) * sigmoid64(-at), 1)
    # 2^-126: what a subnormal factor or result may lose
    tol = 1e-6 * np.abs(want) + 2.0 ** -126 * 2.5 * np.abs(dw).max()
    lo, hi = want - tol, want + tol
    if dtype == torch.bfloat16:  # rounded once: between the roundings of the ends
        lo, hi = (torch.from_numpy(v).float().to(dtype).double().numpy() for v in (lo, hi))
    assert ((got >= lo) & (got <= hi)).all(), np.abs(got / np.where(want, want, 1) - 1).max()


@pytest.mark.parametrize("E,K", [(16, 4), (600, 12)])
def test_renormalised_gradient_of_the_smallest_sigmoid_scores(ep, E, K):
    """Scores of 3e-39 to 1e-38 (good to 2^-149: 5e-7) still have weights of order
    one, so the gradient is finite: w (dw - sum w dw) (1 - s), within 1e-5 of
    scale * max |dw|."""
    rng = np.random.default_rng(K)
    T = 40
    logits = rng.uniform(-88.6, -87.4, (T, E)).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int64)
    dw = (rng.standard_normal((T, K)) * 100).astype(np.float32)
    got = ep.route_backward(torch.from_numpy(dw).cuda(), torch.from_numpy(logits).cuda(),
                            torch.from_numpy(ids).cuda(), score="sigmoid").double().cpu().numpy()
    u = sigmoid64(np.take_along_axis(logits.astype(np.float64), ids, 1))
    w = u / u.sum(1, keepdims=True)
    want = np.zeros((T, E))
    np.put_along_axis(want, ids, w * (dw - (w * dw).sum(1, keepdims=True)) * (1 - u), 1)
    assert np.isfinite(got).all()
    assert np.abs(got - want).max() <= 1e-5 * np.abs(dw).max()
