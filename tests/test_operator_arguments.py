"""Host-side argument checks of the router, the combine's gradient and the
experts' products: bad calls are refused before anything reaches CUDA (no GPU
needed; pointers are never dereferenced)."""
from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

import ops_reference as ref

BAD = 1


@pytest.fixture(scope="module")
def eplib():
    from combine_get_dispatch_04_gb300 import build
    build.build()
    import combine_get_dispatch_04_gb300 as ep
    return ep.load()


P, ODD = C.c_void_p(4096), C.c_void_p(4098)


def test_route_arguments(eplib):
    def call(lg=P, bf16=0, stride=16, bias=None, T=4, E=16, K=4, score=1, G=1, keep=1, idx=P, w=P):
        return eplib.ep_route(lg, bf16, stride, bias, T, E, K, score, G, keep, 1, 1.0, idx, w, None)
    for kw in (dict(lg=None), dict(lg=ODD), dict(stride=15), dict(T=-1), dict(E=0, stride=0),
               dict(E=4097, stride=5000), dict(K=0), dict(K=17), dict(E=64, stride=64, K=33), dict(score=2),
               dict(G=3), dict(G=0), dict(G=4, keep=0), dict(G=4, keep=5), dict(idx=None),
               dict(w=ODD), dict(bias=ODD), dict(E=256, stride=256, G=128)):
        assert call(**kw) == BAD, kw
    assert call(T=0, lg=None, idx=None, w=None) == 0


def test_route_backward_arguments(eplib):
    def call(dw=P, lg=P, stride=16, idx=P, T=4, E=16, K=4, score=0, dl=P):
        return eplib.ep_route_backward(dw, lg, 0, stride, idx, T, E, K, score, 1, 1.0, dl, None, None)
    for kw in (dict(dw=None), dict(lg=None), dict(stride=8), dict(idx=ODD), dict(K=0), dict(K=33),
               dict(score=-1), dict(dl=None), dict(dl=ODD)):
        assert call(**kw) == BAD, kw
    assert call(T=0, dw=None, lg=None, idx=None, dl=None) == 0


def test_combine_backward_arguments(eplib):
    def call(d=P, y=P, H=64, rows=8, idx=P, w=P, T=4, K=2, E=8, R=4, slot=P, dy=P, dw=P):
        return eplib.ep_combine_backward(d, y, H, rows, idx, w, T, K, E, R, slot, dy, dw, None, None)
    for kw in (dict(d=None), dict(d=ODD), dict(y=ODD), dict(y=None), dict(H=12), dict(H=0),
               dict(rows=-1), dict(rows=1 << 31), dict(idx=None), dict(w=None), dict(T=-4),
               dict(K=33), dict(E=7), dict(R=65, E=65), dict(slot=None), dict(dy=ODD)):
        assert call(**kw) == BAD, kw
    assert call(T=0, d=None, y=None, idx=None, w=None, slot=None) == 0
    assert call(dy=None, dw=None) == 0  # nothing asked for

    def ll(d=P, y=P, H=64, rows=8, w=P, T=4, K=2, slot=P, dy=P, dw=P):
        return eplib.ep_ll_combine_backward(d, y, H, rows, w, T, K, slot, dy, dw, None, None)
    for kw in (dict(d=None), dict(y=None), dict(H=4), dict(w=None), dict(slot=None), dict(K=0),
               dict(dy=ODD), dict(rows=-1)):
        assert ll(**kw) == BAD, kw
    assert ll(T=0, d=None, y=None, w=None, slot=None) == 0


def test_experts_arguments(eplib):
    def call(x=P, fp8=0, xs=None, I=256, cnt=P, E=4, cap=8, q=P, sc=P, z=None, group=128, N=64,
             act=0, y=P):
        return eplib.ep_ll_experts_w4(x, fp8, xs, I, cnt, E, cap, q, sc, z, group, N, act, y, None, None)
    for kw in (dict(x=None), dict(x=ODD), dict(fp8=1), dict(fp8=1, xs=P, I=192, group=64), dict(I=0),
               dict(I=192), dict(cnt=None), dict(E=0), dict(E=4097), dict(cap=-1), dict(cap=1 << 30),
               dict(q=None), dict(q=ODD), dict(sc=None), dict(z=ODD), dict(group=16), dict(N=0),
               dict(N=12), dict(act=2), dict(y=None)):
        assert call(**kw) == BAD, kw
    assert call(cap=0, x=None, y=None) == 0


def test_plain_gradient_agrees_with_differences():
    """The 64-bit gradient that the GPU tests compare with, against central
    differences of the 64-bit weights (error h^2 / 6 of a third derivative)."""
    rng = np.random.default_rng(0)
    T, E, K, h = 5, 10, 3, 1e-5
    lg, dw = rng.standard_normal((T, E)), rng.standard_normal((T, K))
    idx = ref.choose(lg, K)
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            g = ref.route_grad(dw, lg, idx, kind, renorm, 1.5)
            for e in range(E):
                d = np.zeros((T, E))
                d[:, e] = h
                num = ((ref.route_weights(lg + d, idx, kind, renorm, 1.5)
                        - ref.route_weights(lg - d, idx, kind, renorm, 1.5)) * dw).sum(1) / (2 * h)
                assert np.abs(g[:, e] - num).max() < 1e-8
