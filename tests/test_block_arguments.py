"""Host-side argument checks of the layer for a few tokens, the norms between two
blocks and the gated activation: bad calls are refused before anything reaches
CUDA (no GPU needed; pointers are never dereferenced)."""
from __future__ import annotations

import ctypes as C

import pytest

BAD, SMALL = 1, 2


@pytest.fixture(scope="module")
def eplib():
    from combine_get_dispatch_04_gb300 import build
    build.build()
    import combine_get_dispatch_04_gb300 as ep
    return ep.load()


def at(n, odd=0):
    """A pointer to a buffer of its own: no two are less than 2^30 bytes apart."""
    return C.c_void_p((n << 30) + odd)


ODD = at(50, 2)


def test_layer_arguments(eplib):
    def call(x=at(1), H=256, N=128, T=4, lg=at(2), bf16=0, stride=16, bias=None, E=16, K=4, score=1, G=1,
             keep=1, q=at(3), s=at(4), z=None, group=128, q2=at(5), s2=at(6), z2=None, group2=64,
             idx=at(7), w=at(8), out=at(9), ws=at(10), n=1 << 24):
        return eplib.ep_layer_w4(x, H, N, T, lg, bf16, stride, bias, E, K, score, G, keep, 1, 1.0, q, s, z,
                                 group, q2, s2, z2, group2, idx, w, out, ws, n, None)
    for kw in (dict(x=None), dict(x=ODD), dict(H=0), dict(H=192), dict(H=130), dict(N=0), dict(N=96),
               dict(T=-1), dict(T=17), dict(lg=None), dict(lg=ODD), dict(stride=15), dict(bias=ODD),
               dict(E=0, stride=0), dict(E=513, stride=2000), dict(K=0), dict(K=17), dict(E=64, stride=64, K=33),
               dict(score=2), dict(G=3), dict(G=0), dict(G=4, keep=0), dict(G=4, keep=5), dict(q=None),
               dict(q=ODD), dict(s=None), dict(s=ODD), dict(z=ODD), dict(group=16), dict(group=0),
               dict(q2=None), dict(q2=ODD), dict(s2=None), dict(z2=ODD), dict(group2=48), dict(idx=None),
               dict(idx=ODD), dict(w=None), dict(w=ODD), dict(out=None), dict(out=ODD), dict(ws=None),
               dict(ws=ODD), dict(H=1 << 16, N=1 << 16), dict(idx=at(1)), dict(w=at(2)),
               dict(out=at(2)), dict(out=at(10)), dict(ws=at(1)), dict(w=at(7)), dict(out=at(7, 64)),
               dict(out=at(3)), dict(ws=at(5)), dict(idx=at(4)), dict(out=at(6, 16)),
               dict(bias=at(11), out=at(11))):
        assert call(**kw) == BAD, kw
    need = eplib.ep_layer_w4_workspace_bytes(4, 128, 4)
    assert need > 2 * 2 * 16 * 128
    assert call(n=need - 1) == SMALL
    assert call(T=0, x=None, lg=None, idx=None, w=None, out=None, ws=None, n=0) == 0
    for bad in ((0, 128, 4), (17, 128, 4), (4, 0, 4), (4, 128, 0), (4, 128, 33)):
        assert eplib.ep_layer_w4_workspace_bytes(*bad) == 0


def test_block_norm_arguments(eplib):
    def call(x=at(1), f32=0, y=at(2), rows=0, w=None, K=0, slot=None, T=4, H=64, gate=None, kind=0,
             post=at(3), pre=at(4), scale=1.0, eps=1e-6, z=at(5), h=at(6), comb=None):
        return eplib.ep_block_norm(x, f32, y, rows, w, K, slot, T, H, gate, kind, post, pre, 0, scale, eps,
                                   z, h, comb, None, None)
    rows = dict(slot=at(7), K=2, rows=8)
    for kw in (dict(x=None), dict(x=ODD), dict(y=ODD), dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=12),
               dict(H=16392), dict(kind=1), dict(gate=at(8)), dict(kind=4, gate=at(8)), dict(kind=-1),
               dict(kind=1, gate=ODD), dict(kind=2, gate=at(8, 2)), dict(post=ODD), dict(pre=ODD),
               dict(pre=None), dict(h=None), dict(z=None), dict(y=None), dict(y=None, z=None),
               dict(y=None, z=None, post=None, pre=None, h=None), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(z=ODD), dict(h=ODD), dict(comb=at(9)), dict(w=at(9)),
               dict(rows, K=0), dict(rows, K=33), dict(rows, rows=-1), dict(rows, rows=1 << 31),
               dict(rows, y=None), dict(rows, comb=ODD), dict(rows, comb=at(2)), dict(rows, comb=at(6)),
               dict(z=at(2)), dict(z=at(1, 64)), dict(h=at(1)), dict(h=at(2, 128)), dict(h=at(5)),
               dict(kind=3, gate=at(5, 16)), dict(z=at(3)), dict(h=at(4)), dict(rows, h=at(7)),
               dict(rows, w=at(8), z=at(8))):
        assert call(**kw) == BAD, kw
    assert call(T=0, x=None, y=None, z=None, h=None, post=None, pre=None) == 0


def test_block_norm_backward_arguments(eplib):
    def call(dz=at(1), dh=at(2), z=at(3), f32=0, y=at(4), T=4, H=64, gate=None, kind=0, post=at(5),
             pre=at(6), eps=1e-6, dx=at(7), dy=at(8), dgate=None, dpost=at(10), dpre=at(11), ws=at(12),
             n=1 << 24):
        return eplib.ep_block_norm_backward(dz, dh, z, f32, y, T, H, gate, kind, post, pre, 0, 1.0, eps,
                                            dx, dy, dgate, dpost, dpre, ws, n, None)
    for kw in (dict(dz=ODD), dict(dh=ODD), dict(dh=None), dict(pre=None), dict(z=None), dict(z=ODD),
               dict(y=None), dict(y=ODD), dict(T=-1), dict(H=4), dict(H=1 << 15), dict(kind=2),
               dict(kind=5, gate=at(9)), dict(gate=at(9)), dict(post=None), dict(eps=0.0), dict(dx=None),
               dict(dx=ODD), dict(dy=ODD), dict(dgate=at(13)), dict(dpost=ODD), dict(dpre=ODD),
               dict(dz=None, dh=None, pre=None, dpre=None), dict(dx=at(1)), dict(dx=at(3, 16)),
               dict(dy=at(4)), dict(dy=at(2, 64)), dict(dy=at(7)), dict(ws=ODD),
               dict(kind=3, gate=at(9), dgate=at(9)), dict(dpost=at(5)), dict(dpre=at(10)), dict(ws=at(7)),
               dict(dx=at(6))):
        assert call(**kw) == BAD, kw
    for bad in ((0, 64), (-1, 64), (4, 12), (4, 1 << 15)):
        assert eplib.ep_block_norm_backward_workspace_bytes(*bad) == 0


def test_swiglu_arguments(eplib):
    def call(gu=at(1), N=128, rows=8, w=None, T=4, K=2, slot=at(2), h=at(3), c=at(4), s=at(5)):
        return eplib.ep_ll_swiglu(gu, N, rows, w, T, K, slot, h, c, s, None, None)
    for kw in (dict(gu=None), dict(gu=ODD), dict(N=0), dict(N=12), dict(N=64), dict(N=136), dict(rows=-1),
               dict(rows=1 << 31), dict(T=-1), dict(K=0), dict(K=33), dict(T=1 << 30, K=8), dict(slot=None),
               dict(h=None), dict(h=ODD), dict(c=None), dict(s=None), dict(c=ODD), dict(s=ODD),
               dict(h=at(1)), dict(c=at(1, 16)), dict(s=at(3)), dict(c=at(3)), dict(s=at(4, 32)), dict(h=at(2)),
               dict(w=at(6), c=at(6))):
        assert call(**kw) == BAD, kw
    assert call(T=0, gu=None, slot=None, h=None) == 0

    def back(dh=at(1), gu=None, c=at(2), s=at(3), N=128, rows=8, w=at(4), T=4, K=2, slot=at(5), d=at(6), dw=at(7)):
        return eplib.ep_ll_swiglu_backward(dh, gu, c, s, N, rows, w, T, K, slot, d, dw, None, None)
    for kw in (dict(dh=None), dict(dh=ODD), dict(gu=at(8)), dict(c=None), dict(s=None), dict(c=None, s=None),
               dict(c=ODD), dict(s=ODD), dict(N=64), dict(N=0), dict(rows=-1), dict(T=-1), dict(K=33),
               dict(slot=None), dict(d=None), dict(d=ODD), dict(d=at(1)), dict(d=at(2, 16)),
               dict(d=at(3)), dict(c=None, s=None, gu=at(6)), dict(c=None, s=None, gu=ODD), dict(d=at(4)),
               dict(dw=at(4)), dict(dw=at(5)), dict(dw=at(6))):
        assert back(**kw) == BAD, kw
    assert back(T=0, dh=None, d=None, slot=None) == 0


def test_streams_without_rows_are_refused(eplib):
    import torch

    import combine_get_dispatch_04_gb300 as ep
    w = torch.ones(8)
    for x in (torch.zeros(()), torch.zeros(8)):
        for call in (lambda: ep.block_norm(x, pre_weight=w), lambda: ep.block_norm(x, x),
                     lambda: ep.block_norm_backward(x, None, x)):
            with pytest.raises(ep.EPError):
                call()
