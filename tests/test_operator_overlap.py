"""Host-side refusals of outputs that overlap the inputs they are computed from
(no GPU needed: the calls are refused before anything reaches CUDA, and the
pointers are never dereferenced)."""
from __future__ import annotations

import ctypes as C

import pytest

BAD = 1
A = 1 << 20


@pytest.fixture(scope="module")
def eplib():
    from combine_get_dispatch_04_gb300 import build
    build.build()
    import combine_get_dispatch_04_gb300 as ep
    return ep.load()


def p(address):
    return C.c_void_p(address)


def test_combine_backward(eplib):
    T, H, rows = 4, 64, 8  # dout: 512 bytes, y and dy: 1024
    far = p(A + (1 << 16))

    def rank(d, y, dy):
        return eplib.ep_combine_backward(d, y, H, rows, far, far, T, 2, 8, 4, far, dy, far, None, None)

    def expert(d, y, dy):
        return eplib.ep_ll_combine_backward(d, y, H, rows, far, T, 2, far, dy, far, None, None)

    for call in (rank, expert):
        assert call(p(A), p(A + 4096), p(A)) == BAD                # dy is dout
        assert call(p(A + 4096), p(A), p(A)) == BAD                # dy is y
        assert call(p(A + 1008), p(A + 4096), p(A)) == BAD         # dout begins in dy's last bytes
        assert call(p(A), p(A + 4096), p(A + 496)) == BAD          # dy begins in dout's last bytes
        assert call(p(A + 4096), p(A), p(A + 1008)) == BAD


def test_route_backward(eplib):
    T, E = 4, 16  # float32: 256 bytes; with a stride of 20: 304
    far = p(A + (1 << 16))

    def call(lg, dl, stride=E, bf16=0):
        return eplib.ep_route_backward(far, lg, bf16, stride, far, T, E, 4, 0, 1, 1.0, dl, None, None)

    assert call(p(A), p(A)) == BAD
    assert call(p(A), p(A + 240)) == BAD
    assert call(p(A + 240), p(A)) == BAD
    assert call(p(A), p(A + 288), stride=20) == BAD
    assert call(p(A), p(A + 112), bf16=1) == BAD


def test_experts(eplib):
    E, cap, I, N = 2, 4, 256, 64  # x: 4096 bytes (E4M3: 2048), y: 1024
    far = p(A + (1 << 16))

    def call(x, y, fp8=0):
        return eplib.ep_ll_experts_w4(x, fp8, far if fp8 else None, I, far, E, cap, far, far, None,
                                      128, N, 0, y, None, None)

    assert call(p(A), p(A)) == BAD
    assert call(p(A), p(A + 4080)) == BAD
    assert call(p(A + 1008), p(A)) == BAD
    assert call(p(A), p(A + 2032), fp8=1) == BAD


@pytest.mark.gpu
def test_buffers_side_by_side_are_taken(ep):
    import torch
    both = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    L = ep.LLLayout(torch.arange(4, dtype=torch.int32, device="cuda").reshape(4, 1), None, None, 1, 1, 4)
    d, w = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((4, 1), device="cuda")
    for y, out in ((both[0], both[1]), (both[1], both[0])):
        dy, _ = ep.ll_combine_backward(d, y, w, L, out=out)
        assert torch.equal(dy, d)
    with pytest.raises(ep.EPError):
        ep.ll_combine_backward(d, both[0], w, L, out=both[0])
    logits = torch.randn((2, 4, 16), device="cuda")
    idx, w = ep.route(logits[0], 4)
    want = ep.route_backward(w, logits[0], idx)
    assert torch.equal(ep.route_backward(w, logits[0], idx, out=logits[1]), want)
    with pytest.raises(ep.EPError):
        ep.route_backward(w, logits[0], idx, out=logits[0])
