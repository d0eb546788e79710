"""The norms between two blocks with the new stream written over the old one."""
from __future__ import annotations

import os
import re

import pytest
import torch

from test_gpu_block_norm import BF16, F32, inputs, rand

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "combine_get_dispatch_04_gb300", "csrc", "ep_block_norm.cu")


def test_a_stream_that_is_written_is_not_read_through_the_read_only_path():
    """ld.global.nc is for memory that nobody writes while the kernel runs."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    forward = text[text.index("void finish_row"):text.index("norm_grad_row_kernel")]
    loads = re.findall(r"load(\S*)\(a\.x\b", forward)
    assert loads == ["<true>"], loads
    plain = text[text.index("void ld_written_32"):text.index("struct Stream8")]
    assert ".nc" not in plain and plain.count("ld.global.L1::no_allocate") == 2


# a warp a row, a block a row of two and of four vectors a thread
@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 8), (2001, 264), (1003, 1032), (701, 2056), (5003, 7168), (300, 16384)])
@pytest.mark.parametrize("stream", [BF16, F32])
@pytest.mark.parametrize("shift", [False, True])
def test_in_place(ep, T, H, stream, shift):
    s = inputs(T, H, "channel", stream, F32, seed=41)
    if shift:  # on a 16-byte, but no 32-byte boundary
        flat = torch.empty(T * H + 32, dtype=stream, device="cuda")
        s["x"] = flat[16 // flat.element_size():][:T * H].view(T, H).copy_(s["x"])
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"], scale=0.5)
    want = ep.block_norm(s["x"], s["y"], **kind)
    before = s["x"].clone()
    for _ in range(3):
        s["x"].copy_(before)
        got = ep.block_norm(s["x"], s["y"], out=s["x"], **kind)
        assert got.z.data_ptr() == s["x"].data_ptr()
        assert torch.equal(got.z, want.z) and torch.equal(got.h, want.h)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,K", [(3001, 7168, 8, 4), (9001, 264, 16, 6)])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_rows_in_place(ep, T, H, E, K, stream):
    s = inputs(T, H, "token", stream, F32, seed=42)
    idx = torch.rand((T, E), generator=s["gen"], device="cuda").topk(K).indices
    idx[torch.rand((T, K), generator=s["gen"], device="cuda") < 0.2] = -1
    L = ep.ll_get_dispatch_layout(idx, E, 1)
    rows = rand(s["gen"], L.num_rows, H, dtype=BF16)
    kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"], scale=0.5)
    want = ep.ll_combine_norm(rows, None, L, s["x"], **kind)
    got = ep.ll_combine_norm(rows, None, L, s["x"], out=s["x"], **kind)
    assert torch.equal(got.z, want.z) and torch.equal(got.h, want.h)
