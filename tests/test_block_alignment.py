"""Slots, top-k weights, their gradient and error words that are not on a 4-byte boundary are refused by
the norms between two blocks and the gated activation before anything reaches CUDA (no GPU needed:
pointers are never dereferenced)."""
from __future__ import annotations

import pytest

from test_block_arguments import BAD, at, eplib  # noqa: F401


@pytest.mark.parametrize("odd", [1, 2, 3])
def test_four_byte_boundaries(eplib, odd):  # noqa: F811
    def norm(slot=at(7), w=at(8), err=at(9)):
        return eplib.ep_block_norm(at(1), 0, at(2), 8, w, 2, slot, 4, 64, None, 0, at(3), at(4), 0, 1.0,
                                   1e-6, at(5), at(6), None, err, None)

    def swiglu(slot=at(2), w=at(6), err=at(9)):
        return eplib.ep_ll_swiglu(at(1), 128, 8, w, 4, 2, slot, at(3), at(4), at(5), err, None)

    def grad(slot=at(5), w=at(4), err=at(9), dw=at(7)):
        return eplib.ep_ll_swiglu_backward(at(1), None, at(2), at(3), 128, 8, w, 4, 2, slot, at(6), dw, err,
                                           None)

    for call in (norm, swiglu, grad):
        for kw in (dict(slot=at(10, odd)), dict(w=at(11, odd)), dict(err=at(12, odd))):
            assert call(**kw) == BAD, (call.__name__, kw)
    assert grad(dw=at(13, odd)) == BAD
