"""Plain 64-bit forms (torch) of the layer for a few tokens, the norms between two
blocks and the gated activation, written from their definitions for the tests,
together with the sums of magnitudes that bound a 32-bit computation's error."""
from __future__ import annotations

import torch

F = torch.float64


def half_step(dtype: torch.dtype) -> float:
    """A rounding to `dtype` is off by at most this, relative to the value."""
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# norms between two blocks
# ---------------------------------------------------------------------------
def rms(v, eps):
    return torch.sqrt(v.square().mean(1, keepdim=True) + eps)


def block_norm(x, y, gate, post, pre, scale, eps):
    """z, h (None without pre) and the magnitudes |x| + |v| that z is added up from."""
    x = x.to(F)
    v = torch.zeros_like(x)
    if y is not None:
        v = y.to(F)
        if post is not None:
            v = v / rms(v, eps) * post.to(F)
        v = scale * v * (1.0 if gate is None else gate.to(F))
    z = x + v
    h = None if pre is None else z / rms(z, eps) * pre.to(F)
    return z, h, x.abs() + v.abs()


def block_norm_grad(dz, dh, z, y, gate, post, pre, scale, eps):
    """The gradient's formula, and for every result the sum of the magnitudes of its terms."""
    z = z.to(F)
    t = torch.zeros_like(z) if dz is None else dz.to(F)
    tm = t.abs()
    out, mag = {}, {}
    if dh is not None:
        r = 1.0 / rms(z, eps)
        d = dh.to(F) * pre.to(F)
        out["dpre_weight"] = (dh.to(F) * z * r).sum(0)
        mag["dpre_weight"] = (dh.to(F) * z * r).abs().sum(0)
        t = t + r * d - r ** 3 * (z * d).mean(1, keepdim=True) * z
        tm = tm + r * d.abs() + r ** 3 * (z * d).abs().mean(1, keepdim=True) * z.abs()
    out["dx"], mag["dx"] = t, tm
    g = torch.ones((), dtype=F, device=z.device) if gate is None else gate.to(F)
    n = None
    if y is not None:
        y = y.to(F)
        n = y
        if post is not None:
            ry = 1.0 / rms(y, eps)
            n = y * ry * post.to(F)
    if gate is not None:
        term, tmag = scale * n * t, (scale * n).abs() * tm
        if gate.dim() == 1:
            out["dgate"], mag["dgate"] = term.sum(0), tmag.sum(0)
        elif gate.shape[1] == 1 and z.shape[1] != 1:
            out["dgate"], mag["dgate"] = term.sum(1, keepdim=True), tmag.sum(1, keepdim=True)
        else:
            out["dgate"], mag["dgate"] = term, tmag
    dn, dm = scale * g * t, (scale * g).abs() * tm
    if post is not None:
        out["dpost_weight"], mag["dpost_weight"] = (dn * y * ry).sum(0), (dm * (y * ry).abs()).sum(0)
        p = post.to(F)
        out["dy"] = ry * dn * p - ry ** 3 * (y * dn * p).mean(1, keepdim=True) * y
        mag["dy"] = (ry * dm * p.abs()
                     + ry ** 3 * (y.abs() * dm * p.abs()).mean(1, keepdim=True) * y.abs())
    else:
        out["dy"], mag["dy"] = dn, dm
    return out, mag


# ---------------------------------------------------------------------------
# gated activation
# ---------------------------------------------------------------------------
def to_8_bits(v):
    """The FP8 dispatch's rounding of bf16 rows: every step in float32, rounded once
    (divisions of two tensors: torch multiplies by a reciprocal where one side is a number)."""
    blocks = v.float().unflatten(1, (-1, 128))
    top = blocks.abs().amax(-1).clamp(min=1e-4)
    most = torch.full_like(top, 448.0)
    codes = (blocks * (most / top)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.flatten(1).view(torch.uint8), top / most


def from_8_bits(codes, scales):
    """Float32 values that the codes stand for (one rounding, as the kernel's)."""
    v = codes.view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128))
    return (v * scales[..., None]).flatten(1)


def swiglu(gate_up, w):
    g, u = gate_up.to(F).chunk(2, dim=1)
    return w.to(F)[:, None] * g * torch.sigmoid(g) * u


def swiglu_grad(dh, gate_up, w):
    """dgate_up, dw (one per row) and the magnitudes of their terms."""
    g, u = gate_up.to(F).chunk(2, dim=1)
    s, o, d = torch.sigmoid(g), torch.sigmoid(-g), dh.to(F)
    wd = w.to(F)[:, None] * d
    grad = torch.cat((wd * u * (s + g * s * o), wd * g * s), 1)
    mag = torch.cat(((wd * u).abs() * (s + g.abs() * s * o), (wd * g * s).abs()), 1)
    return grad, (d * g * s * u).sum(1), mag, (d * g * s * u).abs().sum(1)


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------
def w4(weights, e):
    """The matrix of expert e in 64 bits."""
    q = weights.q[e]
    codes = torch.stack((q & 15, q >> 4), -1).flatten(1).to(F)
    group = codes.shape[1] // weights.scales.shape[2]
    zero = 8.0 if weights.zeros is None else (weights.zeros[e] & 15).to(F).repeat_interleave(group, 1)
    return (codes - zero) * weights.scales[e].to(F).repeat_interleave(group, 1)


def layer(x, idx, w, gate_up, down):
    """out, and a bound of what float32 sums of the two products may be off.

    A product's float32 sum: every group is a chain of 8 (or fewer) matrix instructions of 16 products
    each, scaled and added to the tile's sum, which up to 16 parts join.  A matrix
    instruction may cut what it adds instead of rounding it, so each of the
    chain's links counts 2^-22 of the sum of the magnitudes.  h is off by its
    factors' errors (the slope of silu is at most 1.1), 16 units of 2^-24 for the exponential,
    the divisions and the weight, and 2^-17 for what is left of it beyond two bf16.
    """
    T, H = x.shape
    out = torch.zeros((T, H), dtype=F, device=x.device)
    off = torch.zeros_like(out)

    def links(weights):
        return (8 + weights.scales.shape[2] + 16 + 2) * 2.0 ** -22

    for t in range(T):
        for k in range(idx.shape[1]):
            e = int(idx[t, k])
            if e < 0:
                continue
            m, v = w4(gate_up, e), x[t].to(F)
            p, pm = m @ v, (m.abs() @ v.abs()) * links(gate_up)
            N = p.shape[0] // 2
            silu = p[:N] * torch.sigmoid(p[:N])
            h = w[t, k].to(F) * silu * p[N:]
            hm = w[t, k].to(F).abs() * (1.1 * pm[:N] * (p[N:].abs() + pm[N:]) + silu.abs() * pm[N:])
            hm = hm + h.abs() * (16 * 2.0 ** -24 + 2.0 ** -17)
            d = w4(down, e)
            out[t] += d @ h
            # the down product adds up all chosen experts in one chain
            off[t] += d.abs() @ hm + idx.shape[1] * links(down) * (d.abs() @ h.abs())
    return out, off
