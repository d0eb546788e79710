"""What the operators of a whole mixture-of-experts block cost, case by case.

Five operators around the shuffle, for serving and for training:

  layer               router logits and a few tokens -> the layer's output: choice, both products of
                      the chosen experts with 4-bit weights, the gated activation and the weighted
                      sum over the experts
  norm                what stands between two blocks: the norm of a block's output, its gate and
                      residual scale, the addition to the residual stream and the norm before the
                      next block; the block's output given per token, or as the expert-major rows
                      that a combine would add up first
  norm_grad           its gradient: of the stream, of the block's output, of gate and norm weights
  swiglu              the gated activation on expert-major rows, with the top-k weights, keeping its
                      input in 8 bits (E4M3, one scale per 128 channels) for the backward pass
  swiglu_grad         its gradient from that checkpoint: of gate and up projection and of the weights

`listed()` names the measured cases and `draw()` gives more of the same ranges.  `run()` computes a
case in its plain form (elementary torch operations in 32 bits), or with `own` set through the
library; `exact()` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

_NONE = float("-inf")
_BF16 = torch.bfloat16
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _layer(name, tokens, hidden, inter, experts, topk, score, *, bias=False, groups=1, keep=1,
           renorm=True, scale=1.0, logits="f32", size=128, zeros=False):
    return dict(name=name, op="layer", tokens=tokens, hidden=hidden, inter=inter, experts=experts,
                topk=topk, score=score, bias=bias, groups=groups, keep=keep, renorm=renorm,
                scale=scale, logits=logits, size=size, zeros=zeros)


def _norm(name, tokens, hidden, *, op="norm", stream="bf16", post=True, pre=True, gate="none",
          weights="f32", scale=1.0, experts=0, topk=0, capacity=0, save=False):
    return dict(name=name, op=op, tokens=tokens, hidden=hidden, stream=stream, post=post, pre=pre,
                gate=gate, weights=weights, scale=scale, experts=experts, topk=topk,
                capacity=capacity, save=save)


def _swiglu(name, op, tokens, experts, topk, inter, capacity, *, weighted=True, keep="e4m3",
            masked=0.0):
    return dict(name=name, op=op, tokens=tokens, experts=experts, topk=topk, inter=inter,
                capacity=capacity, weighted=weighted, keep=keep, masked=masked)


def listed():
    return [
        # one token of one request: a decoding step's layer, bound by reading eight experts
        _layer("layer_token", 1, 7168, 2048, 256, 8, "sigmoid", bias=True, groups=8, keep=4,
               scale=2.5),
        # an odd handful of tokens (several requests, or tokens drafted ahead) on smaller experts
        _layer("layer_handful", 5, 4096, 1024, 64, 6, "softmax", logits="bf16", size=64, zeros=True),
        # a small decoding batch: about a hundred experts with one or two tokens each
        _layer("layer_batch", 16, 7168, 2048, 256, 8, "sigmoid", bias=True, groups=8, keep=4,
               scale=2.5),
        # between two blocks of a decoding step
        _norm("norm_token", 1, 7168, gate="channel", weights="bf16"),
        # the decoding batch of the repository (32 ranks of 128 tokens), out of the experts' rows
        _norm("norm_rows_decode", 4096, 7168, scale=0.5, experts=256, topk=8, capacity=192),
        # a prefill batch (8 ranks of 4096 tokens), every token with its own gate
        _norm("norm_prefill", 32768, 7168, gate="token", scale=0.25),
        # training, ragged: a stream in 32 bits and a gate for every token and channel
        _norm("norm_grad_ragged", 997, 2056, op="norm_grad", stream="f32", gate="full"),
        # training: a prefill batch with norms on both sides and a gate for every channel
        _norm("norm_grad_prefill", 32768, 7168, op="norm_grad", gate="channel", weights="bf16",
              scale=0.5),
        # a ragged batch with a row or two an expert, nothing kept: serving with unquantised weights
        _swiglu("swiglu_serving", "swiglu", 61, 256, 8, 2048, 16, weighted=False, keep="none"),
        # training: few experts with thousands of rows, input kept in 8 bits
        _swiglu("swiglu_prefill", "swiglu", 16384, 8, 2, 4096, 4608),
        # gradients: the repository's small batch, and a prefill batch of 8 ranks of 4096 tokens
        _swiglu("swiglu_grad_small", "swiglu_grad", 512, 16, 4, 256, 512, masked=0.05),
        _swiglu("swiglu_grad_prefill", "swiglu_grad", 32768, 256, 8, 2048, 1216),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer", "norm", "norm", "norm_grad", "swiglu", "swiglu_grad"])
    if op == "layer":
        experts, topk = rng.choice([(8, 2), (16, 4), (60, 4), (64, 6), (128, 8), (256, 8)])
        score = rng.choice(["sigmoid", "softmax"])
        groups = rng.choice([1, 4]) if experts >= 64 and score == "sigmoid" else 1
        size = rng.choice([32, 64, 128])
        case = _layer("", _log(rng, 1, 16), size * _log(rng, 1024 // size, 7168 // size),
                      size * _log(rng, 512 // size, 2048 // size), experts, topk, score,
                      bias=score == "sigmoid" and rng.random() < 0.5, groups=groups,
                      keep=2 if groups > 1 else 1, renorm=rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]), logits=rng.choice(["f32", "bf16"]),
                      size=size, zeros=rng.random() < 0.5)
    elif op in ("norm", "norm_grad"):
        hidden = 8 * _log(rng, 16, 896)
        post, pre = rng.choice([(True, True), (True, False), (False, True), (True, True)])
        rows = op == "norm" and rng.random() < 0.4
        tokens = _log(rng, 1, min(32768, 32768 * 7168 // ((12 if rows else 1) * hidden)))
        case = _norm("", tokens, hidden, op=op, stream=rng.choice(["bf16", "f32"]), post=post,
                     pre=pre, gate=rng.choice(["none", "channel", "token", "full"]),
                     weights=rng.choice(["f32", "bf16"]), scale=rng.choice([1.0, 0.25]))
        if rows:
            experts, topk = rng.choice([(8, 2), (16, 4), (64, 6)])
            mean = tokens * topk / experts
            case.update(experts=experts, topk=topk, save=rng.random() < 0.5,
                        capacity=min(tokens, int(mean + 6 * math.sqrt(mean)) + 8))
    else:
        experts, topk = rng.choice([(8, 2), (16, 4), (64, 6), (256, 8)])
        keep = rng.choice(["e4m3", "e4m3", "none" if op == "swiglu" else "bf16"])
        inter = (8 if keep != "e4m3" else 128) * _log(rng, 2 if keep == "e4m3" else 32, 32)
        tokens = _log(rng, 4, max(8, 200_000_000 // (inter * topk)))
        mean = tokens * topk / experts
        case = _swiglu("", op, tokens, experts, topk, inter,
                       min(tokens, int(mean + 6 * math.sqrt(mean)) + 8),
                       weighted=rng.random() < 0.7, keep=keep, masked=rng.choice([0.0, 0.05]))
    del case["name"]
    return case


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _choose(case, gen, device):
    """Distinct experts for every token, uniform; -1 in masked slots."""
    T, E, K = case["tokens"], case["experts"], case["topk"]
    idx = torch.rand((T, E), generator=gen, device=device).topk(K, dim=1).indices
    if case.get("masked"):
        idx[torch.rand((T, K), generator=gen, device=device) < case["masked"]] = -1
    return idx


def _expert_rows(idx, experts, capacity):
    """The expert-major row of every slot (by token, then slot; -1: none) and the experts' counts."""
    flat = idx.reshape(-1)
    live = torch.where(flat >= 0, flat, experts)
    count = torch.bincount(live, minlength=experts + 1)
    order = torch.argsort(live, stable=True)
    first = torch.cumsum(count, 0) - count
    at = torch.empty_like(flat)
    at[order] = torch.arange(flat.numel(), device=flat.device) - first[live[order]]
    row = torch.where((flat >= 0) & (at < capacity), flat * capacity + at, -1)
    return row.reshape(idx.shape).to(torch.int32), count[:experts].to(torch.int32)


def _normal(shape, gen, device, dtype, scale=1.0):
    """Normal values, in pieces of rows so that no 32-bit copy of a large tensor is made."""
    out = torch.empty(shape, dtype=dtype, device=device)
    step = max(1, (1 << 28) // max(1, shape[1]))
    for at in range(0, shape[0], step):
        part = out[at:at + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=device).mul_(scale))
    return out


def _weights4(experts, rows, inner, size, zeros, gen, device):
    """4-bit codes, scales and zero points of weights of about 1/sqrt(inner)."""
    q = torch.randint(0, 256, (experts, rows, inner // 2), dtype=torch.uint8, device=device,
                      generator=gen)
    spread = torch.rand((experts, rows, inner // size), generator=gen, device=device)
    scales = spread.mul_(0.5).add_(0.75).mul_(1.0 / (4.6 * math.sqrt(inner))).to(_BF16)
    zero = None
    if zeros:
        zero = torch.randint(6, 10, scales.shape, dtype=torch.uint8, device=device, generator=gen)
    return q, scales, zero


def _to_8_bits(v):
    """E4M3 values and one scale per 128 channels, as the FP8 dispatch rounds them."""
    blocks = v.float().unflatten(1, (-1, 128))
    top = blocks.abs().amax(-1).clamp_(min=1e-4)
    codes = (blocks * (448.0 / top)[..., None]).to(torch.float8_e4m3fn)
    return codes.reshape(v.shape), top / 448.0


def _rows_of(case, gen, device):
    """The layout of an expert-major case, its top-k weights and its number of rows."""
    idx = _choose(case, gen, device)
    slot, count = _expert_rows(idx, case["experts"], case["capacity"])
    w = torch.softmax(torch.randn(idx.shape, generator=gen, device=device), dim=1)
    return dict(slot=slot, count=count, topk_weights=w), case["experts"] * case["capacity"]


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "layer":
        T, H, N, E = case["tokens"], case["hidden"], case["inter"], case["experts"]
        s["x"] = _normal((T, H), gen, device, _BF16)
        s["logits"] = _normal((T, E), gen, device, _TYPES[case["logits"]], 1.5)
        s["bias"] = torch.randn(E, generator=gen, device=device).mul_(0.1) if case["bias"] else None
        s["gate_up"] = _weights4(E, 2 * N, H, case["size"], case["zeros"], gen, device)
        s["down"] = _weights4(E, H, N, case["size"], case["zeros"], gen, device)
        return s
    if op in ("norm", "norm_grad"):
        T, H = case["tokens"], case["hidden"]
        kind, stream = _TYPES[case["weights"]], _TYPES[case["stream"]]
        if case["experts"]:
            more, rows = _rows_of(case, gen, device)
            s.update(more)
            s["y"] = _normal((rows, H), gen, device, _BF16, 1.5)
        else:
            s["y"] = _normal((T, H), gen, device, _BF16, 1.5)
        s["x"] = _normal((T, H), gen, device, stream, 2.0)  # the stream; its result, for the gradient
        for name in ("post", "pre"):
            s[name] = None
            if case[name]:
                s[name] = torch.randn(H, generator=gen, device=device).mul_(0.2).add_(1.0).to(kind)
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(
            torch.randn(shape, generator=gen, device=device)).to(kind)
        if op == "norm_grad":
            s["dz"] = _normal((T, H), gen, device, stream)
            s["dh"] = _normal((T, H), gen, device, _BF16) if case["pre"] else None
        return s
    more, rows = _rows_of(case, gen, device)
    s.update(more)
    N = case["inter"]
    gate_up = _normal((rows, 2 * N), gen, device, _BF16)
    if op == "swiglu":
        s["gate_up"] = gate_up
        s["h"] = torch.zeros((rows, N), dtype=_BF16, device=device)
        if case["keep"] == "e4m3":
            s["codes"] = torch.zeros((rows, 2 * N), dtype=torch.uint8, device=device)
            s["scales"] = torch.zeros((rows, 2 * N // 128), device=device)
        return s
    if case["keep"] == "e4m3":  # what the forward pass left
        step = max(1, (1 << 28) // (2 * N))
        parts = [_to_8_bits(gate_up[at:at + step]) for at in range(0, rows, step)]
        s["codes"] = torch.cat([p[0].view(torch.uint8) for p in parts])
        s["scales"] = torch.cat([p[1] for p in parts])
    else:
        s["gate_up"] = gate_up
    s["dh"] = _normal((rows, N), gen, device, _BF16)
    s["dgate_up"] = torch.zeros((rows, 2 * N), dtype=_BF16, device=device)
    return s


# ---------------------------------------------------------------------------------------------
# the operators in their plain form
# ---------------------------------------------------------------------------------------------
def _route_plain(s):
    c = s["case"]
    T, E, K = c["tokens"], c["experts"], c["topk"]
    logit = s["logits"].float()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logit))
        key = score if s["bias"] is None else score + s["bias"]
    else:
        e = torch.exp(logit - logit.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
        key = logit
    if c["groups"] > 1:  # a group's score: the sum of its two largest keys
        best = torch.sort(key.reshape(T, c["groups"], -1), dim=2, descending=True, stable=True).values
        order = torch.sort(best[..., 0] + best[..., 1], dim=1, descending=True, stable=True).indices
        kept = torch.zeros((T, c["groups"]), dtype=torch.bool, device=key.device)
        kept.scatter_(1, order[:, :c["keep"]], True)
        key = torch.where(kept.repeat_interleave(E // c["groups"], 1), key, _NONE)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx, w * c["scale"]


def _dequantised(weights, experts):
    q, scales, zeros = (None if v is None else v[experts] for v in weights)
    w = torch.stack((q & 15, q >> 4), -1).reshape(*scales.shape, -1).float()
    w.sub_(8.0 if zeros is None else zeros.float()[..., None])
    return w.mul_(scales.float()[..., None]).flatten(2)


def _layer_plain(s):
    c = s["case"]
    N = c["inter"]
    idx, w = _route_plain(s)
    used = torch.unique(idx)
    x = s["x"].float()
    p = torch.matmul(x[None], _dequantised(s["gate_up"], used).transpose(1, 2))  # [experts, T, 2 N]
    gate, up = p[..., :N], p[..., N:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    named = idx[None, :, :] == used[:, None, None]  # [experts, T, K]
    h = h * torch.where(named, w[None], 0.0).sum(2)[..., None]
    out = torch.matmul(h, _dequantised(s["down"], used).transpose(1, 2)).sum(0)
    return {"out": out.to(_BF16), "topk_idx": idx, "topk_weights": w}


_EPS = 1e-6


def _block_output(s):
    """The block's output per token in 32 bits: given, or the weighted sum of the experts' rows."""
    if not s["case"]["experts"]:
        return s["y"].float()
    row = s["slot"].long()
    picked = s["y"][row.clamp(min=0)].float()
    return (picked * torch.where(row >= 0, s["topk_weights"], 0.0)[..., None]).sum(1)


def _norm_plain(s):
    c = s["case"]
    y = _block_output(s)
    out = {"y": y.to(_BF16)} if c["save"] else {}
    if c["post"]:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS) * s["post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    z = s["x"].float() + c["scale"] * y
    out["z"] = z.to(s["x"].dtype)
    if c["pre"]:
        z = z / torch.sqrt((z * z).mean(1, keepdim=True) + _EPS) * s["pre"].float()
        out["h"] = z.to(_BF16)
    return out


def _norm_grad_plain(s):
    c = s["case"]
    z, dz, out = s["x"].float(), s["dz"].float(), {}
    if c["pre"]:
        dh = s["dh"].float()
        r = 1.0 / torch.sqrt((z * z).mean(1, keepdim=True) + _EPS)
        out["dpre"] = (dh * z * r).sum(0)
        d = dh * s["pre"].float()
        dz = dz + r * d - z * (r * r * r * (z * d).mean(1, keepdim=True))
    out["dx"] = dz.to(s["x"].dtype)
    y = s["y"].float()
    r = 1.0
    if c["post"]:
        r = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS)
    n = y * r
    if s["gate"] is not None:
        dgate = c["scale"] * dz * (n * s["post"].float() if c["post"] else n)
        kind = c["gate"]
        out["dgate"] = (dgate.sum(0) if kind == "channel" else dgate.sum(1, keepdim=True)
                        if kind == "token" else dgate.to(s["gate"].dtype))
    dn = c["scale"] * dz if s["gate"] is None else c["scale"] * dz * s["gate"].float()
    if c["post"]:
        out["dpost"] = (dn * n).sum(0)
        dn = dn * s["post"].float()
        dn = r * dn - y * (r * r * r * (y * dn).mean(1, keepdim=True))
    out["dy"] = dn.to(_BF16)
    return out


def _swiglu_plain(s):
    c = s["case"]
    row = s["slot"].long()
    live = row >= 0
    used = row[live]
    g, u = s["gate_up"][used].float().chunk(2, dim=1)
    h = g / (1.0 + torch.exp(-g)) * u
    if c["weighted"]:
        h = h * s["topk_weights"][live][:, None]
    out = {"h": torch.zeros_like(s["h"])}
    out["h"][used] = h.to(_BF16)
    if c["keep"] == "e4m3":
        codes, scales = _to_8_bits(s["gate_up"][used])
        out["codes"] = torch.zeros_like(s["codes"])
        out["codes"][used] = codes.view(torch.uint8)
        out["codes"] = out["codes"].view(torch.float8_e4m3fn)
        out["scales"] = torch.zeros_like(s["scales"])
        out["scales"][used] = scales
    return out


def _kept(s, used):
    """Gate and up projection of rows `used`, in 32 bits."""
    if s["case"]["keep"] != "e4m3":
        return s["gate_up"][used].float()
    codes = s["codes"][used].view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128))
    return (codes * s["scales"][used][..., None]).flatten(1)


def _swiglu_grad_plain(s):
    c = s["case"]
    row = s["slot"].long()
    live = row >= 0
    used = row[live]
    g, u = _kept(s, used).chunk(2, dim=1)
    dh = s["dh"][used].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    out = {}
    if c["weighted"]:
        out["dweights"] = torch.zeros_like(s["topk_weights"])
        out["dweights"][live] = (dh * (g * sig * u)).sum(1)
        dh = dh * s["topk_weights"][live][:, None]
    out["dgate_up"] = torch.zeros_like(s["dgate_up"])
    out["dgate_up"][used] = torch.cat((dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig), 1).to(_BF16)
    return out


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"layer": _layer_plain, "norm": _norm_plain, "norm_grad": _norm_grad_plain,
                "swiglu": _swiglu_plain, "swiglu_grad": _swiglu_grad_plain}[op](s)
    import combine_get_dispatch_04_gb300 as ep
    if op == "layer":
        out, idx, w = ep.layer_w4(s["x"], s["logits"], ep.W4Weights(*s["gate_up"]),
                                  ep.W4Weights(*s["down"]), c["topk"], score=c["score"],
                                  bias=s["bias"], num_groups=c["groups"], topk_groups=c["keep"],
                                  renormalize=c["renorm"], scale=c["scale"])
        return {"out": out, "topk_idx": idx, "topk_weights": w}
    if op == "norm":
        kind = dict(gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"], scale=c["scale"],
                    eps=_EPS)
        if c["experts"]:
            layout = ep.LLLayout(s["slot"], s["count"], None, c["experts"], 1, c["capacity"])
            r = ep.ll_combine_norm(s["y"], s["topk_weights"], layout, s["x"], save=c["save"], **kind)
        else:
            r = ep.block_norm(s["x"], s["y"], **kind)
        out = {"z": r.z}
        if c["pre"]:
            out["h"] = r.h
        if c["save"]:
            out["y"] = r.y
        return out
    if op == "norm_grad":
        r = ep.block_norm_backward(s["dz"], s["dh"], s["x"], s["y"], gate=s["gate"],
                                   post_weight=s["post"], pre_weight=s["pre"], scale=c["scale"],
                                   eps=_EPS)
        out = {"dx": r.dx, "dy": r.dy}
        for name, value in (("dgate", r.dgate), ("dpost", r.dpost_weight), ("dpre", r.dpre_weight)):
            if value is not None:
                out[name] = value
        return out
    layout = ep.LLLayout(s["slot"], s["count"], None, c["experts"], 1, c["capacity"])
    w = s["topk_weights"] if c["weighted"] else None
    kept = ep.Checkpoint8(s["codes"], s["scales"]) if c["keep"] == "e4m3" else None
    if op == "swiglu":
        h = ep.ll_swiglu(s["gate_up"], layout, w, checkpoint=kept, out=s["h"])
        if kept is None:
            return {"h": h}
        return {"h": h, "codes": kept.codes.view(torch.float8_e4m3fn), "scales": kept.scales}
    d, dw = ep.ll_swiglu_backward(s["dh"], kept or s["gate_up"], layout, w, out=s["dgate_up"])
    return {"dgate_up": d} if w is None else {"dgate_up": d, "dweights": dw}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    op, T = case["op"], case["tokens"]
    if op == "layer":
        H, N, E, K = case["hidden"], case["inter"], case["experts"], case["topk"]
        size, busy = case["size"], E * (1.0 - (1.0 - K / E) ** T)
        per = 0.5 + (3 if case["zeros"] else 2) / size  # bytes of a weight
        return {"bytes": int(busy * 3 * H * N * per + T * (4 * H + E * 4)),
                "flops": int(6.0 * T * K * H * N)}
    if op in ("norm", "norm_grad"):
        H, stream = case["hidden"], 4 if case["stream"] == "f32" else 2
        kind = 4 if case["weights"] == "f32" else 2
        full = T * H * kind if case["gate"] == "full" else 0
        if op == "norm":
            read = T * (case["topk"] or 1) * 2
            return {"bytes": H * (read + T * (2 * stream + (2 if case["pre"] else 0)
                                              + (2 if case["save"] else 0))) + full,
                    "flops": H * T * (8 + 2 * case["topk"])}
        return {"bytes": H * T * (3 * stream + 4 + (2 if case["pre"] else 0)) + 2 * full,
                "flops": 30 * H * T}
    rows, N = T * case["topk"] * (1.0 - case["masked"]), case["inter"]
    kept = 2 * N * (1 + 4 / 128)
    if op == "swiglu":
        return {"bytes": int(rows * (6 * N + (kept if case["keep"] == "e4m3" else 0))),
                "flops": int(rows * N * 10)}
    return {"bytes": int(rows * (6 * N + (kept if case["keep"] == "e4m3" else 4 * N))),
            "flops": int(rows * N * 20)}


# ---------------------------------------------------------------------------------------------
# the same results from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        return {"layer": _layer_exact, "norm": _norm_exact, "norm_grad": _norm_grad_exact,
                "swiglu": _swiglu_exact, "swiglu_grad": _swiglu_grad_exact}[op](s)


def _matrix64(weights, e, size):
    q, scales, zeros = weights
    codes = torch.empty((q.shape[1], 2 * q.shape[2]), dtype=torch.float64, device=q.device)
    codes[:, 0::2], codes[:, 1::2] = (q[e] % 16).double(), torch.div(q[e], 16, rounding_mode="floor").double()
    shift = 8.0 if zeros is None else zeros[e].double().repeat_interleave(size, 1)
    return (codes - shift) * scales[e].double().repeat_interleave(size, 1)


def _layer_exact(s):
    c = s["case"]
    E, K, N = c["experts"], c["topk"], c["inter"]
    logit = s["logits"].double()
    score = torch.sigmoid(logit) if c["score"] == "sigmoid" else torch.softmax(logit, 1)
    key = logit if c["score"] != "sigmoid" else score
    if s["bias"] is not None:
        key = key + s["bias"].double()
    if c["groups"] > 1:
        parts = key.unflatten(1, (c["groups"], -1))
        best = parts.topk(2, dim=2).values.sum(2).topk(c["keep"], dim=1).indices
        allowed = (torch.arange(c["groups"], device=key.device)[None, :, None] == best[:, None, :]).any(2)
        key = parts.masked_fill(~allowed[..., None], _NONE).flatten(1)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    x = s["x"].double()
    out = torch.zeros_like(x)
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        p = x[t] @ _matrix64(s["gate_up"], e, c["size"]).t()
        h = p[:, :N] * torch.sigmoid(p[:, :N]) * p[:, N:]
        out[t] += w[t, k][:, None] * (h @ _matrix64(s["down"], e, c["size"]).t())
    return {"out": out, "topk_idx": None, "topk_weights": w}


def _rms64(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + _EPS)


def _norm_exact(s):
    c = s["case"]
    if c["experts"]:
        y = torch.zeros(s["x"].shape, dtype=torch.float64, device=s["x"].device)
        for k in range(c["topk"]):
            t = torch.nonzero(s["slot"][:, k] >= 0).reshape(-1)
            y[t] += s["topk_weights"][t, k].double()[:, None] * s["y"][s["slot"][t, k].long()].double()
    else:
        y = s["y"].double()
    out = {"y": y.clone()} if c["save"] else {}
    if c["post"]:
        y = y * _rms64(y) * s["post"].double()
    gate = 1.0 if s["gate"] is None else s["gate"].double()
    z = s["x"].double() + c["scale"] * gate * y
    out["z"] = z
    if c["pre"]:
        out["h"] = z * _rms64(z) * s["pre"].double()
    return out


def _norm_grad_exact(s):
    """By automatic differentiation of the definition, a slice of tokens at a time."""
    c = s["case"]
    T, H = s["x"].shape
    names = [n for n in ("post", "pre", "gate") if s[n] is not None]
    out = {"dx": torch.empty((T, H), dtype=torch.float64, device=s["x"].device),
           "dy": torch.empty((T, H), dtype=torch.float64, device=s["x"].device)}
    step = max(1, (1 << 25) // H)
    with torch.enable_grad():
        for at in range(0, T, step):
            part = slice(at, at + step)
            # the stream's gradient is that of its result, through both of its uses
            z = s["x"][part].double().requires_grad_(True)
            y = s["y"][part].double().requires_grad_(True)
            leaf = {n: (s[n][part] if n == "gate" and c["gate"] != "channel" else s[n])
                    .double().requires_grad_(True) for n in names}
            total = s["dz"][part].double()
            if c["pre"]:
                h = z * _rms64(z) * leaf["pre"]
                dz, dpre = torch.autograd.grad(h, (z, leaf["pre"]), s["dh"][part].double())
                total = total + dz
                out["dpre"] = out.get("dpre", 0.0) + dpre
            out["dx"][part] = total
            v = y * _rms64(y) * leaf["post"] if c["post"] else y * 1.0
            if s["gate"] is not None:
                v = v * leaf["gate"]
            wanted = [n for n in names if n != "pre"]
            got = torch.autograd.grad(c["scale"] * v, [y] + [leaf[n] for n in wanted], total)
            out["dy"][part] = got[0]
            for n, g in zip(wanted, got[1:]):
                if n == "gate" and c["gate"] != "channel":
                    out.setdefault("dgate", []).append(g)
                else:
                    out["d" + n] = out.get("d" + n, 0.0) + g
    if isinstance(out.get("dgate"), list):
        out["dgate"] = torch.cat(out["dgate"])
    return out


def _swiglu_exact(s):
    c = s["case"]
    N = c["inter"]
    out = {"h": torch.zeros(s["h"].shape, dtype=torch.float64, device=s["h"].device)}
    if c["keep"] == "e4m3":
        out["codes"] = torch.zeros(s["codes"].shape, dtype=torch.float64, device=s["h"].device)
        out["scales"] = torch.zeros(s["scales"].shape, dtype=torch.float64, device=s["h"].device)
    for k in range(c["topk"]):
        t = torch.nonzero(s["slot"][:, k] >= 0).reshape(-1)
        r = s["slot"][t, k].long()
        v = s["gate_up"][r].double()
        w = s["topk_weights"][t, k].double()[:, None] if c["weighted"] else 1.0
        out["h"][r] = w * torch.sigmoid(v[:, :N]) * v[:, :N] * v[:, N:]
        if c["keep"] == "e4m3":
            scale = v.unflatten(1, (-1, 128)).abs().amax(2).clamp(min=1e-4) / 448.0
            out["scales"][r] = scale
            out["codes"][r] = v / scale.repeat_interleave(128, 1)
    return out


def _swiglu_grad_exact(s):
    c = s["case"]
    N = c["inter"]
    out = {"dgate_up": torch.zeros(s["dgate_up"].shape, dtype=torch.float64, device=s["dh"].device)}
    dw = torch.zeros(s["slot"].shape, dtype=torch.float64, device=s["dh"].device)
    step = max(1, (1 << 25) // N)
    for k in range(c["topk"]):
        chosen = torch.nonzero(s["slot"][:, k] >= 0).reshape(-1)
        for t in chosen.split(step):
            r = s["slot"][t, k].long()
            if c["keep"] == "e4m3":
                v = s["codes"][r].view(torch.float8_e4m3fn).double()
                v = v * s["scales"][r].double().repeat_interleave(128, 1)
            else:
                v = s["gate_up"][r].double()
            g, u, d = v[:, :N], v[:, N:], s["dh"][r].double()
            silu = g * torch.sigmoid(g)
            dw[t, k] = (d * silu * u).sum(1)
            if c["weighted"]:
                d = d * s["topk_weights"][t, k].double()[:, None]
            slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
            out["dgate_up"][r] = torch.cat((d * u * slope, d * silu), 1)
    if c["weighted"]:
        out["dweights"] = dw
    return out
