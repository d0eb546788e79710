"""What the operators around the token shuffle cost, case by case.

Four operators, each the neighbour of a step that the library has:

  route               router logits [T, E] -> the top-k experts of every token and their weights,
                      which is what the layout and the combine take
  route_grad          the gradient of those weights with respect to the logits
  experts_w4          the experts' products on the rows that the expert-major dispatch delivers,
                      with 4-bit weights and one scale per group of input channels, plain or with
                      the gated activation
  combine_grad        the gradient of the combine: of every expert output row and of every weight

`listed()` names the measured cases and `draw()` gives more of the same ranges.  `run()` computes a
case in its plain form (elementary torch operations in 32 bits), or with `own` set through the
library; `exact()` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

_NONE = float("-inf")


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _route(name, tokens, experts, topk, score, *, bias=False, groups=1, keep=1, renorm=True,
           scale=1.0, dtype="f32", masked=0.0):
    return dict(name=name, op="route", tokens=tokens, experts=experts, topk=topk, score=score,
                bias=bias, groups=groups, keep=keep, renorm=renorm, scale=scale, dtype=dtype,
                masked=masked)


def _experts(name, tokens, experts, topk, inner, outer, *, group=128, act="none", rows="bf16",
             zeros=False, capacity=0, zipf=0.0):
    return dict(name=name, op="experts_w4", tokens=tokens, experts=experts, topk=topk, inner=inner,
                outer=outer, group=group, act=act, rows=rows, zeros=zeros, capacity=capacity,
                zipf=zipf)


def _combine(name, layout, tokens, hidden, experts, topk, ranks, *, capacity=0, masked=0.0,
             zipf=0.0):
    return dict(name=name, op="combine_grad", layout=layout, tokens=tokens, hidden=hidden,
                experts=experts, topk=topk, ranks=ranks, capacity=capacity, masked=masked, zipf=zipf)


def listed():
    return [
        # one token of one request: what the router adds to the latency of a decoding step
        _route("route_token", 1, 256, 8, "sigmoid", bias=True, groups=8, keep=4, scale=2.5),
        # the decoding batch of the repository (32 ranks of 128 tokens), groups and a balance bias
        _route("route_decode", 4096, 256, 8, "sigmoid", bias=True, groups=8, keep=4, scale=2.5),
        # the repository's largest batch (16 ranks of 8192 tokens), some experts switched off
        _route("route_large", 131072, 64, 6, "softmax", dtype="bf16", masked=0.03),
        # training: the router's gradient on a prefill batch of 8 ranks of 4096 tokens
        dict(_route("", 32768, 256, 8, "sigmoid", scale=2.5), op="route_grad",
             name="route_grad_prefill"),
        # training without renormalised weights: every logit of the token has a gradient
        dict(_route("", 131072, 64, 6, "softmax", renorm=False, dtype="bf16"), op="route_grad",
             name="route_grad_dense"),
        # one token against the 8 experts it chose: bound by reading their weights
        _experts("experts_token", 1, 256, 8, 7168, 2048, act="swiglu", capacity=1),
        # a small ragged decoding batch: about one row an expert, some experts with none
        _experts("experts_small_batch", 61, 256, 8, 2048, 7168, group=64, zeros=True, capacity=16),
        # the decoding batch on FP8 rows, as the low-latency dispatch leaves them
        _experts("experts_decode_fp8", 4096, 256, 8, 7168, 2048, act="swiglu", rows="fp8",
                 capacity=192),
        # prompts: few experts with thousands of rows each
        _experts("experts_prefill", 16384, 8, 2, 4096, 4096, capacity=4608),
        # gradients of the combine: a small batch, expert-major decoding rows, and the
        # rank-major rows of the skewed batch
        _combine("combine_grad_tiny", "rank", 512, 256, 16, 4, 4),
        _combine("combine_grad_expert", "expert", 4096, 7168, 256, 8, 32, capacity=192),
        _combine("combine_grad_skewed", "rank", 131072, 4096, 64, 6, 16, masked=0.05, zipf=1.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "experts_w4", "combine_grad"])
    if op in ("route", "route_grad"):
        experts, topk = rng.choice([(8, 2), (16, 4), (60, 4), (64, 6), (128, 8), (160, 6), (256, 8)])
        score = rng.choice(["sigmoid", "softmax"])
        groups = rng.choice([1, 4]) if experts % 8 == 0 and experts >= 64 and score == "sigmoid" else 1
        case = _route("", _log(rng, 1, 131072), experts, topk, score,
                      bias=score == "sigmoid" and rng.random() < 0.5, groups=groups,
                      keep=2 if groups > 1 else 1, renorm=rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]),
                      masked=rng.choice([0.0, 0.03]) if experts >= 64 and op == "route" else 0.0)
        case["op"] = op
    elif op == "experts_w4":
        group = rng.choice([32, 64, 128])
        rows = rng.choice(["bf16", "bf16", "fp8"])
        step = 128 if rows == "fp8" else group
        experts, topk = rng.choice([(8, 2), (16, 4), (64, 6), (128, 8)])
        tokens = _log(rng, 1, 4096)
        mean = tokens * topk / experts
        case = _experts("", tokens, experts, topk, step * _log(rng, max(2, 512 // step), 4096 // step),
                        8 * _log(rng, 32, 448), group=group, act=rng.choice(["none", "swiglu"]),
                        rows=rows, zeros=rng.random() < 0.5,
                        capacity=min(tokens, int(mean + 6 * math.sqrt(mean)) + 8))
    else:
        experts, topk = rng.choice([(8, 2), (16, 4), (64, 6), (256, 8)])
        layout = rng.choice(["rank", "expert"])
        ranks = rng.choice([4, 8])
        hidden = 8 * _log(rng, 32, 896)
        tokens = ranks * _log(rng, 8, max(16, 128_000_000 // (ranks * hidden)))
        mean = tokens * topk / experts
        case = _combine("", layout, tokens, hidden, experts, topk, ranks,
                        capacity=min(tokens, int(mean + 6 * math.sqrt(mean)) + 8),
                        masked=rng.choice([0.0, 0.05]))
    del case["name"]
    return case


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _choose(case, gen, device):
    """Distinct experts for every token, uniform or by popularity; -1 in masked slots."""
    T, E, K = case["tokens"], case["experts"], case["topk"]
    g = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device=device).clamp_(1e-7, 1 - 1e-6)))
    if case["zipf"]:
        g -= case["zipf"] * torch.log(torch.arange(1, E + 1, device=device, dtype=torch.float32))
    idx = g.topk(K, dim=1).indices
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


def _rank_rows(idx, experts, ranks):
    """The rank-major row of every (token, rank) pair (by rank, then token; -1: none)."""
    T = idx.shape[0]
    dest = torch.where(idx >= 0, idx // (experts // ranks), ranks)
    sent = torch.zeros((T, ranks + 1), dtype=torch.bool, device=idx.device)
    sent.scatter_(1, dest, True)
    sent = sent[:, :ranks]
    place = torch.cumsum(sent.t().reshape(-1).to(torch.int64), 0).reshape(ranks, T).t() - 1
    return torch.where(sent, place, -1).to(torch.int32).contiguous()


def _normal(shape, gen, device, dtype, scale=1.0):
    """Normal values, in pieces of rows so that no 32-bit copy of a large tensor is made."""
    out = torch.empty(shape, dtype=dtype, device=device)
    step = max(1, (1 << 28) // max(1, shape[1]))
    for at in range(0, shape[0], step):
        part = out[at:at + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=device).mul_(scale))
    return out


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, K = case["tokens"], case["experts"], case["topk"]
        logits = torch.randn((T, E), generator=gen, device=device).mul_(1.5)
        if case["masked"]:  # experts that are switched off for a token
            logits[torch.rand((T, E), generator=gen, device=device) < case["masked"]] = _NONE
        if case["dtype"] == "bf16":
            logits = logits.to(torch.bfloat16)
        s = dict(case=case, logits=logits, bias=None)
        if case["bias"]:
            s["bias"] = torch.randn(E, generator=gen, device=device).mul_(0.1)
        if op == "route_grad":
            s["topk_idx"] = torch.topk(logits.float(), K, dim=1).indices.contiguous()
            s["dweights"] = torch.randn((T, K), generator=gen, device=device)
        return s
    if op == "experts_w4":
        E, cap, K, N = case["experts"], case["capacity"], case["inner"], case["outer"]
        G = case["group"]
        _, count = _expert_rows(_choose(case, gen, device), E, cap)
        out_rows = 2 * N if case["act"] == "swiglu" else N
        rows = _normal((E * cap, K), gen, device, torch.bfloat16)
        scales = None
        if case["rows"] == "fp8":  # E4M3 codes and one scale per 128 channels
            blocks = rows.float().reshape(E * cap, K // 128, 128)
            scales = blocks.abs().amax(-1).clamp_(min=1e-4).div_(448.0)
            rows = (blocks / scales[..., None]).to(torch.float8_e4m3fn).reshape(E * cap, K)
            rows = rows.view(torch.uint8)
            del blocks
        s = dict(case=case, rows=rows, row_scales=scales, count=count)
        s["q"] = torch.randint(0, 256, (E, out_rows, K // 2), dtype=torch.uint8, device=device,
                               generator=gen)
        # weights of about 1/sqrt(K): 4-bit values have a deviation of 4.6 around their zero
        spread = torch.rand((E, out_rows, K // G), generator=gen, device=device).mul_(0.5).add_(0.75)
        s["scales"] = spread.mul_(1.0 / (4.6 * math.sqrt(K))).to(torch.bfloat16)
        s["zeros"] = None
        if case["zeros"]:
            s["zeros"] = torch.randint(6, 10, (E, out_rows, K // G), dtype=torch.uint8, device=device,
                                       generator=gen)
        s["out"] = torch.zeros((E * cap, N), dtype=torch.bfloat16, device=device)
        return s
    T, H, E, K, R = (case[n] for n in ("tokens", "hidden", "experts", "topk", "ranks"))
    idx = _choose(case, gen, device)
    w = torch.softmax(torch.randn((T, K), generator=gen, device=device), dim=1)
    s = dict(case=case, topk_idx=idx, topk_weights=w, dout=_normal((T, H), gen, device, torch.bfloat16))
    if case["layout"] == "expert":
        s["slot"], s["count"] = _expert_rows(idx, E, case["capacity"])
        rows = E * case["capacity"]
    else:
        s["slot"] = _rank_rows(idx, E, R)
        rows = T * min(K, R)  # the receive buffer of a dispatch that asks for no exact size
    s["y"] = _normal((rows, H), gen, device, torch.bfloat16)
    s["dy"] = torch.zeros((rows, H), dtype=torch.bfloat16, device=device)
    return s


# ---------------------------------------------------------------------------------------------
# the operators in their plain form
# ---------------------------------------------------------------------------------------------
def _route_plain(s):
    c = s["case"]
    T, E, K = c["tokens"], c["experts"], c["topk"]
    logit = s["logits"].float()
    on = logit > _NONE
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logit))
        key = score if s["bias"] is None else score + s["bias"]
    else:
        top = logit.amax(1, keepdim=True)
        e = torch.where(on, torch.exp(logit - torch.where(top > _NONE, top, 0.0)), 0.0)
        score = e / e.sum(1, keepdim=True).clamp(min=1e-38)
        key = logit
    key = torch.where(on, key, _NONE)
    if c["groups"] > 1:  # a group's score: the sum of its two largest keys
        best = torch.sort(key.reshape(T, c["groups"], -1), dim=2, descending=True, stable=True).values
        second = torch.where(best[..., 1] > _NONE, best[..., 1], 0.0)
        order = torch.sort(best[..., 0] + second, dim=1, descending=True, stable=True).indices
        kept = torch.zeros((T, c["groups"]), dtype=torch.bool, device=key.device)
        kept.scatter_(1, order[:, :c["keep"]], True)
        key = torch.where(kept.repeat_interleave(E // c["groups"], 1), key, _NONE)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K]
    w = torch.where(val > _NONE, score.gather(1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"topk_idx": torch.where(val > _NONE, idx, -1), "topk_weights": w * c["scale"]}


def _route_grad_plain(s):
    c = s["case"]
    logit, idx, dw = s["logits"].float(), s["topk_idx"], s["dweights"] * c["scale"]
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logit))
    else:
        e = torch.exp(logit - logit.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    u = score.gather(1, idx)
    if c["renorm"]:
        total = u.sum(1, keepdim=True)
        du = (dw - (dw * u / total).sum(1, keepdim=True)) / total
    else:
        du = dw
    dscore = torch.zeros_like(score).scatter_add_(1, idx, du)
    if c["score"] == "sigmoid":
        grad = dscore * score * (1.0 - score)
    else:
        grad = score * (dscore - (score * dscore).sum(1, keepdim=True))
    return {"dlogits": grad.to(s["logits"].dtype)}


def _experts_plain(s):
    c = s["case"]
    E, cap, K, N, G = c["experts"], c["capacity"], c["inner"], c["outer"], c["group"]
    most = max(1, min(cap, int(s["count"].max())))
    busy = torch.nonzero(s["count"] > 0).reshape(-1)
    x = s["rows"].reshape(E, cap, K)[busy, :most]
    if c["rows"] == "fp8":
        x = x.view(torch.float8_e4m3fn).float().reshape(-1, most, K // 128, 128)
        x = x * s["row_scales"].reshape(E, cap, K // 128)[busy, :most][..., None]
    x = x.float().reshape(-1, most, K)
    q = s["q"][busy]
    w = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], q.shape[1], K // G, G).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"][busy].float()[..., None]
    w = w.sub_(zero).mul_(s["scales"][busy].float()[..., None]).reshape(q.shape[0], q.shape[1], K)
    y = torch.matmul(x, w.transpose(1, 2))
    if c["act"] == "swiglu":
        gate, up = y[..., :N], y[..., N:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    live = torch.arange(most, device=x.device)[None, :, None] < s["count"][busy][:, None, None]
    out = torch.zeros((E, cap, N), dtype=torch.bfloat16, device=x.device)
    out[busy, :most] = torch.where(live, y, 0.0).to(torch.bfloat16)
    return {"y": out.reshape(E * cap, N)}


def _slots_of(s):
    """The row of every top-k slot, [T, K], -1: none."""
    c, slot, idx = s["case"], s["slot"].long(), s["topk_idx"]
    if c["layout"] == "expert":
        return slot
    dest = (idx // (c["experts"] // c["ranks"])).clamp(min=0)
    return torch.where(idx >= 0, slot.gather(1, dest), -1)


def _combine_grad_plain(s):
    c = s["case"]
    T, H = s["dout"].shape
    row = _slots_of(s)
    live = row >= 0
    dout = s["dout"].float()
    picked = s["y"][row.clamp(min=0).reshape(-1)].reshape(T, -1, H).float()
    dw = torch.where(live, (picked * dout[:, None, :]).sum(-1), 0.0)
    del picked
    # the weight of every row: the sum over the slots that name it
    weight = torch.zeros(s["y"].shape[0], device=dout.device)
    weight.index_add_(0, row[live], s["topk_weights"][live])
    owner = torch.full((s["y"].shape[0],), -1, dtype=torch.int64, device=dout.device)
    owner[row[live]] = torch.nonzero(live)[:, 0]
    used = torch.nonzero(owner >= 0).reshape(-1)
    dy = torch.zeros_like(s["y"])
    dy[used] = (weight[used, None] * dout[owner[used]]).to(torch.bfloat16)
    return {"dy": dy, "dweights": dw}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"route": _route_plain, "route_grad": _route_grad_plain, "experts_w4": _experts_plain,
                "combine_grad": _combine_grad_plain}[op](s)
    import combine_get_dispatch_04_gb300 as ep
    if op == "route":
        idx, w = ep.route(s["logits"], c["topk"], score=c["score"], bias=s["bias"],
                          num_groups=c["groups"], topk_groups=c["keep"], renormalize=c["renorm"],
                          scale=c["scale"])
        return {"topk_idx": idx, "topk_weights": w}
    if op == "route_grad":
        return {"dlogits": ep.route_backward(s["dweights"], s["logits"], s["topk_idx"],
                                             score=c["score"], renormalize=c["renorm"],
                                             scale=c["scale"])}
    E, cap = c["experts"], c.get("capacity", 0)
    if op == "experts_w4":
        layout = ep.LLLayout(None, s["count"], None, E, 1, cap)
        return {"y": ep.ll_experts_w4(s["rows"], ep.W4Weights(s["q"], s["scales"], s["zeros"]), layout,
                                      x_scales=s["row_scales"], act=c["act"], out=s["out"])}
    if c["layout"] == "expert":
        layout = ep.LLLayout(s["slot"], s["count"], None, E, c["ranks"], cap)
        dy, dw = ep.ll_combine_backward(s["dout"], s["y"], s["topk_weights"], layout, out=s["dy"])
    else:
        layout = ep.Layout(None, None, None, s["slot"], None, E, c["ranks"])
        dy, dw = ep.combine_backward(s["dout"], s["y"], s["topk_idx"], s["topk_weights"], layout,
                                     out=s["dy"])
    return {"dy": dy, "dweights": dw}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    T, E, K = case["tokens"], case["experts"], case["topk"]
    if op in ("route", "route_grad"):
        size = 4 if case["dtype"] == "f32" else 2
        if op == "route":
            return {"bytes": T * E * size + T * K * 12, "flops": T * E * 4}
        # with renormalised or sigmoid weights only the chosen logits matter
        read = K if case["renorm"] or case["score"] == "sigmoid" else E
        return {"bytes": T * (E + read) * size + T * K * 12, "flops": T * E * 4}
    if op == "experts_w4":
        I, N, G = case["inner"], case["outer"], case["group"]
        out_rows = 2 * N if case["act"] == "swiglu" else N
        rows = T * K
        busy = E * (1.0 - (1.0 - K / E) ** T)
        weights = busy * out_rows * (I // 2 + I // G * (3 if case["zeros"] else 2))
        row = I + I // 128 * 4 if case["rows"] == "fp8" else 2 * I
        return {"bytes": int(weights + rows * (row + 2 * N)), "flops": int(2.0 * rows * I * out_rows)}
    H = case["hidden"]
    if case["layout"] == "expert":
        rows = T * K * (1 - case["masked"])
    elif case["zipf"]:
        rows = 3.924 * T  # distinct ranks of a token, counted on the skewed batch
    else:
        local = E // case["ranks"]
        rows = case["ranks"] * T * (1.0 - math.comb(E - local, K) / math.comb(E, K))
    return {"bytes": int(2 * H * (T + 2 * rows) + T * K * 16), "flops": int(4.0 * H * rows)}


# ---------------------------------------------------------------------------------------------
# the same results from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("route", "route_grad"):
            return _route_exact(s) if op == "route" else _route_grad_exact(s)
        return _experts_exact(s) if op == "experts_w4" else _combine_grad_exact(s)


def _score64(logit, kind):
    return torch.sigmoid(logit) if kind == "sigmoid" else torch.softmax(logit, 1)


def _route_exact(s):
    c = s["case"]
    E, K = c["experts"], c["topk"]
    logit = s["logits"].double()
    score = _score64(logit, c["score"])
    key = score if s["bias"] is None else score + s["bias"].double()
    key = key.masked_fill(torch.isinf(logit), _NONE)
    size = E // c["groups"]
    if c["groups"] > 1:
        parts = key.unflatten(1, (c["groups"], size))
        rank = parts.topk(2, dim=2).values.sum(2).topk(c["keep"], dim=1).indices
        allowed = (torch.arange(E, device=key.device) // size)[None, :, None] == rank[:, None, :]
        key = key.masked_fill(~allowed.any(2), _NONE)
    idx = key.topk(K, dim=1).indices
    # experts of equal keys count in the order of their indices: the weights are equal too
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"topk_idx": None, "topk_weights": w * c["scale"]}


def _route_grad_exact(s):
    c = s["case"]
    logit = s["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        w = _score64(logit, c["score"]).gather(1, s["topk_idx"])
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (w * c["scale"] * s["dweights"].double()).sum().backward()
    return {"dlogits": logit.grad}


def _experts_exact(s):
    c = s["case"]
    E, cap, K, N, G = c["experts"], c["capacity"], c["inner"], c["outer"], c["group"]
    if 2.0 * c["tokens"] * c["topk"] * K * s["q"].shape[1] > 4e12:
        return None
    y = torch.zeros((E * cap, N), dtype=torch.float64, device=s["rows"].device)
    for e, n in enumerate(s["count"].tolist()):
        n = min(n, cap)
        if n == 0:
            continue
        x = s["rows"][e * cap:e * cap + n]
        if c["rows"] == "fp8":
            x = x.view(torch.float8_e4m3fn).to(torch.float64)
            x = x * s["row_scales"][e * cap:e * cap + n].double().repeat_interleave(128, 1)
        q = s["q"][e].to(torch.int16)
        w = torch.empty((q.shape[0], K), dtype=torch.float64, device=q.device)
        w[:, 0::2], w[:, 1::2] = (q % 16).double(), torch.div(q, 16, rounding_mode="floor").double()
        if s["zeros"] is None:
            w -= 8.0
        else:
            w -= s["zeros"][e].double().repeat_interleave(G, 1)
        w *= s["scales"][e].double().repeat_interleave(G, 1)
        p = x.double() @ w.t()
        if c["act"] == "swiglu":
            p = p[:, :N] * torch.sigmoid(p[:, :N]) * p[:, N:]
        y[e * cap:e * cap + n] = p
    return {"y": y}


def _combine_grad_exact(s):
    T, H = s["dout"].shape
    row, w = _slots_of(s), s["topk_weights"].double()
    dw = torch.zeros(row.shape, dtype=torch.float64, device=row.device)
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=row.device)
    step = max(1, (1 << 27) // H)
    for at in range(0, T, step):
        d = s["dout"][at:at + step].double()
        for k in range(row.shape[1]):
            t = torch.nonzero(row[at:at + step, k] >= 0).reshape(-1)
            r = row[at + t, k]
            dw[at + t, k] = (s["y"][r].double() * d[t]).sum(1)
            dy[r] += w[at + t, k][:, None] * d[t]
    return {"dy": dy, "dweights": dw}
