"""The router, its balance loss and the experts' products: plain forms, cases and the calls of the framework's operators.

Each case names its operator in "op":
  "route"    scores -> group-limited top-k -> indices and weights (forward)
  "train"    the same with counts and balance loss, then the gradient of both in the logits
  "balance"  counts and balance loss of given indices, and the gradient in the logits
  "linear"   y = act(x W^T + b) + residual, one dense product or one per expert segment of a row pool
  "linear_backward"   dx, dW, db of the same
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LOWEST = {torch.float32: -3.4028234663852886e38, torch.bfloat16: -3.3895313892515355e38}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of the DeepSeek-V3 example: 8 ranks x 128 tokens, 256 experts in 8 groups
        route("route decode", 128, 256, 8, score="sigmoid", bias=True, groups=8, topk_groups=4),
        # one prefill step of the same
        route("route prefill", 4096, 256, 8, score="sigmoid", bias=True, groups=8, topk_groups=4),
        # a training step's router, mid-size: ragged ranks, bf16 logits, masked experts and empty rows
        route("router train mid", 2048, 128, 8, op="train", dtype="bf16", ragged=True, masked=True),
        # the loss over sequences for routing decided elsewhere, skewed experts
        route("balance sequences", 4096, 256, 8, op="balance", score="sigmoid", seq_len=1024),
        # the smallest batch: 8 ranks x 16 tokens, 32 experts, top-4
        route("balance tiny", 16, 32, 4, op="balance"),
        # the router's own projection at decode size, f32 logits
        linear("gate decode", 1, 1024, 7168, 256, out="f32"),
        # one token through a dense layer: weights are all there is to read
        linear("single token", 1, 1, 4096, 4096, act="gelu", bias=True, residual=True),
        # an odd dense layer
        linear("dense odd", 1, 1003, 1000, 777, act="gelu", bias=True, residual=True),
        # gated experts' first product at decode size: 8 ranks x 128 tokens x top-8 over 256 experts
        linear("experts decode", 256, 8192, 7168, 512, act="swiglu"),
        # gated experts' first product at prefill size, pre-activation kept for training, 5 % of slots dropped
        linear("experts prefill", 128, 124518, 4096, 2048, act="swiglu", bias=True, preact=True),
        # its backward pass
        linear("experts backward", 128, 124518, 4096, 2048, op="linear_backward", act="swiglu", bias=True),
        # the smallest experts' backward pass, SiLU
        linear("experts backward tiny", 32, 512, 256, 512, op="linear_backward", act="silu", bias=True),
    ]


def route(name, tokens, experts, topk, op="route", score="softmax", dtype="f32", bias=False, groups=1, topk_groups=1, normalize=True, scale=2.5,
          seq_len=0, ragged=False, masked=False, world=8):
    c = {"op": op, "world": world, "tokens": tokens, "experts": experts, "topk": topk, "score": score, "dtype": dtype, "bias": bias, "groups": groups,
         "topk_groups": topk_groups, "normalize": normalize, "scale": scale, "seq_len": seq_len, "ragged": ragged, "masked": masked}
    return {"name": name, **c} if name else c


def linear(name, groups, rows, k, n, op="linear", act="none", bias=False, residual=False, preact=False, out="bf16", skew=0.0):
    c = {"op": op, "groups": groups, "rows": rows, "k": k, "n": n, "act": act, "bias": bias, "residual": residual, "preact": preact, "out": out, "skew": skew}
    return {"name": name, **c} if name else c


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["route", "train", "balance", "linear", "linear", "linear_backward"])
    if op in ("route", "train", "balance"):
        groups, topk = rng.choice([1, 1, 4, 8]), rng.randint(1, 12)
        experts = groups * max(log(16, 384) // groups, topk if groups == 1 else 4)
        topk_groups = max(1, groups // 2)
        topk = min(topk, topk_groups * (experts // groups))
        score = rng.choice(["softmax", "sigmoid"])
        return route(None, log(16, 4096), experts, topk, op=op, score=score, dtype=rng.choice(["f32", "bf16"]), bias=score == "sigmoid" and op != "balance" and rng.random() < 0.5,
                     groups=groups, topk_groups=topk_groups, normalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), seq_len=rng.choice([0, 0, log(16, 2048)]),
                     ragged=rng.random() < 0.5, masked=rng.random() < 0.3, world=rng.choice([1, 4, 8]))
    groups = rng.choice([1, 1, 8, 32, 128])
    rows, k = log(1, 4096) if groups == 1 else groups * log(1, 512), 8 * log(16, 768)
    n = min(log(100, 4096), (1 << 30) // (groups * k))
    act = rng.choice(["none", "relu", "gelu", "silu", "swiglu"])
    if op == "linear_backward":
        return linear(None, groups, rows, k, n, op=op, act=act, bias=rng.random() < 0.5, skew=rng.choice([0.0, 1.0]))
    return linear(None, groups, rows, k, n, act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5, preact=act != "none" and rng.random() < 0.5, skew=rng.choice([0.0, 1.0]))


def work(case):
    c = case
    if c["op"] in ("route", "train", "balance"):
        n, e, k, size = sum(tokens_of(c)), c["experts"], c["topk"], 4 if c["dtype"] == "f32" else 2
        padded = c["world"] * c["tokens"]
        slots, segs = 8 * k, 4 * e * segments(c)
        if c["op"] == "route":
            return {"bytes": n * e * size + padded * slots, "flops": 4 * n * e}
        back = n * e * size + padded * e * size + segs  # logits once more, gradient of every row
        if c["op"] == "train":
            return {"bytes": n * e * size + padded * slots + segs + back + n * slots, "flops": 16 * n * e}
        return {"bytes": n * e * size + 4 * n * k + segs + back, "flops": 14 * n * e}
    g, m, k, n = c["groups"], c["rows"], c["k"], c["n"]
    nw, out = n * (2 if c["act"] == "swiglu" else 1), 4 if c["out"] == "f32" else 2
    if g > 1:
        g = min(g, m)  # experts that can hold a row
    if c["op"] == "linear":
        moved = 2 * m * k + 2 * g * nw * k + out * m * n * (2 if c["residual"] else 1) + (2 * m * nw if c["preact"] else 0) + (4 * g * nw if c["bias"] else 0)
        return {"bytes": moved, "flops": 2 * m * nw * k}
    moved = 2 * (2 * m * k) + 2 * g * nw * k + 2 * c["groups"] * nw * k + 2 * m * n + (2 * m * nw if c["act"] != "none" else 0) + (4 * c["groups"] * nw if c["bias"] else 0)
    return {"bytes": moved, "flops": 4 * m * nw * k}


# ------------------------------------------------------------------------------------------ inputs

def tokens_of(c):
    """Tokens that each source rank holds, at most c["tokens"]; a ragged batch has a full rank and an empty one."""
    t, r = c["tokens"], c["world"]
    if not c["ragged"] or r == 1:
        return [t] * r
    return [t] + [t - (t * (37 * i % 61)) // 97 for i in range(1, r - 1)] + [0]


def segments(c):
    return c["world"] * -(-c["tokens"] // c["seq_len"]) if c["seq_len"] else 1


def gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 64 + stream)
    return g


def normal(g, *shape, dtype=torch.float32, std=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    return x.normal_(0.0, std, generator=g)


def counts_of(c, seed):
    """Rows of each expert: a multinomial draw, of equal or (skew) of Zipf popularity."""
    p = np.arange(1, c["groups"] + 1, dtype=np.float64) ** -c["skew"]
    return np.random.RandomState(seed % (1 << 32)).multinomial(c["rows"], p / p.sum())


def prepare_router(c, seed):
    r, t, e, k = c["world"], c["tokens"], c["experts"], c["topk"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = {"case": c, "ntok": tokens_of(c)}
    # logits of unit spread around each expert's popularity
    x = normal(gen(seed, 1), r, t, e) + 0.5 * normal(gen(seed, 2), e)
    if c["masked"]:  # some experts are closed to some tokens, by -inf or by the type's lowest value, and some rows have none left
        u = torch.rand((r, t, e), generator=gen(seed, 3), device=DEV)
        x = torch.where(u < 0.05, -math.inf, torch.where(u < 0.1, LOWEST[dt], x))
        x = torch.where(torch.rand((r, t, 1), generator=gen(seed, 4), device=DEV) < 0.01, -math.inf, x)
    s["logits"] = x.to(dt)
    s["bias"] = normal(gen(seed, 5), e, std=0.05) if c["bias"] else None
    s["valid"] = torch.arange(t, device=DEV)[None, :] < torch.tensor(s["ntok"], device=DEV)[:, None]
    if c["op"] == "balance":  # skewed routing, decided elsewhere: 2 % of the slots are dropped
        keys = normal(gen(seed, 6), r, t, e) - 1.2 * torch.log(torch.arange(1, e + 1, device=DEV, dtype=torch.float32))
        idx = keys.topk(k, -1).indices.to(torch.int32)
        drop = torch.rand((r, t, k), generator=gen(seed, 7), device=DEV) < 0.02
        s["indices"] = torch.where(drop, -1, idx).contiguous()
    if c["op"] == "train":
        s["d_weights"] = normal(gen(seed, 8), r, t, k)
    if c["op"] != "route":
        s["d_loss"] = torch.rand((), generator=gen(seed, 9), device=DEV) + 0.5
    if own:
        from combine_route_layout_gb300 import EpRouterConfig, EpRouterOp
        s["router"] = EpRouterOp(EpRouterConfig(
            world_size=r, max_num_inp_token_per_rank=t, num_experts=e, num_experts_per_token=k, logits_dtype=dt, score_func=c["score"],
            num_groups=c["groups"], topk_groups=c["topk_groups"], normalize_weights=c["normalize"], route_scale=c["scale"], seq_len=c["seq_len"],
            balance_coef=0.01))
    return s


def prepare_linear(c, seed):
    g, m, k, n = c["groups"], c["rows"], c["k"], c["n"]
    nw, bf = n * (2 if c["act"] == "swiglu" else 1), torch.bfloat16
    s = {"case": c}
    if g == 1:
        counts, begins, pool = [m], [0], m
    else:  # each expert's segment is padded to whole 128-row blocks
        counts = [int(v) for v in counts_of(c, seed)]
        padded = [-(-v // 128) * 128 for v in counts]
        begins = [sum(padded[:i]) for i in range(g)]
        pool = m + 127 * g
        s["begin"] = torch.tensor(begins, dtype=torch.int32, device=DEV)
        s["count"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
    s["segments"] = [(i, b, b + v) for i, (b, v) in enumerate(zip(begins, counts)) if v]
    s["x"] = normal(gen(seed, 1), pool, k, dtype=bf)
    s["w"] = normal(gen(seed, 2), g, nw, k, dtype=bf, std=k ** -0.5)
    s["b"] = normal(gen(seed, 3), g, nw, std=0.1) if c["bias"] else None
    out = torch.float32 if c["out"] == "f32" else bf
    if c["op"] == "linear":
        s["r"] = normal(gen(seed, 4), pool, n, dtype=out) if c["residual"] else None
        # rows of no expert are never written
        s["y"] = torch.zeros((pool, n), dtype=out, device=DEV)
        s["z"] = torch.zeros((pool, nw), dtype=bf, device=DEV) if c["preact"] else None
    else:
        s["dy"] = normal(gen(seed, 5), pool, n, dtype=bf)
        s["z"] = normal(gen(seed, 6), pool, nw, dtype=bf) if c["act"] != "none" else None
        s["dx"] = torch.zeros((pool, k), dtype=bf, device=DEV)
    if own:
        from combine_route_layout_gb300 import EpLinearConfig, EpLinearOp
        s["linear"] = EpLinearOp(EpLinearConfig(num_groups=g, in_features=k, out_features=n, max_rows=pool, out_dtype=out, activation=c["act"]),
                                 backward=c["op"] != "linear")
    return s


def prepare(case, seed):
    return (prepare_linear if case["op"].startswith("linear") else prepare_router)(case, seed)


# ------------------------------------------------------------------------------------------ plain forms

def scores_of(s):
    """(masked, scores that select, group scores' function, probabilities) of the logits in 32 bits."""
    c, l = s["case"], s["logits"].float()
    open_ = (l > LOWEST[s["logits"].dtype]) & s["valid"][..., None]
    if c["score"] == "softmax":
        m = torch.where(open_, l, -math.inf).amax(-1, keepdim=True)
        p = torch.where(open_, torch.exp(l - m), 0.0)
        select = l
    else:
        p = torch.where(open_, 1.0 / (1.0 + torch.exp(-l)), 0.0)
        select = p if s["bias"] is None else p + s["bias"]
    return open_, torch.where(open_, select, -math.inf), p


def pick(s, select):
    """The k best experts of the best groups, ties to the lowest index; -1 where none is left."""
    c = s["case"]
    if c["groups"] > 1:
        r, t, e = select.shape
        by = select.view(r, t, c["groups"], e // c["groups"]).sort(dim=-1, descending=True, stable=True).values
        best = by[..., 0]
        if c["score"] == "sigmoid" and by.shape[-1] > 1:
            best = best + torch.where(by[..., 1] > -math.inf, by[..., 1], 0.0)
        order = best.sort(dim=-1, descending=True, stable=True).indices[..., :c["topk_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(-1, order, True)
        select = torch.where(kept.repeat_interleave(e // c["groups"], dim=-1), select, -math.inf)
    top = select.sort(dim=-1, descending=True, stable=True)
    at, value = top.indices[..., :c["topk"]], top.values[..., :c["topk"]]
    return torch.where(value > -math.inf, at, -1)


def over(a, b):
    """a / b, and zero where b is."""
    return torch.where(b > 0, a / torch.where(b > 0, b, 1.0), 0.0)


def weights_of(s, at, p):
    c = s["case"]
    there = at >= 0
    q = torch.where(there, p.gather(-1, at.clamp(min=0)), 0.0)
    if c["normalize"]:
        if c["score"] == "softmax":  # of the selected alone: their own largest logit keeps the sum from vanishing
            l = torch.where(there, s["logits"].float().gather(-1, at.clamp(min=0)), -math.inf)
            q = torch.where(there, torch.exp(l - l.amax(-1, keepdim=True)), 0.0)
        q = over(q, q.sum(-1, keepdim=True))
    elif c["score"] == "softmax":
        q = over(q, p.sum(-1, keepdim=True))
    return q


def plain_loss(s, at, p):
    """Per-segment counts, the loss, and the gradient of the loss in the probabilities."""
    c = s["case"]
    r, t, e, k = c["world"], c["tokens"], c["experts"], c["topk"]
    length = c["seq_len"] or r * t
    per = -(-t // c["seq_len"]) if c["seq_len"] else 1
    token = torch.arange(t, device=DEV)
    seg = (torch.arange(r, device=DEV)[:, None] * per + token // length if c["seq_len"] else torch.zeros((r, 1), dtype=torch.int64, device=DEV)).expand(r, t)
    there = (at >= 0) & s["valid"][..., None]
    cell = torch.where(there, seg[..., None] * e + at, r * per * e if c["seq_len"] else e)
    n_seg = segments(c)
    counts = torch.zeros(n_seg * e + 1, dtype=torch.int64, device=DEV).index_add_(0, cell.reshape(-1), torch.ones_like(cell.reshape(-1)))[:-1].view(n_seg, e)
    held = torch.zeros(n_seg, device=DEV).index_add_(0, seg.reshape(-1), s["valid"].reshape(-1).float())
    prob = over(p, p.sum(-1, keepdim=True))
    mean = over(torch.zeros(n_seg, e, device=DEV).index_add_(0, seg.reshape(-1), prob.reshape(-1, e)), held[:, None])
    share = over(counts.float() * e, held[:, None] * k)
    full = (held > 0).sum().clamp(min=1)
    loss = 0.01 * (share * mean).sum() / full
    grad = (0.01 / full) * over(share, held[:, None])
    return counts.to(torch.int32), loss, grad[seg], prob


def plain_grad_weights(s, at, p, q):
    """Gradient of the weights in the logits."""
    c, d = s["case"], s["d_weights"] * s["case"]["scale"]
    there = at >= 0
    d = torch.where(there, d, 0.0)
    if c["score"] == "softmax":
        each = q * (d - (q * d).sum(-1, keepdim=True)) if c["normalize"] else q * d
    else:
        s_k = torch.where(there, p.gather(-1, at.clamp(min=0)), 0.0)
        each = (over(d - (q * d).sum(-1, keepdim=True), s_k.sum(-1, keepdim=True)) if c["normalize"] else d) * s_k * (1.0 - s_k)
    g = torch.zeros_like(p).scatter_add_(-1, at.clamp(min=0), torch.where(there, each, 0.0))
    if c["score"] == "softmax" and not c["normalize"]:
        g = g - over(p, p.sum(-1, keepdim=True)) * (q * d).sum(-1, keepdim=True)
    return g


def plain_router(s):
    c = s["case"]
    open_, select, p = scores_of(s)
    at = pick(s, select) if c["op"] != "balance" else s["indices"].long()
    q = weights_of(s, at, p) if c["op"] != "balance" else None
    if c["op"] == "route":
        return {"weights": q * c["scale"], "indices": at.to(torch.int32)}
    counts, loss, g, prob = plain_loss(s, at, p)
    g = g * s["d_loss"]
    inner = g - (g * prob).sum(-1, keepdim=True)
    d = prob * inner * (1.0 if c["score"] == "softmax" else 1.0 - p)
    out = {"counts": counts, "loss": loss}
    if c["op"] == "train":
        d = d + plain_grad_weights(s, at, p, q)
        out |= {"weights": q * c["scale"], "indices": at.to(torch.int32)}
    return out | {"d_logits": torch.where(open_, d, 0.0).to(s["logits"].dtype)}


def plain_act(act, z):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return g / (1.0 + torch.exp(-g)) * u
    return z


def plain_slope(act, z):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-z))
        return e * (1.0 + z * (1.0 - e))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    return torch.ones_like(z)


def plain_dz(act, z, dy):
    if act == "none":
        return dy
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return torch.cat((dy * u * plain_slope("silu", g), dy * plain_act("silu", g)), -1)
    return dy * plain_slope(act, z)


def plain_linear(s):
    c = s["case"]
    for e, a, b in s["segments"]:
        z = s["x"][a:b].float() @ s["w"][e].float().t()
        if c["bias"]:
            z = z + s["b"][e]
        y = plain_act(c["act"], z)
        s["y"][a:b] = y + s["r"][a:b].float() if c["residual"] else y
        if c["preact"]:
            s["z"][a:b] = z
    return {"y": s["y"]} | ({"z": s["z"]} if c["preact"] else {})


def plain_linear_backward(s):
    c = s["case"]
    dw = torch.zeros_like(s["w"])
    db = torch.zeros(s["w"].shape[:2], dtype=torch.float32, device=DEV) if c["bias"] else None
    for e, a, b in s["segments"]:
        dz = plain_dz(c["act"], None if s["z"] is None else s["z"][a:b].float(), s["dy"][a:b].float())
        s["dx"][a:b] = dz @ s["w"][e].float()
        dw[e] = dz.t() @ s["x"][a:b].float()
        if c["bias"]:
            db[e] = dz.sum(0)
    return {"dx": s["dx"], "dw": dw} | ({"db": db} if c["bias"] else {})


# ------------------------------------------------------------------------------------------ the framework's calls

def own_router(s):
    c, op = s["case"], s["router"]
    if c["op"] == "route":
        weights, indices = op.forward(s["logits"], s["bias"], num_tokens=s["ntok"])
        return {"weights": weights, "indices": indices}
    if c["op"] == "train":
        weights, indices, counts, loss = op.forward(s["logits"], s["bias"], num_tokens=s["ntok"], balance=True)
        d = op.backward(s["logits"], indices, d_weights=s["d_weights"], counts=counts, d_loss=s["d_loss"], num_tokens=s["ntok"])
        return {"counts": counts, "loss": loss, "weights": weights, "indices": indices, "d_logits": d}
    counts, loss = op.balance_loss(s["logits"], s["indices"], num_tokens=s["ntok"])
    d = op.backward(s["logits"], s["indices"], counts=counts, d_loss=s["d_loss"], num_tokens=s["ntok"])
    return {"counts": counts, "loss": loss, "d_logits": d}


def own_linear(s):
    c, op = s["case"], s["linear"]
    at = {"row_begin": s["begin"], "row_count": s["count"]} if c["groups"] > 1 else {}
    if c["op"] == "linear":
        op.forward(s["x"], s["w"], bias=s["b"], residual=s["r"], out=s["y"], preact=s["z"], **at)
        return {"y": s["y"]} | ({"z": s["z"]} if c["preact"] else {})
    dx, dw, db = op.backward(s["dy"], s["x"], s["w"], preact=s["z"], want_dbias=c["bias"], dx=s["dx"], **at)
    return {"dx": dx, "dw": dw} | ({"db": db} if c["bias"] else {})


def run(state):
    linear_ = state["case"]["op"].startswith("linear")
    if own:
        return own_linear(state) if linear_ else own_router(state)
    if linear_:
        return plain_linear(state) if state["case"]["op"] == "linear" else plain_linear_backward(state)
    return plain_router(state)


# ------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return (exact_linear if case["op"].startswith("linear") else exact_router)(s)


def exact_pick(s, low, shut):
    """One best expert after another, of the best groups found the same way; scores are the 32-bit values that the definition compares."""
    c = s["case"]
    score = low if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-low)) + (0.0 if s["bias"] is None else s["bias"])
    score = score.masked_fill(shut, -math.inf)

    def best(v):
        top = v.amax(-1, keepdim=True)
        place = torch.arange(v.shape[-1], device=DEV).expand_as(v).masked_fill(v < top, v.shape[-1]).amin(-1, keepdim=True)
        return top, place

    if c["groups"] > 1:
        by = score.unflatten(-1, (c["groups"], -1))
        first, place = best(by)
        worth = first
        if c["score"] == "sigmoid":
            second = best(by.scatter(-1, place, -math.inf))[0]
            worth = first + second.masked_fill(second == -math.inf, 0.0)
        worth, keep = worth[..., 0], torch.zeros(by.shape[:-1], dtype=torch.bool, device=DEV)
        for _ in range(c["topk_groups"]):
            top, place = best(worth.masked_fill(keep, -math.inf))
            keep = keep | (torch.zeros_like(keep).scatter(-1, place, True) & (top > -math.inf))
        score = by.masked_fill(~keep[..., None], -math.inf).flatten(-2)
    picked = []
    for _ in range(c["topk"]):
        top, place = best(score)
        picked.append(place.masked_fill(top == -math.inf, -1))
        score = score.scatter(-1, place, -math.inf)
    return torch.cat(picked, -1)


def exact_router(s):
    """From the definition in 64 bits; which experts are selected goes by the scores as they are in 32 bits."""
    c = s["case"]
    r, t, e, k = c["world"], c["tokens"], c["experts"], c["topk"]
    low = s["logits"].float()
    shut = ~(low > LOWEST[s["logits"].dtype]) | ~s["valid"][..., None]
    l = low.double().masked_fill(shut, -math.inf)
    if c["score"] == "softmax":
        top = l.amax(-1, keepdim=True)
        raw = torch.exp(l - top.masked_fill(top == -math.inf, 0.0))
    else:
        raw = torch.sigmoid(l)
    total = raw.sum(-1, keepdim=True)
    prob = raw / total.masked_fill(total == 0, 1.0)
    if c["op"] == "balance":
        at = s["indices"].long().masked_fill(~s["valid"][..., None], -1)
    else:
        at = exact_pick(s, low, shut)
    hot = torch.zeros((r, t, e + 1), dtype=torch.float64, device=DEV)
    hot.scatter_add_(-1, at.masked_fill(at < 0, e), torch.ones_like(at, dtype=torch.float64))
    hot = hot[..., :e]
    out, d = {}, torch.zeros_like(raw)
    if c["op"] != "balance":
        chosen = raw * hot
        if c["normalize"] and c["score"] == "softmax":
            best = l.masked_fill(hot == 0, -math.inf).amax(-1, keepdim=True)
            chosen = torch.exp(l - best.masked_fill(best == -math.inf, 0.0)) * hot
        sums = chosen.sum(-1, keepdim=True) if c["normalize"] else total if c["score"] == "softmax" else torch.ones_like(total)
        sums = sums.masked_fill(sums == 0, 1.0)
        share = chosen / sums
        w = share.gather(-1, at.clamp(min=0)).masked_fill(at < 0, 0.0) * c["scale"]
        out |= {"weights": w, "indices": None}
        if c["op"] == "route":
            return out
        up = torch.zeros_like(hot).scatter_add_(-1, at.clamp(min=0), (s["d_weights"].double() * c["scale"]).masked_fill(at < 0, 0.0))
        mean = (share * up).sum(-1, keepdim=True)
        if c["score"] == "softmax":
            d = share * (up - mean) if c["normalize"] else share * up - prob * mean
        else:
            d = ((up - mean) / sums if c["normalize"] else up) * hot * raw * (1 - raw)
    length = c["seq_len"] or t
    pieces = [(i, a, min(a + length, s["ntok"][i])) for i in range(r) for a in range(0, t, length)]
    scale = float(s["d_loss"].double())
    if not c["seq_len"]:  # all ranks are one segment
        held = sum(s["ntok"])
        f = hot.sum((0, 1)) * e / (k * max(held, 1))
        loss = 0.01 * (f * prob.sum((0, 1))).sum() / max(held, 1)
        g = (0.01 * scale / max(held, 1) * f).expand(r, t, e)
    else:
        full = max(1, sum(b > a for _, a, b in pieces))
        loss, g = torch.zeros((), dtype=torch.float64, device=DEV), torch.zeros_like(raw)
        for i, a, b in pieces:
            if b > a:
                f = hot[i, a:b].sum(0) * e / (k * (b - a))
                loss = loss + 0.01 / full * (f * prob[i, a:b].sum(0)).sum() / (b - a)
                g[i, a:b] = 0.01 * scale / full / (b - a) * f
    slope = prob if c["score"] == "softmax" else prob * (1 - raw)
    d = d + slope * (g - (g * prob).sum(-1, keepdim=True))
    return out | {"counts": None, "loss": loss, "d_logits": d.masked_fill(shut, 0.0)}


def exact_linear(s):
    c = s["case"]
    n, act = c["n"], c["act"]
    forward = c["op"] == "linear"
    pool = s["x"].shape[0]
    outs = {"y": (pool, n)} if forward else {"dx": (pool, c["k"]), "dw": tuple(s["w"].shape)}
    if c["preact"] and forward:
        outs["z"] = tuple(s["z"].shape)
    if c["bias"] and not forward:
        outs["db"] = tuple(s["w"].shape[:2])
    outs = {name: torch.zeros(shape, dtype=torch.float64, device=DEV) for name, shape in outs.items()}
    for e, a, b in s["segments"]:
        x, w = s["x"][a:b].double(), s["w"][e].double()
        if forward:
            z = torch.matmul(x, w.T) + (s["b"][e].double() if c["bias"] else 0.0)
        elif act != "none":
            z = s["z"][a:b].double()
        if act == "swiglu":
            sig = torch.sigmoid(z[:, :n])
            h, slope = z[:, :n] * sig, sig * (1 + z[:, :n] * (1 - sig))
            y, dz = h * z[:, n:], lambda dy: torch.cat((dy * z[:, n:] * slope, dy * h), 1)  # noqa: E731
        elif act == "silu":
            sig = torch.sigmoid(z)
            y, dz = z * sig, lambda dy: dy * sig * (1 + z * (1 - sig))  # noqa: E731
        elif act == "gelu":
            phi = torch.special.ndtr(z)
            y, dz = z * phi, lambda dy: dy * (phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))  # noqa: E731
        elif act == "relu":
            y, dz = torch.relu(z), lambda dy: dy * (z > 0)  # noqa: E731
        else:
            y, dz = (z if forward else None), lambda dy: dy  # noqa: E731
        if forward:
            outs["y"][a:b] = y + (s["r"][a:b].double() if c["residual"] else 0.0)
            if c["preact"]:
                outs["z"][a:b] = z
        else:
            d = dz(s["dy"][a:b].double())
            outs["dx"][a:b] = torch.matmul(d, w)
            outs["dw"][e] = torch.matmul(d.T, x)
            if c["bias"]:
                outs["db"][e] = d.sum(0)
    return outs
