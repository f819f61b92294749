"""The block-quantised products with their quantisers and the norms around a block: plain forms, cases and the calls of the framework's operators.

Each case names its operator in "op":
  "quantize"          rows of a pool to E4M3 codes with an f32 scale for each 128 of a row, dense or per expert segment
  "quantize_weight"   matrices to E4M3 codes with an f32 scale for each 128 x 128
  "product"           y = act(x W^T + b) + residual of such x and W, one dense product or one per expert segment of a row pool
  "product_backward"  dx, dW, db of the same: dx of dz quantised by rows, dW of dz and x themselves
  "norm"              stream = residual + alpha gate norm(block), out = norm(stream): a block's end and the next one's beginning
  "norm_backward"     the gradients of the same
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the gated experts' hidden rows between their two products, mid-size shape with 5 % of slots dropped
        quantize("rows prefill", 128, 124518, 2048),
        # an optimiser's new weights of 32 experts' first product
        quantize("weights", 32, 4096, 4096, op="quantize_weight"),
        # one token through a dense layer: weights are all there is to read
        product("single token", 1, 1, 4096, 4096, act="gelu", bias=True, residual=True),
        # an odd dense layer, f32 results
        product("dense odd", 1, 1003, 1008, 777, act="silu", bias=True, residual=True, out="f32"),
        # gated experts' first product at decode size: 8 ranks x 128 tokens x top-8 over 256 experts
        product("experts decode", 256, 8192, 7168, 512, act="swiglu"),
        # gated experts' first product at prefill size, pre-activation kept for training
        product("experts prefill", 128, 124518, 4096, 2048, act="swiglu", bias=True, preact=True),
        # its backward pass
        product("experts backward", 128, 124518, 4096, 2048, op="product_backward", act="swiglu", bias=True),
        # the smallest experts' backward pass, SiLU
        product("experts backward tiny", 32, 512, 256, 512, op="product_backward", act="silu", bias=True),
        # 8 ranks x 16 tokens of a decode step: combine's f32 sums join the stream, the next block reads E4M3
        norm("norm decode", 128, 7168, block="f32", quant=True),
        # one prefill step of 8 ranks x 4096 tokens with a norm and a gate behind the block too
        norm("norm prefill", 32768, 7168, post=True, gate="feature", alpha=0.5),
        # a training step's backward pass, mid-size: 8 ranks x 2048 tokens, a gate for each token
        norm("norm backward", 16384, 4096, op="norm_backward", post=True, gate="token", alpha=0.5),
        # a small odd one over an f32 stream
        norm("norm backward odd", 1003, 1000, op="norm_backward", gate="feature", stream="f32", block="f32"),
    ]


def quantize(name, groups, rows, k, op="quantize", dtype="bf16", skew=0.0):
    c = {"op": op, "groups": groups, "rows": rows, "k": k, "dtype": dtype, "skew": skew}
    return {"name": name, **c} if name else c


def product(name, groups, rows, k, n, op="product", act="none", bias=False, residual=False, preact=False, out="bf16", skew=0.0):
    c = {"op": op, "groups": groups, "rows": rows, "k": k, "n": n, "act": act, "bias": bias, "residual": residual, "preact": preact, "out": out, "skew": skew}
    return {"name": name, **c} if name else c


def norm(name, rows, k, op="norm", post=False, gate="none", alpha=1.0, quant=False, stream="bf16", block="bf16"):
    c = {"op": op, "rows": rows, "k": k, "post": post, "gate": gate, "alpha": alpha, "quant": quant, "stream": stream, "block": block}
    return {"name": name, **c} if name else c


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["quantize", "quantize_weight", "product", "product", "product_backward", "norm", "norm_backward"])
    if op == "quantize_weight":
        return quantize(None, log(1, 32), log(1, 4096), 16 * log(8, 256), op=op, dtype=rng.choice(["bf16", "f32"]))
    if op.startswith("norm"):
        rows, k = log(1, 16384), 8 * log(8, 896)
        types = {"stream": rng.choice(["bf16", "bf16", "f32"]), "block": rng.choice(["bf16", "f32"])}
        return norm(None, rows, k, op=op, post=rng.random() < 0.5, gate=rng.choice(["none", "token", "feature"]), alpha=rng.choice([1.0, 0.5, 0.22]),
                    quant=op == "norm" and rng.random() < 0.5, **types)
    groups = rng.choice([1, 1, 8, 32, 128])
    rows, k, skew = log(1, 4096) if groups == 1 else groups * log(1, 512), 16 * log(8, 384), rng.choice([0.0, 0.5])
    if op == "quantize":
        return quantize(None, groups, rows, k, dtype=rng.choice(["bf16", "f32"]), skew=skew)
    n = min(log(100, 4096), (1 << 30) // (groups * k))
    act, bias = rng.choice(["none", "relu", "gelu", "silu", "swiglu"]), rng.random() < 0.5
    if op == "product_backward":
        return product(None, groups, rows, k, n, op=op, act=act, bias=bias, skew=skew)
    return product(None, groups, rows, k, n, act=act, bias=bias, residual=rng.random() < 0.5, preact=act != "none" and rng.random() < 0.5,
                   out=rng.choice(["bf16", "bf16", "f32"]), skew=skew)


def blocks(n):
    return -(-n // 128)


def work(case):
    c = case
    m, k = c["rows"], c["k"]
    if c["op"].startswith("quantize"):
        size = 4 if c["dtype"] == "f32" else 2
        if c["op"] == "quantize":
            return {"bytes": m * k * (size + 1) + 4 * m * blocks(k), "flops": 4 * m * k}
        return {"bytes": c["groups"] * (m * k * (size + 1) + 4 * blocks(m) * blocks(k)), "flops": 4 * c["groups"] * m * k}
    if c["op"].startswith("norm"):
        stream, block = (4 if c[t] == "f32" else 2 for t in ("stream", "block"))
        side = 4 * k * (1 + c["post"] + (c["gate"] == "feature")) + (4 * m if c["gate"] == "token" else 0)
        if c["op"] == "norm":
            return {"bytes": m * (k * (2 * stream + block) + (k + 4 * blocks(k) if c["quant"] else 2 * k)) + side, "flops": 12 * m * k}
        return {"bytes": m * k * (2 + 3 * stream + 2 * block) + 2 * side, "flops": 24 * m * k}
    g, n = c["groups"], c["n"]
    nw, out = n * (2 if c["act"] == "swiglu" else 1), 4 if c["out"] == "f32" else 2
    held = min(g, m)  # experts that can hold a row
    x, w = m * (k + 4 * blocks(k)), held * (nw * k + 4 * blocks(n) * (nw // n) * blocks(k))
    bias = 4 * g * nw if c["bias"] else 0
    if c["op"] == "product":
        return {"bytes": x + w + out * m * n * (2 if c["residual"] else 1) + (2 * m * nw if c["preact"] else 0) + bias, "flops": 2 * m * nw * k}
    return {"bytes": x + w + 2 * m * k + 2 * g * nw * k + out * m * n + (2 * m * nw if c["act"] != "none" else 0) + bias, "flops": 4 * m * nw * k}


# ------------------------------------------------------------------------------------------ inputs

def gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 64 + stream)
    return g


def normal(g, *shape, dtype=torch.float32, std=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    return x.normal_(0.0, std, generator=g)


def uneven(seed, stream, rows, k, dtype):
    """Rows of different magnitudes, as tokens have them."""
    return (normal(gen(seed, stream), rows, k) * torch.exp(0.5 * normal(gen(seed, stream + 1), rows, 1))).to(dtype)


def segments(s, c, seed):
    """Rows of each expert, a multinomial draw of equal or (skew) of Zipf popularity, in segments padded to whole 128-row blocks."""
    g, m = c["groups"], c["rows"]
    if g == 1:
        counts, begins, s["pool"] = np.array([m]), np.array([0]), m
    else:
        p = np.arange(1, g + 1, dtype=np.float64) ** -c["skew"]
        counts = np.random.RandomState(seed % (1 << 32)).multinomial(m, p / p.sum())
        padded = -(-counts // 128) * 128
        begins, s["pool"] = np.cumsum(padded) - padded, m + 127 * g
        s["begin"] = torch.tensor(begins, dtype=torch.int32, device=DEV)
        s["count"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
    # pool row of each expert's rows, experts side by side, and which of them there are
    i, most = np.arange(counts.max()), s["pool"] - 1
    s["at"] = torch.tensor(np.minimum(begins[:, None] + i, most), device=DEV)
    s["held"] = torch.tensor(i < counts[:, None], device=DEV)
    s["rows"] = s["at"][s["held"]]


def prepare(case, seed):
    c = case
    m, k = c["rows"], c["k"]
    s = {"case": c}
    if c["op"] == "quantize_weight":
        g = c["groups"]
        s["x"] = normal(gen(seed, 1), g, m, k, dtype=TYPES[c["dtype"]], std=k ** -0.5)
        if own:
            from combine_route_layout_gb300 import EpQuantConfig, EpQuantOp
            s["op"] = EpQuantOp(EpQuantConfig(num_groups=g, features=k, max_rows=m, block_rows=128, dtype=TYPES[c["dtype"]]))
    elif c["op"] == "quantize":
        segments(s, c, seed)
        s["x"] = uneven(seed, 1, s["pool"], k, TYPES[c["dtype"]])
        # rows of no expert are never written
        s["codes"] = torch.zeros((s["pool"], k), dtype=torch.float8_e4m3fn, device=DEV)
        s["scales"] = torch.zeros((s["pool"], blocks(k)), device=DEV)
        if own:
            from combine_route_layout_gb300 import EpQuantConfig, EpQuantOp
            s["op"] = EpQuantOp(EpQuantConfig(num_groups=c["groups"], features=k, max_rows=s["pool"], dtype=TYPES[c["dtype"]]))
    elif c["op"].startswith("norm"):
        prepare_norm(s, c, seed)
    else:
        prepare_product(s, c, seed)
    return s


def prepare_product(s, c, seed):
    k, n, bf = c["k"], c["n"], torch.bfloat16
    parts = 2 if c["act"] == "swiglu" else 1
    g, nw, out = c["groups"], n * parts, TYPES[c["out"]]
    segments(s, c, seed)
    pool = s["pool"]
    s["x"], s["xs"] = plain_quantize(uneven(seed, 1, pool, k, bf))
    codes, scales = plain_quantize_weight(normal(gen(seed, 3), g * parts, n, k, dtype=bf, std=k ** -0.5))
    s["w"], s["ws"] = codes.view(g, nw, k), scales.view(g, parts * blocks(n), blocks(k))
    s["b"] = normal(gen(seed, 4), g, nw, std=0.1) if c["bias"] else None
    if c["op"] == "product":
        s["r"] = normal(gen(seed, 5), pool, n, dtype=out) if c["residual"] else None
        s["y"] = torch.zeros((pool, n), dtype=out, device=DEV)
        s["z"] = torch.zeros((pool, nw), dtype=bf, device=DEV) if c["preact"] else None
    else:
        s["dy"] = uneven(seed, 6, pool, n, out)
        s["z"] = normal(gen(seed, 8), pool, nw, dtype=bf) if c["act"] != "none" else None
        s["dx"] = torch.zeros((pool, k), dtype=bf, device=DEV)
    if own:
        from combine_route_layout_gb300 import EpLinearConfig, EpQuantLinearOp
        s["op"] = EpQuantLinearOp(EpLinearConfig(num_groups=g, in_features=k, out_features=n, max_rows=pool, out_dtype=out, activation=c["act"]),
                                  backward=c["op"] != "product")


def prepare_norm(s, c, seed):
    m, k = c["rows"], c["k"]
    stream, block = TYPES[c["stream"]], TYPES[c["block"]]
    s["weight"] = 1.0 + 0.1 * normal(gen(seed, 1), k)
    s["weight_post"] = 1.0 + 0.1 * normal(gen(seed, 2), k) if c["post"] else None
    s["gate"] = None if c["gate"] == "none" else torch.sigmoid(normal(gen(seed, 3), m if c["gate"] == "token" else k))
    s["block"] = uneven(seed, 4, m, k, block)
    s["x"] = uneven(seed, 6, m, k, stream)  # the residual; in the backward pass the stream
    if c["op"] != "norm":
        s["dout"], s["dstream"] = normal(gen(seed, 8), m, k, dtype=torch.bfloat16), normal(gen(seed, 9), m, k, dtype=stream)
        both = [1.0 / torch.sqrt(s[t].double().square().mean(-1) + EPS) for t in ("x", "block")]
        s["stats"] = torch.stack(both if c["post"] else [both[0], torch.ones_like(both[0])], -1).float()
    if own:
        from combine_route_layout_gb300 import EpNormConfig, EpNormOp
        s["op"] = EpNormOp(EpNormConfig(hidden_dim=k, max_rows=m, eps=EPS, post_norm=c["post"], gate=c["gate"], residual_scale=c["alpha"], stream_dtype=stream,
                                        block_dtype=block, quant_type="fp8_e4m3_block128" if c["quant"] else "none"), backward=c["op"] != "norm")


# ------------------------------------------------------------------------------------------ plain forms

def in_blocks(x, *dims):
    """`x` with each of its last dimensions in `dims` cut into blocks of 128, zeros behind the last."""
    pad = [p for d in reversed(range(x.dim())) for p in (0, -x.shape[d] % 128 if d - x.dim() in dims else 0)]
    x = torch.nn.functional.pad(x.float(), pad)
    return x.unflatten(-1, (-1, 128)) if dims == (-1,) else x.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))


def scale_of(amax):
    """amax / 448 rounded once: by a tensor, since a division by a number may become a product."""
    return amax / amax.new_full((), 448.0)


def codes_of(v, scale):
    """E4M3 codes of v / scale; those of a block of zeros are zeros."""
    return torch.where(scale > 0, v / torch.where(scale > 0, scale, 1.0), v).to(torch.float8_e4m3fn)


def plain_quantize(x):
    v = in_blocks(x, -1)
    scale = scale_of(v.abs().amax(-1, keepdim=True))
    return codes_of(v, scale).flatten(-2)[..., :x.shape[-1]].contiguous(), scale[..., 0]


def plain_quantize_weight(x):
    v = in_blocks(x, -1, -2)
    scale = scale_of(v.abs().amax((-1, -3), keepdim=True))
    codes = codes_of(v, scale).flatten(-2).flatten(-3, -2)[:, :x.shape[-2], :x.shape[-1]]
    return codes.contiguous(), scale[..., 0, :, 0]


def values_of(codes, scale):
    """What codes with a scale for each 128 of a row stand for, in 32 bits."""
    return codes.float() * scale.repeat_interleave(128, -1)[..., :codes.shape[-1]]


def weights_of(s):
    c = s["case"]
    n, k, g = c["n"], c["k"], c["groups"]
    w = s["w"].view(-1, n, k)
    scale = s["ws"].view(-1, blocks(n), blocks(k)).repeat_interleave(128, -2)[:, :n]
    return values_of(w, scale).view(g, -1, k)


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


def beside(s, t):
    """Rows of the pool, experts side by side, zeros where an expert has fewer."""
    return torch.where(s["held"][..., None], t[s["at"]].float(), 0.0)


def into(s, name, t):
    s[name][s["rows"]] = t[s["held"]].to(s[name].dtype)


def plain_product(s):
    c = s["case"]
    z = torch.bmm(beside(s, values_of(s["x"], s["xs"])), weights_of(s).transpose(1, 2))
    if c["bias"]:
        z = z + s["b"][:, None]
    y = plain_act(c["act"], z)
    into(s, "y", y + beside(s, s["r"]) if c["residual"] else y)
    if c["preact"]:
        into(s, "z", z)
    return {"y": s["y"]} | ({"z": s["z"]} if c["preact"] else {})


def plain_product_backward(s):
    c = s["case"]
    dz = plain_dz(c["act"], None if s["z"] is None else beside(s, s["z"]), beside(s, s["dy"]))
    parts = dz.unflatten(-1, (-1, c["n"]))  # gate's and up's blocks are their own
    low = values_of(*plain_quantize(parts)).flatten(-2)
    into(s, "dx", torch.bmm(low, weights_of(s)))
    dw = torch.bmm(dz.transpose(1, 2), beside(s, values_of(s["x"], s["xs"]))).to(torch.bfloat16)
    return {"dx": s["dx"], "dw": dw} | ({"db": dz.sum(1)} if c["bias"] else {})


def rsqrt_mean(v):
    return 1.0 / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)


def gate_of(s):
    return 1.0 if s["gate"] is None else s["gate"][:, None] if s["case"]["gate"] == "token" else s["gate"]


def plain_norm(s):
    c, y = s["case"], s["block"].float()
    post = rsqrt_mean(y) if c["post"] else torch.ones_like(y[:, :1])
    u = y * post * s["weight_post"] if c["post"] else y
    stream = s["x"].float() + c["alpha"] * gate_of(s) * u
    r = rsqrt_mean(stream)
    h = stream * r * s["weight"]
    out = {"stream": stream.to(s["x"].dtype), "stats": torch.cat((r, post), -1)}
    if c["quant"]:
        codes, scales = plain_quantize(h)
        return out | {"codes": codes, "scales": scales}
    return out | {"out": h.to(torch.bfloat16)}


def plain_norm_backward(s):
    c, y, alpha = s["case"], s["block"].float(), s["case"]["alpha"]
    r, post = s["stats"][:, :1], s["stats"][:, 1:]
    unit = s["x"].float() * r
    d = s["dout"].float() * s["weight"]
    t = s["dstream"].float() + r * (d - unit * (d * unit).mean(-1, keepdim=True))
    unit_y = y * post
    u = unit_y * s["weight_post"] if c["post"] else y
    du = alpha * gate_of(s) * t
    d_block = du
    if c["post"]:
        e = du * s["weight_post"]
        d_block = post * (e - unit_y * (e * unit_y).mean(-1, keepdim=True))
    out = {"d_residual": t.to(s["x"].dtype), "d_block": d_block.to(s["block"].dtype), "d_weight": (s["dout"].float() * unit).sum(0)}
    if c["post"]:
        out["d_weight_post"] = (du * unit_y).sum(0)
    if s["gate"] is not None:
        out["d_gate"] = alpha * (u * t).sum(-1 if c["gate"] == "token" else 0)
    return out


def plain(s):
    op = s["case"]["op"]
    if op == "quantize":
        codes, scales = plain_quantize(s["x"][s["rows"]])
        s["codes"].view(torch.uint8)[s["rows"]] = codes.view(torch.uint8)
        s["scales"][s["rows"]] = scales
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "quantize_weight":
        codes, scales = plain_quantize_weight(s["x"])
        return {"codes": codes, "scales": scales}
    return {"product": plain_product, "product_backward": plain_product_backward, "norm": plain_norm, "norm_backward": plain_norm_backward}[op](s)


# ------------------------------------------------------------------------------------------ the framework's calls

def framework(s):
    c, op = s["case"], s["op"]
    at = {"row_begin": s["begin"], "row_count": s["count"]} if "begin" in s else {}
    if c["op"] == "quantize":
        codes, scales = op.quantize(s["x"], codes=s["codes"], scales=s["scales"], **at)
        return {"codes": codes, "scales": scales}
    if c["op"] == "quantize_weight":
        codes, scales = op.quantize(s["x"])
        return {"codes": codes, "scales": scales}
    if c["op"] == "product":
        op.forward(s["x"], s["xs"], s["w"], s["ws"], bias=s["b"], residual=s["r"], out=s["y"], preact=s["z"], **at)
        return {"y": s["y"]} | ({"z": s["z"]} if c["preact"] else {})
    if c["op"] == "product_backward":
        dx, dw, db = op.backward(s["dy"], s["x"], s["xs"], s["w"], s["ws"], preact=s["z"], want_dbias=c["bias"], dx=s["dx"], **at)
        return {"dx": dx, "dw": dw} | ({"db": db} if c["bias"] else {})
    if c["op"] == "norm":
        stream, out, scales, stats = op.forward(s["x"], s["weight"], block=s["block"], weight_post=s["weight_post"], gate=s["gate"])
        return {"stream": stream, "stats": stats} | ({"codes": out, "scales": scales} if c["quant"] else {"out": out})
    g = op.backward(s["dout"], s["x"], s["weight"], s["stats"], d_stream=s["dstream"], block=s["block"], weight_post=s["weight_post"], gate=s["gate"])
    out = {"d_residual": g[0], "d_block": g[1], "d_weight": g[2]}
    return out | ({"d_weight_post": g[3]} if c["post"] else {}) | ({"d_gate": g[4]} if s["gate"] is not None else {})


def run(state):
    return framework(state) if own else plain(state)


# ------------------------------------------------------------------------------------------ 64 bits

def nearest_e4m3(v):
    """v rounded to the nearest multiple of E4M3's step at its magnitude, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step


def exact_codes(x, each):
    """(codes, scales) of a matrix (or many) by the definition: blocks of each[0] rows and 128 columns, the scale rounded to 32 bits."""
    rows, cols = x.shape[-2:]
    r, k = each, 128
    full = torch.zeros(x.shape[:-2] + (-(-rows // r) * r, -(-cols // k) * k), dtype=torch.float64, device=DEV)
    full[..., :rows, :cols] = x
    cut = full.view(x.shape[:-2] + (-1, r, full.shape[-1] // k, k))
    scale = (cut.abs().amax((-1, -3)) / 448.0).float().double()
    by = scale.masked_fill(scale == 0, 1.0)[..., :, None, :, None]
    return nearest_e4m3(cut / by).view(full.shape)[..., :rows, :cols], scale


def exact_weights(s):
    c = s["case"]
    g, n, k = c["groups"], c["n"], c["k"]
    row = torch.arange(s["w"].shape[1], device=DEV)
    scale = s["ws"].double()[:, row // n * blocks(n) + row % n // 128]
    return s["w"].double() * scale[:, :, torch.arange(k, device=DEV) // 128]


def exact_rows(s, t):
    return t.double()[s["at"]].masked_fill(~s["held"][..., None], 0.0)


def exact_x(s):
    col = torch.arange(s["case"]["k"], device=DEV) // 128
    return exact_rows(s, s["x"]) * exact_rows(s, s["xs"])[..., col]


def exact_pool(s, t):
    out = torch.zeros((s["pool"], t.shape[-1]), dtype=torch.float64, device=DEV)
    out[s["rows"]] = t[s["held"]]
    return out


def exact_product(s):
    c = s["case"]
    n, act = c["n"], c["act"]
    z = torch.matmul(exact_x(s), exact_weights(s).mT)
    if c["bias"]:
        z += s["b"].double().unsqueeze(1)
    if act == "swiglu":
        y = z[..., :n] * torch.sigmoid(z[..., :n]) * z[..., n:]
    elif act == "silu":
        y = z * torch.sigmoid(z)
    elif act == "gelu":
        y = z * torch.special.ndtr(z)
    else:
        y = torch.relu(z) if act == "relu" else z
    if c["residual"]:
        y = y + exact_rows(s, s["r"])
    return {"y": exact_pool(s, y)} | ({"z": exact_pool(s, z)} if c["preact"] else {})


def exact_product_backward(s):
    c = s["case"]
    n, act, dy = c["n"], c["act"], exact_rows(s, s["dy"])
    z = None if act == "none" else exact_rows(s, s["z"])
    if act == "swiglu":
        gate, up = z[..., :n], z[..., n:]
        sig = torch.sigmoid(gate)
        halves = [dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig]
    elif act == "silu":
        sig = torch.sigmoid(z)
        halves = [dy * sig * (1 + z * (1 - sig))]
    elif act == "gelu":
        halves = [dy * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))]
    else:
        halves = [dy * (z > 0) if act == "relu" else dy]
    dz = torch.cat(halves, -1)
    half = torch.stack(halves)
    codes, scales = exact_codes(half, 1)
    low = codes * scales[..., torch.arange(n, device=DEV) // 128]
    dx = torch.matmul(low.movedim(0, -2).flatten(-2), exact_weights(s))
    out = {"dx": exact_pool(s, dx), "dw": torch.matmul(dz.mT, exact_x(s))}
    return out | ({"db": dz.sum(1)} if c["bias"] else {})


def exact_norm(s):
    c = s["case"]
    x, y = s["x"].double(), s["block"].double()
    gate = torch.ones((), dtype=torch.float64, device=DEV) if s["gate"] is None else s["gate"].double().unsqueeze(-1) if c["gate"] == "token" else s["gate"].double()
    root = lambda v: torch.rsqrt((v * v).sum(-1) / c["k"] + EPS).unsqueeze(-1)  # noqa: E731
    by_y = root(y) if c["post"] else torch.ones_like(y[:, :1])
    if c["op"] == "norm":
        x = x + c["alpha"] * gate * (y * by_y * s["weight_post"].double() if c["post"] else y)
        h = x * root(x) * s["weight"].double()
        out = {"stream": x, "stats": torch.cat((root(x), by_y), 1)}
        if c["quant"]:
            codes, scales = exact_codes(h, 1)
            return out | {"codes": codes, "scales": scales}
        return out | {"out": h}
    a, b = s["stats"].double().split(1, 1)
    dh = s["dout"].double()
    v = dh * s["weight"].double()
    t = s["dstream"].double() + v * a - x * a ** 3 * (v * x).sum(-1, keepdim=True) / c["k"]
    out = {"d_residual": t, "d_weight": (dh * x * a).sum(0)}
    w = s["weight_post"].double() if c["post"] else torch.ones_like(y[0])
    if s["gate"] is not None:
        out["d_gate"] = (c["alpha"] * t * y * b * w).sum(1 if c["gate"] == "token" else 0)
    du = c["alpha"] * gate * t
    out["d_block"] = du
    if c["post"]:
        out["d_weight_post"] = (du * y * b).sum(0)
        out["d_block"] = du * w * b - y * b ** 3 * (du * w * y).sum(-1, keepdim=True) / c["k"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize_weight":
        codes, scales = exact_codes(s["x"].double(), 128)
        return {"codes": codes, "scales": scales}
    if op == "quantize":
        codes, scales = exact_codes(s["x"].double()[s["rows"]], 1)
        full = [torch.zeros((s["pool"], v.shape[-1]), dtype=torch.float64, device=DEV).index_copy_(0, s["rows"], v) for v in (codes, scales)]
        return {"codes": full[0], "scales": full[1]}
    return exact_product(s) if op == "product" else exact_product_backward(s) if op == "product_backward" else exact_norm(s)
