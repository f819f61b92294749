"""GPU tests of the router, its balance loss and the experts' products against
plain 64-bit implementations, at the sizes and masks where they can go wrong.

Tolerances. A sum of n f32 terms, in any order and with steps that round or cut
off, is off by at most n * 2^-23 of the sum of magnitudes; exp, erf and division
add a few 2^-24. Router rows sum a few hundred terms that decay quickly, so
1e-5 of the largest magnitude bounds them; products use n * 2^-23 with their own
n. bf16 results have one rounding more, half of bf16's spacing, which is 2^-7 of
the value at most: 2^-8. dx and dW go through dz rounded to bf16: each of their
terms is off by at most 2^-8 of itself, so 2^-8 of the sum of the terms'
magnitudes bounds that part.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32_LOWEST = -3.4028234663852886e38
BF16_LOWEST = -3.3895313892515355e38


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def ulp_close(got, want, dtype, scale=None, terms=84):
    """|got - want| within the bounds above; `scale`: sums of magnitudes (of `terms` terms)."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    mag = want.abs() if scale is None else torch.maximum(want.abs(), scale.double().cpu())
    top = mag.max() if mag.numel() else 0.0
    bound = max(84, terms) * 2.0 ** -23 * (mag + top) + (want.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    off = (got - want).abs() - bound
    assert (off <= 0).all(), f"{float(off.max())} over the bound at {int(off.argmax())}"


# --------------------------------------------------------------------- router

def plain_route(cfg, l, bias, ntok):
    """Indices by the definition, row by row, in numpy on the f32 scores."""
    R, T, E = l.shape
    k, G = cfg.num_experts_per_token, cfg.num_groups
    low = F32_LOWEST if cfg.logits_dtype == torch.float32 else BF16_LOWEST
    lf = l.float().cpu()
    # scores as the definition rounds them, on the device whose exp is meant
    if cfg.score_func == "sigmoid":
        s = (1.0 / (1.0 + torch.exp(-l.float())))
        c = (s if bias is None else s + bias).cpu().numpy()
    else:
        c = lf.numpy()
    open_ = (lf.numpy() > low) & (lf.numpy() < np.inf)
    idx = np.full((R, T, k), -1, np.int32)
    for r in range(R):
        for t in range(ntok[r]):
            left = [e for e in range(E) if open_[r, t, e]]
            if G > 1:
                size = E // G
                worth = {}
                for g in range(G):
                    best = sorted((c[r, t, e] for e in left if e // size == g), reverse=True)[:2]
                    if best:
                        worth[g] = best[0] if cfg.score_func == "softmax" or len(best) < 2 \
                            else np.float32(best[0] + best[1])
                kept = sorted(worth, key=lambda g: (-worth[g], g))[:cfg.topk_groups]
                left = [e for e in left if e // size in kept]
            pick = sorted(left, key=lambda e: (-c[r, t, e], e))[:k]
            idx[r, t, :len(pick)] = pick
    return torch.from_numpy(idx)


def router_math(cfg, l, idx, ntok):
    """(weights, loss, counts) in f64 with autograd through l (f64 leaf)."""
    R, T, E = l.shape
    k = cfg.num_experts_per_token
    low = F32_LOWEST if cfg.logits_dtype == torch.float32 else BF16_LOWEST
    dead = ~((l.detach() > low) & (l.detach() < math.inf))
    weights = torch.zeros((R, T, k), dtype=torch.float64)
    length = cfg.seq_len or T
    segs = {}
    for r in range(R):
        for t in range(ntok[r]):
            segs.setdefault((r, t // length) if cfg.seq_len else (0, 0), []).append((r, t))
    n_seg = R * -(-T // cfg.seq_len) if cfg.seq_len else 1
    per = -(-T // length)
    counts = torch.zeros((n_seg, E), dtype=torch.int64)
    rows, loss = [], torch.zeros((), dtype=torch.float64)
    w_rows = {}
    for r in range(R):
        for t in range(ntok[r]):
            x = l[r, t].masked_fill(dead[r, t], -math.inf)
            if dead[r, t].all():
                w_rows[r, t] = (None, torch.zeros(E, dtype=torch.float64))
                continue
            if cfg.score_func == "softmax":
                p = torch.softmax(x, -1)
                raw = p
            else:
                raw = torch.sigmoid(x)
                p = raw / raw.sum() if float(raw.detach().sum()) > 0 else raw * 0
            at = [int(e) for e in idx[r, t] if e >= 0 and not dead[r, t, e]]
            q = raw[at]
            if cfg.normalize_weights and at:
                q = torch.softmax(x[at], -1) if cfg.score_func == "softmax" else q / q.sum()
            w_rows[r, t] = (q * cfg.route_scale, p)
    out = []
    for (r, t), (q, p) in w_rows.items():
        if q is None:
            continue
        slots = [j for j in range(k) if idx[r, t, j] >= 0 and not dead[r, t, idx[r, t, j]]]
        out.append(((r, t), slots, q))
    weights = torch.zeros((R, T, k), dtype=torch.float64)
    flat = []
    for (r, t), slots, q in out:
        row = torch.zeros(k, dtype=torch.float64)
        row = row.index_put((torch.tensor(slots, dtype=torch.long),), q) if slots else row
        flat.append(((r, t), row))
    for (r, t), row in flat:
        weights[r, t] = row.detach()
    for key, members in segs.items():
        s = key[0] * per + key[1] if cfg.seq_len else 0
        for r, t in members:
            for e in idx[r, t].tolist():
                if 0 <= e < E:
                    counts[s, e] += 1
        P = sum(w_rows[m][1] for m in members) / len(members)
        f = counts[s].double() * E / (k * len(members))
        loss = loss + (f * P).sum() / len(segs)
    return weights, cfg.balance_coef * loss, counts, flat


def make_logits(cfg, seed, masked):
    g = torch.Generator().manual_seed(seed)
    R, T, E = cfg.world_size, cfg.max_num_inp_token_per_rank, cfg.num_experts
    l = torch.randn((R, T, E), generator=g)
    if masked:
        low = F32_LOWEST if cfg.logits_dtype == torch.float32 else BF16_LOWEST
        u = torch.rand((R, T, E), generator=g)
        l = torch.where(u < 0.2, torch.tensor(-math.inf), torch.where(u < 0.4, torch.tensor(low), l))
        l[0, 0] = -math.inf                       # a row with nothing left
        if T > 1:
            l[0, 1] = low
            l[0, 1, E - 1] = 0.25                 # a row with one expert left
    return l.to(cfg.logits_dtype).to(DEV)


ROUTER = [
    # world, T, E, k, score, groups, topk_groups, normalize, dtype, seq_len, masked, ntok, bias
    (1, 1, 1, 1, "softmax", 1, 1, True, torch.float32, 0, False, None, False),
    (1, 1, 8, 8, "sigmoid", 1, 1, True, torch.bfloat16, 0, False, None, True),
    (2, 5, 33, 4, "softmax", 1, 1, False, torch.float32, 2, True, [5, 3], False),
    (3, 70, 60, 6, "sigmoid", 6, 2, True, torch.float32, 0, True, [70, 0, 65], True),
    (2, 66, 64, 4, "softmax", 4, 2, True, torch.bfloat16, 64, True, [66, 64], False),
    (8, 16, 128, 8, "sigmoid", 8, 4, False, torch.bfloat16, 7, False, [16, 0, 1, 7, 8, 14, 15, 16], True),
    (1, 130, 256, 8, "sigmoid", 8, 4, True, torch.float32, 100, False, [129], True),
    (1, 9, 257, 32, "softmax", 1, 1, False, torch.float32, 0, True, None, False),
    (2, 3, 1000, 12, "sigmoid", 20, 3, True, torch.float32, 0, True, [3, 2], False),
    (1, 4, 1024, 32, "softmax", 32, 32, True, torch.bfloat16, 0, False, None, False),
]


def router_config(layer, c, coef=0.7):
    world, T, E, k, score, groups, tg, norm, dt, seq, masked, ntok, bias = c
    return layer.EpRouterConfig(world, T, E, k, logits_dtype=dt, score_func=score, num_groups=groups, topk_groups=tg,
                                normalize_weights=norm, route_scale=1.5, seq_len=seq, balance_coef=coef)


@pytest.mark.parametrize("c", ROUTER)
def test_router_forward_and_backward(layer, c):
    cfg = router_config(layer, c)
    masked, bias = c[10], c[12]
    ntok = c[11] or [cfg.max_num_inp_token_per_rank] * cfg.world_size
    l = make_logits(cfg, 5, masked)
    E, k = cfg.num_experts, cfg.num_experts_per_token
    b = torch.linspace(-0.3, 0.3, E, device=DEV).roll(3) if bias else None
    op = layer.EpRouterOp(cfg)
    w, idx, counts, loss = op.forward(l, b, num_tokens=c[11], balance=True)
    w2, idx2 = op.forward(l, b, num_tokens=c[11])
    assert torch.equal(w, w2) and torch.equal(idx, idx2)
    op.sync()
    want = plain_route(cfg, l, b, ntok)
    assert torch.equal(idx.cpu(), want)

    leaf = l.double().cpu().requires_grad_(True)
    wt, ls, ct, flat = router_math(cfg, leaf, want, ntok)
    ulp_close(w, wt, torch.float32)
    ulp_close(loss, ls.detach(), torch.float32)
    assert torch.equal(counts.cpu().long(), ct)
    for r in range(cfg.world_size):
        assert (idx[r, ntok[r]:] == -1).all() and (w[r, ntok[r]:] == 0).all()

    gen = torch.Generator().manual_seed(9)
    dw = torch.randn(w.shape, generator=gen)
    total = sum(((row * dw[r, t].double()).sum() for (r, t), row in flat), torch.zeros((), dtype=torch.float64))
    both = total + 1.25 * ls
    parts = [torch.autograd.grad(v, leaf, retain_graph=True, allow_unused=True)[0] if v.requires_grad else None
             for v in (total, 1.25 * ls, both)]
    low = F32_LOWEST if cfg.logits_dtype == torch.float32 else BF16_LOWEST
    dead = ~(leaf.detach() > low)
    parts = [torch.zeros_like(leaf) if p is None else torch.nan_to_num(p, nan=0.0).masked_fill(dead, 0.0) for p in parts]
    d_loss = torch.tensor(1.25, device=DEV)
    d1 = op.backward(l, idx, d_weights=dw.to(DEV), num_tokens=c[11])
    d2 = op.backward(l, counts=counts, d_loss=d_loss, num_tokens=c[11])
    d3 = op.backward(l, idx, d_weights=dw.to(DEV), counts=counts, d_loss=d_loss, num_tokens=c[11])
    for got, ref in zip((d1, d2, d3), parts):
        ulp_close(got, ref, cfg.logits_dtype, scale=torch.full_like(ref, 1.0) * (parts[0].abs().max() + parts[1].abs().max()))
        assert (got.cpu()[dead] == 0).all()

    got_counts, got_loss = op.balance_loss(l, idx, num_tokens=c[11])
    assert torch.equal(got_counts, counts) and torch.equal(got_loss, loss)
    op.sync()


def test_router_gradient_matches_differences(layer):
    """Central differences of sum(w * g) + loss in each logit of a row, f32:
    a step of 2^-6 leaves an error of h^2 / 6 times the third derivative
    (at most about 2 of these functions, times the gradient's scale of 2) and
    f32 rounding of 2^-24 * 4 / h; 1e-3 bounds both."""
    for score, norm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        cfg = layer.EpRouterConfig(1, 2, 12, 3, score_func=score, normalize_weights=norm)
        op = layer.EpRouterOp(cfg)
        l = 0.5 * torch.arange(24, device=DEV, dtype=torch.float32).reshape(1, 2, 12).sin() * 3
        g = torch.tensor([[[1.0, -2.0, 0.5], [0.3, 0.7, -1.0]]], device=DEV)
        w, idx, counts, loss = op.forward(l, balance=True)
        one = torch.ones((), device=DEV)
        d = op.backward(l, idx, d_weights=g, counts=counts, d_loss=one)
        h = 2.0 ** -6
        for t in range(2):
            for e in range(12):
                v = []
                for s in (h, -h):
                    m = l.clone()
                    m[0, t, e] += s
                    w2, idx2, c2, l2 = op.forward(m, balance=True)
                    assert torch.equal(idx2, idx)      # the step crosses no selection
                    v.append(float((w2.double() * g).sum() + l2.double()))
                assert abs((v[0] - v[1]) / (2 * h) - float(d[0, t, e])) < 1e-3


def test_sigmoid_scores_are_the_formula_s_own_bits(layer):
    """The scores that selection compares are 1 / (1 + exp(-l)) with each step
    rounded to f32. A grid of 2^-24 over l in [-1.11, 0] puts 1 + exp(-l) on
    every float in [2, 4): every significand a reciprocal can have. The rest of
    the range, and the far side of exp's, is sampled."""
    cfg = layer.EpRouterConfig(1, 1 << 18, 32, 32, score_func="sigmoid", normalize_weights=False)
    op = layer.EpRouterOp(cfg)
    n = 32 << 18
    fine = [-(torch.arange(n, device=DEV, dtype=torch.float64) + i * n) * 2.0 ** -24 for i in range(3)]
    gen = torch.Generator(device=DEV).manual_seed(4)
    wide = (torch.rand(n, generator=gen, device=DEV, dtype=torch.float64) * 2 - 1) * 120
    tiny = torch.randn(n, generator=gen, device=DEV, dtype=torch.float64) * 1e-4
    for l in (*fine, wide, tiny):
        l = l.float().view(1, -1, 32)
        w, idx = op.forward(l)
        s = 1.0 / (1.0 + torch.exp(-l))
        assert torch.equal(w, s.gather(-1, idx.long()))
        assert (w[..., :-1] >= w[..., 1:]).all()
        assert torch.equal(idx.sort(-1).values, torch.arange(32, device=DEV, dtype=torch.int32).expand_as(idx))


def test_router_over_2_31_logits(layer):
    """Offsets past 32 bits: 8 x 300,000 rows of 1,024 bf16 logits."""
    cfg = layer.EpRouterConfig(8, 300000, 1024, 2, logits_dtype=torch.bfloat16, balance_coef=2.0)
    op = layer.EpRouterOp(cfg)
    l = torch.zeros((8, 300000, 1024), dtype=torch.bfloat16, device=DEV)
    l[7, 299990:, 5] = 2.0
    l[7, 299990:, 1000] = 1.0
    l[7, 299990:, 1001:1005] = 0.5
    w, idx, counts, loss = op.forward(l, balance=True)
    assert idx[7, -1].tolist() == [5, 1000] and idx[0, 0].tolist() == [0, 1] and idx[7, 299989].tolist() == [0, 1]
    assert counts[0, 5] == 10 and counts[0, 1000] == 10 and counts[0, 0] == 2400000 - 10
    d = op.backward(l, idx, d_weights=torch.ones_like(w), counts=counts, d_loss=loss)
    small = layer.EpRouterOp(layer.EpRouterConfig(1, 16, 1024, 2, logits_dtype=torch.bfloat16))
    tail = l[7:, -16:].contiguous()
    assert torch.equal(small.forward(tail)[0], w[7:, -16:])
    assert torch.isfinite(d[7, -16:].float()).all() and (d[7, -1] != 0).any()


def test_router_ties_and_signed_zeros(layer):
    cfg = layer.EpRouterConfig(1, 3, 40, 5)
    op = layer.EpRouterOp(cfg)
    l = torch.zeros((1, 3, 40), device=DEV)
    l[0, 1, ::2] = -0.0
    l[0, 2, 7] = 1.0
    l[0, 2, 33] = 1.0
    w, idx = op.forward(l)
    assert idx[0, 0].tolist() == [0, 1, 2, 3, 4]
    assert idx[0, 1].tolist() == [0, 1, 2, 3, 4]
    assert idx[0, 2].tolist() == [7, 33, 0, 1, 2]
    assert torch.allclose(w.sum(-1), torch.ones_like(w.sum(-1)), atol=1e-6)


def test_router_extreme_logits(layer):
    """Logits of +-1e30 and beyond exp's range give finite weights and gradients."""
    cfg = layer.EpRouterConfig(1, 4, 16, 4, score_func="softmax")
    op = layer.EpRouterOp(cfg)
    l = torch.zeros((1, 4, 16), device=DEV)
    l[0, 0, 3] = 1e30
    l[0, 1] = -1e30
    l[0, 2, :8] = 200.0
    l[0, 3, 0] = -200.0
    w, idx, counts, loss = op.forward(l, balance=True)
    d = op.backward(l, idx, d_weights=torch.ones_like(w), counts=counts, d_loss=loss)
    assert torch.isfinite(w).all() and torch.isfinite(loss) and torch.isfinite(d).all()
    assert w[0, 0].tolist() == [1.0, 0.0, 0.0, 0.0] and idx[0, 0].tolist() == [3, 0, 1, 2]
    assert w[0, 1].tolist() == [0.25] * 4
    sig = layer.EpRouterOp(layer.EpRouterConfig(1, 4, 16, 4, score_func="sigmoid"))
    w, idx, counts, loss = sig.forward(l, balance=True)
    d = sig.backward(l, idx, d_weights=torch.ones_like(w), counts=counts, d_loss=loss)
    assert torch.isfinite(w).all() and torch.isfinite(loss) and torch.isfinite(d).all()
    assert (w[0, 1] == 0).all()                # every score underflowed
    op.sync()


def test_router_reports_bad_values(layer):
    from combine_route_layout_gb300 import ep
    cfg = layer.EpRouterConfig(1, 4, 16, 2)
    op = layer.EpRouterOp(cfg)
    l = torch.randn((1, 4, 16), device=DEV)
    l[0, 1, 5] = math.nan
    l[0, 2, 6] = math.inf
    w, idx = op.forward(l)
    with pytest.raises(ep.EpError) as ei:
        op.sync()
    assert ei.value.status == ep.EP_ERR_INVALID_ARG
    assert (idx >= 0).all() and 5 not in idx[0, 1].tolist() and 6 not in idx[0, 2].tolist()
    assert torch.isfinite(w).all()
    op.sync()                                   # reported once
    idx[0, 0, 0] = 16
    idx[0, 3, 1] = -7
    counts, _ = op.balance_loss(torch.zeros_like(l), idx)
    with pytest.raises(ep.EpError) as ei:
        op.sync()
    assert ei.value.status == ep.EP_ERR_INVALID_INDEX
    assert int(counts.sum()) == 6


@pytest.mark.parametrize("E,groups,stay", [(256, 1, 1), (256, 8, 4), (256, 32, 2), (96, 4, 2), (30, 3, 2), (7, 1, 1)])
def test_router_bias_that_is_not_finite(layer, E, groups, stay):
    """A bias of -inf or NaN leaves its expert out of the selection, NaN is reported; rows
    with no expert left hold index -1 and weight 0."""
    from combine_route_layout_gb300 import ep
    g = torch.Generator(device="cpu").manual_seed(E + groups)
    k = 4
    op = layer.EpRouterOp(layer.EpRouterConfig(1, 37, E, k, score_func="sigmoid", num_groups=groups,
                                               topk_groups=stay))
    l = torch.randn((1, 37, E), generator=g).to(DEV)
    w, idx = op.forward(l, bias=torch.full((E,), -math.inf, device=DEV))
    op.sync()
    assert (idx == -1).all() and (w == 0).all()
    w, idx = op.forward(l, bias=torch.full((E,), math.nan, device=DEV))
    with pytest.raises(ep.EpError) as ei:
        op.sync()
    assert ei.value.status == ep.EP_ERR_INVALID_ARG
    assert (idx == -1).all() and (w == 0).all()
    bias = torch.zeros(E)
    bias[0], bias[E // 2], bias[E - 1] = math.nan, -math.inf, math.nan
    w, idx = op.forward(l, bias=bias.to(DEV))
    with pytest.raises(ep.EpError):
        op.sync()
    out = bias.clone()
    out[[0, E // 2, E - 1]] = -math.inf
    w2, idx2 = op.forward(l, bias=out.to(DEV))
    op.sync()
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    assert not torch.isin(idx, torch.tensor([0, E // 2, E - 1], device=DEV)).any()
    assert (idx >= 0).all() and torch.allclose(w.sum(-1), torch.ones((), device=DEV), rtol=0, atol=7 * 2.0 ** -24)


def test_router_on_another_stream_and_in_a_graph(layer):
    cfg = layer.EpRouterConfig(4, 64, 64, 6, score_func="sigmoid")
    op = layer.EpRouterOp(cfg)
    l = torch.randn((4, 64, 64), device=DEV)
    want = op.forward(l, balance=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = op.forward(l, balance=True)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    fresh = layer.EpRouterOp(cfg)               # first call captured
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fresh.forward(l, balance=True)
    l2 = torch.randn((4, 64, 64), device=DEV)
    l.copy_(l2)
    g.replay()
    g.replay()
    again = op.forward(l2, balance=True)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    fresh.sync()


# ---------------------------------------------------------- experts' products

def act64(act, z):
    if act == "swiglu":
        a, u = z.chunk(2, -1)
        return torch.nn.functional.silu(a) * u
    return {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
            "gelu": torch.nn.functional.gelu}[act](z)


# groups, K, N, counts, act, bias, residual, out dtype, dweight dtype
LINEAR = [
    (1, 8, 1, [1], "none", True, True, torch.bfloat16, torch.bfloat16),
    (1, 72, 33, [3], "gelu", True, True, torch.float32, torch.float32),
    (1, 264, 300, [257], "silu", False, True, torch.bfloat16, torch.bfloat16),
    (3, 136, 257, [31, 0, 129], "relu", True, False, torch.bfloat16, torch.float32),
    (5, 64, 96, [0, 1, 16, 33, 300], "swiglu", True, True, torch.bfloat16, torch.bfloat16),
    (4, 200, 7, [65, 64, 63, 1], "swiglu", False, False, torch.float32, torch.bfloat16),
    (2, 512, 129, [700, 2500], "none", True, False, torch.float32, torch.float32),
    (40, 128, 64, [i % 7 * 11 for i in range(40)], "gelu", True, False, torch.bfloat16, torch.bfloat16),
    (2, 1000, 520, [1, 2], "silu", True, True, torch.bfloat16, torch.bfloat16),
    # one and two dense rows; contractions cut into parts, forward and dW, and joined
    (1, 2056, 40, [1], "swiglu", True, True, torch.bfloat16, torch.bfloat16),
    (1, 1032, 9, [2], "gelu", True, True, torch.float32, torch.bfloat16),
    (1, 4104, 96, [5], "none", True, True, torch.float32, torch.float32),
    (1, 4096, 200, [70], "relu", False, False, torch.bfloat16, torch.bfloat16),
    (2, 2048, 300, [3, 40], "swiglu", True, False, torch.bfloat16, torch.bfloat16),
    (1, 64, 72, [5003], "silu", True, False, torch.bfloat16, torch.bfloat16),
    (3, 72, 40, [0, 2500, 17], "none", True, False, torch.bfloat16, torch.float32),
]


class Product:
    """Inputs of one product; the rows outside the segments hold NaN."""

    def __init__(self, layer, c, packed=True, seed=3):
        self.c = c
        G, K, N, counts, act, bias, residual, out, dw = c
        gen = torch.Generator().manual_seed(seed)
        self.begins, at = [], 0
        for n in counts:
            self.begins.append(at)
            at += -(-n // 128) * 128 if packed else n + 3    # tight segments, any alignment
        self.dense = G == 1 and not packed
        rows = counts[0] if self.dense else at + 5
        self.rows = max(rows, 1)
        Nw = N * (2 if act == "swiglu" else 1)
        bf = torch.bfloat16
        used = torch.zeros(self.rows, dtype=torch.bool)
        for b, n in zip(self.begins, counts):
            used[b:b + n] = True
        self.used = used

        def pool(cols, dt):
            t = torch.randn((self.rows, cols), generator=gen).to(dt)
            t[~used] = math.nan
            return t.to(DEV)

        self.x, self.dy = pool(K, bf), pool(N, out)
        self.w = (torch.randn((G, Nw, K), generator=gen) * K ** -0.5).to(bf).to(DEV)
        self.b = torch.randn((G, Nw), generator=gen).to(DEV) if bias else None
        self.r = pool(N, out) if residual else None
        self.z = torch.full((self.rows, Nw), math.nan, dtype=bf, device=DEV)
        self.y = torch.full((self.rows, N), 7.0, dtype=out, device=DEV)
        self.dx = torch.full((self.rows, K), 7.0, dtype=bf, device=DEV)
        self.cfg = layer.EpLinearConfig(G, K, N, self.rows, out_dtype=out, weight_grad_dtype=dw, activation=act)
        self.at = {} if self.dense else {
            "row_begin": torch.tensor(self.begins, dtype=torch.int32, device=DEV),
            "row_count": torch.tensor(counts, dtype=torch.int32, device=DEV)}


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("c", LINEAR)
def test_linear_forward_and_backward(layer, c, packed):
    G, K, N, counts, act, bias, residual, out, dwt = c
    t = Product(layer, c, packed)
    op = layer.EpLinearOp(t.cfg, backward=True)
    op.forward(t.x, t.w, t.b, t.r, out=t.y, preact=t.z, **t.at)
    y2 = op.forward(t.x, t.w, t.b, t.r, out=torch.full_like(t.y, 7.0), **t.at)
    assert torch.equal(y2, t.y)                       # the same without preact
    dx, dw, db = op.backward(t.dy, t.x, t.w, t.z, want_dbias=True, dx=t.dx, **t.at)
    op.sync()
    keep = ~t.used.to(DEV)
    assert (t.y[keep] == 7.0).all() and (dx[keep] == 7.0).all() and torch.isnan(t.z[keep]).all()
    for g, (a, n) in enumerate(zip(t.begins, counts)):
        s = slice(a, a + n)
        if n == 0:
            assert (dw[g] == 0).all() and (db[g] == 0).all()
            continue
        x, w = t.x[s].double(), t.w[g].double()
        z = x @ w.t() + (t.b[g].double() if bias else 0.0)
        mag = x.abs() @ w.abs().t() + 1.0
        ulp_close(t.z[s], z, torch.bfloat16, scale=mag, terms=K)
        r = t.r[s].double() if residual else torch.zeros((), dtype=torch.float64, device=DEV)
        if act == "swiglu":
            zg, zu = z.chunk(2, -1)
            mag = mag[:, :N] * zu.abs() + mag[:, N:] * (zg.abs() + 1.0)
        ulp_close(t.y[s], act64(act, z) + r, out, scale=mag + r.abs(), terms=K)

        zs = t.z[s].double().requires_grad_(True)     # the backward pass starts from the stored z
        (dz,) = torch.autograd.grad((act64(act, zs) * t.dy[s].double()).sum(), zs)
        dz_mag = dz.abs() + 1e-3 * t.dy[s].double().abs().max()
        ulp_close(db[g], dz.sum(0), torch.float32, scale=dz_mag.sum(0), terms=n)
        for got, ref, m, dt, terms in ((dx[s], dz @ w, dz_mag @ w.abs(), torch.bfloat16, dz.shape[1]),
                                       (dw[g], dz.t() @ x, dz_mag.t() @ x.abs(), dwt, n)):
            got, ref = got.double(), ref.double()
            assert torch.isfinite(got).all()
            rounded = act != "none" or out == torch.float32     # dz had to be rounded
            bound = max(84, terms) * 2.0 ** -23 * (m + m.max()) + (m * 2.0 ** -8 if rounded else 0.0) + \
                (ref.abs() * 2.0 ** -8 if dt == torch.bfloat16 else 0.0)
            assert ((got - ref).abs() <= bound).all(), float(((got - ref).abs() - bound).max())


def test_linear_gradient_matches_differences(layer):
    """d(sum(y * g)) by central differences in entries of x, W and b, f32
    output. x and W move by bf16 steps; the function is smooth (SiLU), so a
    step h leaves h^2 / 6 of a third derivative of at most about 1 per term,
    and dz's rounding 2^-8 of the gradient's terms: 2 % of the gradient's scale
    bounds both."""
    G, K, N = 2, 16, 24
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((10, K), generator=gen).bfloat16().to(DEV)
    w = (torch.randn((G, N, K), generator=gen) * 0.25).bfloat16().to(DEV)
    b = torch.randn((G, N), generator=gen).to(DEV)
    g = torch.randn((10, N), generator=gen).to(DEV)
    at = {"row_begin": torch.tensor([0, 4], dtype=torch.int32, device=DEV),
          "row_count": torch.tensor([4, 6], dtype=torch.int32, device=DEV)}
    op = layer.EpLinearOp(layer.EpLinearConfig(G, K, N, 10, out_dtype=torch.float32, weight_grad_dtype=torch.float32,
                                               activation="silu"), backward=True)
    z = torch.empty((10, N), dtype=torch.bfloat16, device=DEV)
    op.forward(x, w, b, preact=z, **at)
    dx, dw, db = op.backward(g, x, w, z, want_dbias=True, **at)

    def value(x, w, b):
        return float((op.forward(x, w, b, **at).double() * g.double()).sum())

    for which, grad, places in (("x", dx, [(0, 0), (3, 15), (9, 7)]), ("w", dw, [(0, 0, 0), (1, 23, 15), (1, 3, 8)]),
                                ("b", db, [(0, 1), (1, 22)])):
        for place in places:
            moved = []
            for sign in (1, -1):
                t = {"x": x.clone(), "w": w.clone(), "b": b.clone()}
                t[which][place] += sign * 2.0 ** -5
                moved.append((float(t[which][place]), value(t["x"], t["w"], t["b"])))
            slope = (moved[0][1] - moved[1][1]) / (moved[0][0] - moved[1][0])
            assert abs(slope - float(grad[place])) < 0.02 * (1.0 + float(grad.float().abs().max()))


@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
def test_linear_keeps_nan_and_infinity_in_their_rows(layer, act, rows):
    """A NaN or an infinity in a row of x reaches that row's results as it does in the formula,
    and no other row's."""
    bf = torch.bfloat16
    K, N = 64, 40
    Nw = N * (2 if act == "swiglu" else 1)
    g = torch.Generator().manual_seed(5)
    x = torch.randn((rows, K), generator=g).to(bf).to(DEV)
    w = torch.randn((1, Nw, K), generator=g).to(bf).to(DEV)
    dy = torch.randn((rows, N), generator=g).to(bf).to(DEV)
    op = layer.EpLinearOp(layer.EpLinearConfig(1, K, N, rows, activation=act), backward=True)
    z = torch.empty((rows, Nw), dtype=bf, device=DEV)
    y = op.forward(x, w, preact=z)
    dx, _, _ = op.backward(dy, x, w, z)
    for value in (math.nan, math.inf):
        x2 = x.clone()
        x2[0, 3] = value
        z2 = torch.empty_like(z)
        y2 = op.forward(x2, w, preact=z2)
        dx2, _, _ = op.backward(dy, x2, w, z2)
        assert torch.equal(y2[1:], y[1:]) and torch.equal(dx2[1:], dx[1:])
        want = x2.double() @ w[0].double().t()
        assert torch.equal(z2[0].isnan(), want[0].isnan()) and torch.equal(z2[0].isinf(), want[0].isinf())
        assert torch.equal(z2[0][z2[0].isinf()].double(), want[0][want[0].isinf()])
        if math.isnan(value):
            assert y2[0].isnan().all() and (act in ("none", "relu") or dx2[0].isnan().all())
        elif act in ("none", "relu"):
            assert torch.equal(y2[0].double(), act64(act, want)[0])
    op.sync()


def test_linear_residual_may_be_the_output(layer):
    t = Product(layer, (1, 128, 200, [77], "gelu", True, True, torch.bfloat16, torch.bfloat16), packed=False)
    op = layer.EpLinearOp(t.cfg)
    want = op.forward(t.x, t.w, t.b, t.r)
    got = t.r.clone()
    op.forward(t.x, t.w, t.b, got, out=got)
    assert torch.equal(got, want)


def test_linear_cuts_segments_that_leave_the_pool(layer):
    from combine_route_layout_gb300 import ep
    K, N, rows = 64, 40, 50
    op = layer.EpLinearOp(layer.EpLinearConfig(4, K, N, rows), backward=True)
    x = torch.randn((rows, K), device=DEV).bfloat16()
    w = torch.randn((4, N, K), device=DEV).bfloat16()
    at = {"row_begin": torch.tensor([0, 40, -3, 60], dtype=torch.int32, device=DEV),
          "row_count": torch.tensor([10, 20, 2, 5], dtype=torch.int32, device=DEV)}
    y = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
    op.forward(x, w, out=y, **at)
    with pytest.raises(ep.EpError) as ei:
        op.sync()
    assert ei.value.status == ep.EP_ERR_INVALID_INDEX
    op.sync()
    ulp_close(y[:10], x[:10].double() @ w[0].double().t(), torch.bfloat16, scale=x[:10].double().abs() @ w[0].double().abs().t())
    ulp_close(y[40:], x[40:].double() @ w[1].double().t(), torch.bfloat16, scale=x[40:].double().abs() @ w[1].double().abs().t())
    assert (y[10:40] == 0).all()


def test_linear_over_2_31_values(layer):
    """Offsets past 32 bits in y, z, dy and dz: 270,000 rows of 8,192."""
    rows, K, N = 270000, 64, 8192
    cfg = layer.EpLinearConfig(2, K, N, rows, activation="relu")
    op = layer.EpLinearOp(cfg, backward=True)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((rows, K), generator=gen, device=DEV).bfloat16()
    w = torch.randn((2, N, K), generator=gen, device=DEV).bfloat16()
    at = {"row_begin": torch.tensor([0, rows - 300], dtype=torch.int32, device=DEV),
          "row_count": torch.tensor([rows - 300, 300], dtype=torch.int32, device=DEV)}
    z = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    y = op.forward(x, w, preact=z, **at)
    dy = torch.ones((rows, N), dtype=torch.bfloat16, device=DEV)
    dx, dw, db = op.backward(dy, x, w, z, want_dbias=True, **at)
    op.sync()
    s = slice(rows - 300, rows)
    ref = x[s].double() @ w[1].double().t()
    ulp_close(z[s], ref, torch.bfloat16, scale=x[s].double().abs() @ w[1].double().abs().t())
    assert torch.equal(y[s], z[s].clamp(min=0))
    g = (z[s] > 0).double()
    ulp_close(dx[s], g @ w[1].double(), torch.bfloat16, scale=g @ w[1].double().abs(), terms=N)
    ulp_close(dw[1], g.t() @ x[s].double(), torch.bfloat16, scale=g.t() @ x[s].double().abs(), terms=300)
    ulp_close(db[1], g.sum(0), torch.float32)
    g0 = (z[:rows - 300] > 0).sum(0)
    assert (db[0].long() - g0).abs().max() <= rows * 2.0 ** -23 * rows


def test_linear_in_a_graph_with_changing_counts(layer):
    """Counts are read on the device: a captured product follows them."""
    t = Product(layer, (3, 64, 48, [100, 1, 128], "swiglu", True, False, torch.bfloat16, torch.bfloat16))
    op = layer.EpLinearOp(t.cfg, backward=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(t.x, t.w, t.b, out=t.y, preact=t.z, **t.at)
        grads = op.backward(t.dy, t.x, t.w, t.z, want_dbias=True, dx=t.dx, **t.at)
    for counts in ([100, 1, 128], [3, 0, 60], [0, 0, 0]):
        t.at["row_count"].copy_(torch.tensor(counts, dtype=torch.int32))
        g.replay()
        y = torch.full_like(t.y, 7.0)
        z = torch.zeros_like(t.z)
        op.forward(t.x, t.w, t.b, out=y, preact=z, **t.at)
        dx, dw, db = op.backward(t.dy, t.x, t.w, z, want_dbias=True, **t.at)
        for b, n in zip(t.begins, counts):
            assert torch.equal(y[b:b + n], t.y[b:b + n]) and torch.equal(dx[b:b + n], grads[0][b:b + n])
        assert torch.equal(dw, grads[1]) and torch.equal(db, grads[2])
    op.sync()


def test_linear_over_dispatch_standard_moe(layer):
    """The packed layout's own arrays are the segments: each row of the pool
    gets its expert's product, on ragged ranks and with dropped slots."""
    from combine_route_layout_gb300 import EpDispatchCombineConfig, EpDispatchCombineOp
    R, T, H, Er, k, N = 4, 40, 256, 5, 3, 96
    gen = torch.Generator().manual_seed(2)
    idx = torch.stack([torch.randperm(R * Er, generator=gen)[:k] for _ in range(R * T)]).reshape(R, T, k).int()
    idx[torch.rand(idx.shape, generator=gen) < 0.1] = -1
    x = torch.randn((R, T, H), generator=gen).bfloat16().to(DEV)
    disp = EpDispatchCombineOp(EpDispatchCombineConfig(
        torch.bfloat16, R, H, 0, 4, 4, T, Er, k, standard_moe=True))
    v = disp.dispatch_standard_moe(x, torch.ones((R, T, k), device=DEV), None, idx.to(DEV), num_tokens=[40, 0, 17, 39])
    pool = v["packed_recv_x"]
    op = layer.EpLinearOp(layer.EpLinearConfig(R * Er, H, N, pool.shape[0], groups_per_base=Er))
    w = (torch.randn((R * Er, N, H), generator=gen) / 16).bfloat16().to(DEV)
    y = op.forward(pool, w, row_begin=v["expert_offset"], row_count=v["packed_recv_count"], row_base=v["rank_base"])
    disp.sync()
    op.sync()
    seen = 0
    for r in range(R):
        for e in range(Er):
            b, n = int(v["rank_base"][r]) + int(v["expert_offset"][r, e]), int(v["packed_recv_count"][r, e])
            a, ww = pool[b:b + n].double(), w[r * Er + e].double()
            if n:
                ulp_close(y[b:b + n], a @ ww.t(), torch.bfloat16, scale=a.abs() @ ww.abs().t())
            seen += n
    assert seen > 100


def test_errors_are_reported_when_every_call_was_captured(layer):
    from combine_route_layout_gb300 import ep
    router = layer.EpRouterOp(layer.EpRouterConfig(1, 4, 8, 2))
    l = torch.zeros((1, 4, 8), device=DEV)
    linear = layer.EpLinearOp(layer.EpLinearConfig(2, 16, 8, 10))
    x = torch.zeros((10, 16), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((2, 8, 16), dtype=torch.bfloat16, device=DEV)
    count = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    begin = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    router.sync()                                   # nothing ran: nothing to report
    linear.sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        router.forward(l)
        linear.forward(x, w, row_begin=begin, row_count=count)
    router.sync()
    linear.sync()
    g.replay()
    router.sync()
    linear.sync()
    l[0, 2, 3] = math.nan
    count[1] = 6
    g.replay()
    for op, status in ((router, ep.EP_ERR_INVALID_ARG), (linear, ep.EP_ERR_INVALID_INDEX)):
        with pytest.raises(ep.EpError) as ei:
            op.sync()
        assert ei.value.status == status
        op.sync()


# ----------------------------------------------------------- the whole layer

def load_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_moe_layer_example_gradients(layer):
    """The example's outputs and gradients against autograd in 64 bits over the
    same routing, on ragged ranks. Every product rounds its result to bf16, and
    the chain has four of them on the way to w_gate, so 2^-8 times a few of the
    largest gradient bounds the difference: 3 % of it is taken."""
    ex = load_example()
    R, T, H, inner, E_r, k = 2, 24, 64, 48, 3, 2
    m = ex.MoeLayer(R, T, H, inner, E_r, k, 1)
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((R, T, H), generator=gen, device=DEV).bfloat16()
    dy = torch.randn((R, T, H), generator=gen, device=DEV).bfloat16().float()
    ntok = [T, T - 7]
    y, loss = m.forward(x, num_tokens=ntok, balance=True)
    one = torch.ones((), device=DEV)
    dy[1, T - 7:] = 0
    got = m.backward(dy, one)
    m.sync()
    idx = m.saved[4].long()
    xd = x.double().requires_grad_(True)
    ws = [w.double().requires_grad_(True) for w in (m.w_gate, m.w_up, m.w_down)]
    s = torch.sigmoid(xd @ ws[0][0].t())
    valid = torch.arange(T, device=DEV)[None] < torch.tensor(ntok, device=DEV)[:, None]
    held = (idx >= 0) & valid[..., None]
    q = s.gather(-1, idx.clamp(min=0)) * held
    wt = q / q.sum(-1, keepdim=True).clamp(min=1e-30)
    z = torch.einsum("rth,eoh->rteo", xd, ws[1])
    h = torch.nn.functional.silu(z[..., :inner]) * z[..., inner:]
    full = torch.einsum("rtei,ehi->rteh", h, ws[2])
    out = (wt[..., None] * full.gather(2, idx.clamp(min=0)[..., None].expand(-1, -1, -1, H))).sum(2)
    p = s / s.sum(-1, keepdim=True) * valid[..., None]
    n = sum(ntok)
    counts = torch.zeros(R * E_r, device=DEV, dtype=torch.float64).index_add_(0, idx[held], torch.ones(int(held.sum()), device=DEV, dtype=torch.float64))
    bal = 0.01 * (counts * R * E_r / (k * n) * p.sum((0, 1)) / n).sum()
    assert (y.double() - out).abs()[valid].max() < 0.03 * out.abs().max()
    assert abs(float(loss) - float(bal.detach())) < 1e-3 * float(bal.detach())
    refs = torch.autograd.grad((out * dy.double()).sum() + bal, [*ws, xd])
    for g, ref in zip(got, refs):
        ref = ref.detach()
        assert torch.isfinite(g.float()).all()
        sel = valid if g.shape == x.shape else slice(None)
        assert (g.double() - ref)[sel].abs().max() < 0.03 * ref.abs().max()


def test_moe_layer_example_trains(layer):
    losses = load_example().train(steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:]))
