"""GPU tests of the norms around a block against 64 bits: odd sizes, one row and
many, every gate, each type, quantised results, and the gradients, against the
formulas and against differences.

Tolerances. A row's sums have H positive (or mixed) f32 terms: off by at most
H * 2^-23 of the sum of magnitudes, usually far less; the square root, the division
and the products behind them add 2^-22 each. bf16 results have one rounding more,
2^-8 of the value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def normal(seed, *shape, dtype=torch.float32, scale=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(shape, device=DEV).normal_(generator=g)
    if scale:   # rows of different magnitudes
        x = x * torch.exp(1.5 * torch.empty((shape[0], 1), device=DEV).normal_(generator=g))
    return x.to(dtype)


class Case:
    def __init__(self, layer, rows, h, post=False, gate="none", alpha=1.0, stream=BF16, block=BF16, quant=False, has_block=True, eps=1e-5,
                 spare=0, backward=False):
        self.rows, self.h, self.post, self.gate_kind, self.alpha, self.eps = rows, h, post and has_block, gate, alpha, eps
        self.op = layer.EpNormOp(layer.EpNormConfig(h, rows + spare, eps=eps, post_norm=post, gate=gate, residual_scale=alpha, stream_dtype=stream,
                                                    block_dtype=block, quant_type="fp8_e4m3_block128" if quant else "none"), backward=backward)
        self.x = normal(1, rows, h, dtype=stream, scale=True)
        self.w = 1 + 0.3 * normal(2, h)
        self.y = normal(3, rows, h, dtype=block, scale=True) if has_block else None
        self.wp = 1 + 0.3 * normal(4, h) if self.post else None
        self.g = None if gate == "none" or not has_block else normal(5, rows if gate == "token" else h)

    def args(self):
        return dict(block=self.y, weight_post=self.wp, gate=self.g)

    def gate64(self, g):
        return 1.0 if g is None else g[:, None] if self.gate_kind == "token" else g

    def forward64(self, x, w, y=None, wp=None, g=None):
        """(stream, out, rms, rms of the block)"""
        root = lambda v: (v.square().mean(-1, keepdim=True) + self.eps).rsqrt()  # noqa: E731
        ry = torch.ones_like(x[:, :1])
        s = x
        if y is not None:
            u = y
            if self.post:
                ry = root(y)
                u = y * ry * wp
            s = x + self.alpha * self.gate64(g) * u
        return s, s * root(s) * w, root(s), ry

    def leaves64(self):
        return {n: t.double().requires_grad_() for n, t in (("x", self.x), ("w", self.w), ("y", self.y), ("wp", self.wp), ("g", self.g)) if t is not None}


def within(got, want, bound, what):
    assert got.shape == want.shape, what
    off = (got.double() - want).abs() - bound
    assert torch.isfinite(got.double()).all() and (off <= 0).all(), f"{what}: {float(off.max())} over the bound"


def rounding(dtype):
    return 2.0 ** -8 if dtype == BF16 else 2.0 ** -24


def check_codes(codes, scales, want, bound):
    """Codes and scales of values that are within `bound` of `want`."""
    n = want.shape[-1]
    pad = lambda t: torch.nn.functional.pad(t, (0, -n % 128)).unflatten(-1, (-1, 128))  # noqa: E731
    cut = lambda t: t.flatten(-2)[:, :n]  # noqa: E731
    amax, most = pad(want).abs().amax(-1, keepdim=True), pad(bound).amax(-1, keepdim=True)
    assert ((scales.double()[..., None] - amax / 448).abs() <= most / 448 + 2.0 ** -23 * amax / 448).all()
    # half a step of the code, whose values go up to 448 (a step of 32), around a value that is off by `bound`
    value = pad(codes.double()) * scales.double()[..., None]
    step = torch.exp2(torch.floor(torch.log2((pad(want).abs() / scales.double()[..., None].clamp(min=1e-30)).clamp(min=2.0 ** -6))) - 3.0)
    assert ((cut(value) - want).abs() <= cut(step * 0.51 * scales.double()[..., None] + 2 * most)).all()


@pytest.mark.parametrize("stream,block", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("post,gate,alpha", [(False, "none", 1.0), (True, "none", 0.5), (False, "token", 0.22), (True, "token", 1.0),
                                             (False, "feature", 1.0), (True, "feature", 0.5)])
@pytest.mark.parametrize("rows,h", [(1, 8), (3, 136), (5, 1000), (2, 7168), (700, 256), (401, 2056), (330, 16384), (1, 16384)])
def test_forward(layer, rows, h, post, gate, alpha, stream, block):
    for quant in (False, True):
        c = Case(layer, rows, h, post, gate, alpha, stream, block, quant, spare=2)
        s, out, scales, stats = c.op.forward(c.x, c.w, **c.args())
        want = c.forward64(*(None if t is None else t.double() for t in (c.x, c.w, c.y, c.wp, c.g)))
        sums = h * 2.0 ** -23
        size = c.x.double().abs() + (want[0] - c.x.double()).abs()
        tol_s = (sums if post else 0) * size + 2.0 ** -21 * size
        within(s, want[0], tol_s + rounding(stream) * (want[0].abs() + tol_s), "stream")
        # the root's relative error: half of the sum's, and the errors of the stream's terms
        tol_r = sums + 2.0 ** -21 + (tol_s / size.clamp(min=1e-30)).amax(-1, keepdim=True) * 4
        within(stats[:, :1], want[2], tol_r * want[2], "rms")
        within(stats[:, 1:], want[3], (sums + 2.0 ** -21) * want[3], "rms of the block")
        tol = tol_s * (want[2] * c.w.double()).abs() + (tol_r + 2.0 ** -21) * want[1].abs()
        if quant:
            assert out.dtype == E4M3 and scales.shape == (rows, -(-h // 128))
            check_codes(out, scales, want[1], tol)
        else:
            assert scales is None
            within(out, want[1], tol + 2.0 ** -8 * (want[1].abs() + tol), "out")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("rows,h", [(1, 128), (7, 7168), (600, 520)])
def test_first_norm_has_no_block(layer, rows, h, quant):
    c = Case(layer, rows, h, post=True, gate="token", has_block=False, quant=quant, backward=True)
    c.wp = c.g = None
    s, out, scales, stats = c.op.forward(c.x, c.w)
    assert s is c.x and (stats[:, 1] == 1).all()
    leaves = {n: t.double().requires_grad_() for n, t in (("x", c.x), ("w", c.w))}
    want = c.forward64(leaves["x"], leaves["w"])[1]
    tol = (h * 2.0 ** -23 + 2.0 ** -20) * want.detach().abs()
    if quant:
        check_codes(out, scales, want.detach(), tol)
    else:
        within(out, want.detach(), tol + 2.0 ** -8 * want.detach().abs(), "out")
    d = normal(9, rows, h, dtype=BF16)
    want.backward(d.double())
    got = c.op.backward(d, s, c.w, stats)
    assert got[1] is None and got[3] is None and got[4] is None
    size = leaves["x"].grad.abs() + (d.double() * c.w.double() * stats[:, :1].double()).abs()
    size = size + size.mean(-1, keepdim=True) * 4
    tol = (h * 2.0 ** -23 + 2.0 ** -19) * size
    within(got[0], leaves["x"].grad, tol + 2.0 ** -8 * (leaves["x"].grad.abs() + tol), "d_residual")
    terms = (d.double() * c.x.double() * stats[:, :1].double()).abs().sum(0)
    within(got[2], leaves["w"].grad, (rows * 2.0 ** -23 + h * 2.0 ** -24 + 2.0 ** -20) * terms, "d_weight")


@pytest.mark.parametrize("stream,block", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("post,gate,alpha", [(False, "none", 1.0), (True, "none", 0.5), (False, "token", 0.22), (True, "token", 1.0),
                                             (False, "feature", 1.0), (True, "feature", 0.5)])
@pytest.mark.parametrize("rows,h,with_stream", [(1, 8, True), (3, 136, False), (5, 1000, True), (2, 7168, True), (700, 256, True),
                                                (401, 2056, False), (320, 16384, True)])
def test_backward(layer, rows, h, with_stream, post, gate, alpha, stream, block):
    """Against the formulas in 64 bits, from the same stored stream and stats: each result's
    error is its terms' f32 steps and a rounding."""
    c = Case(layer, rows, h, post, gate, alpha, stream, block, backward=True)
    s = normal(6, rows, h, dtype=stream, scale=True)
    stats = torch.stack([1.0 / (t.double().square().mean(-1) + c.eps).sqrt() for t in (s, c.y)], -1).float()
    if not post:
        stats[:, 1] = 1
    d = normal(7, rows, h, dtype=BF16)
    ds = normal(8, rows, h, dtype=stream) if with_stream else None
    got = c.op.backward(d, s, c.w, stats, d_stream=ds, **c.args())
    r, ry = stats[:, :1].double(), stats[:, 1:].double()
    n, v = s.double() * r, d.double() * c.w.double()
    mean = (v * n).mean(-1, keepdim=True)
    t0 = torch.zeros_like(n) if ds is None else ds.double()
    t = t0 + r * (v - n * mean)
    size = t0.abs() + r * (v.abs() + n.abs() * (v * n).abs().mean(-1, keepdim=True))
    steps = h * 2.0 ** -23 + 2.0 ** -20
    tol_t = steps * size
    within(got[0], t, tol_t + rounding(stream) * (t.abs() + tol_t), "d_residual")
    y = c.y.double()
    n_y = y * ry
    wp = c.wp.double() if post else 1.0
    gate64 = c.gate64(None if c.g is None else c.g.double())
    du = alpha * gate64 * t
    tol_du = (alpha * gate64 * torch.ones_like(t)).abs() * (tol_t + 2.0 ** -22 * t.abs())
    if post:
        e = du * wp
        want = ry * (e - n_y * (e * n_y).mean(-1, keepdim=True))
        tol_e = tol_du * wp.abs()
        tol = ry * (tol_e + n_y.abs() * (tol_e * n_y.abs()).mean(-1, keepdim=True)) + \
            steps * ry * (e.abs() + n_y.abs() * (e * n_y).abs().mean(-1, keepdim=True))
    else:
        want, tol = du, tol_du
    within(got[1], want, tol + rounding(block) * (want.abs() + tol), "d_block")
    rows_steps = rows * 2.0 ** -23 + 2.0 ** -21
    within(got[2], (d.double() * n).sum(0), rows_steps * (d.double() * n).abs().sum(0), "d_weight")
    if post:
        within(got[3], (du * n_y).sum(0), rows_steps * (du * n_y).abs().sum(0) + (tol_du * n_y.abs()).sum(0), "d_weight_post")
    else:
        assert got[3] is None
    u = n_y * wp
    if gate == "none":
        assert got[4] is None
    else:
        over = -1 if gate == "token" else 0
        count = h if gate == "token" else rows
        want = alpha * (u * t).sum(over)
        within(got[4], want, alpha * ((count * 2.0 ** -23 + 2.0 ** -20) * (u * t).abs() + u.abs() * tol_t).sum(over), "d_gate")


def test_gradients_are_those_of_the_forward_pass(layer):
    """Autograd through the 64-bit forward pass, and differences of the kernel's own."""
    for post in (False, True):
        for gate in ("token", "feature"):
            c = Case(layer, 33, 264, post, gate, 0.7, F32, F32, backward=True)
            s, out, _, stats = c.op.forward(c.x, c.w, **c.args())
            leaves = c.leaves64()
            stream64, out64 = c.forward64(**leaves)[:2]
            d, ds = normal(20, 33, 264, dtype=BF16), normal(21, 33, 264)
            (stream64 * ds.double()).sum().add((out64 * d.double()).sum()).backward()
            got = c.op.backward(d, s, c.w, stats, d_stream=ds, **c.args())
            for name, g in zip(("x", "y", "w", "wp", "g"), got):
                if name in leaves:
                    want = leaves[name].grad
                    top = float(want.abs().max())
                    # 264 columns, 33 rows: sums of at most that many terms of the largest one's size
                    within(g, want, torch.full_like(want, 300 * 2.0 ** -22 * top) + 2.0 ** -18 * want.abs(), name)
            # a difference along a direction: bf16 outputs are averaged over all of them
            way = normal(22, 33, 264)
            step = 2.0 ** -6
            loss = []
            for sign in (1, -1):
                s2, o2, _, _ = c.op.forward(c.x + sign * step * way, c.w, **c.args())
                loss.append(float((s2.double() * ds.double()).sum() + (o2.double() * d.double()).sum()))
            slope = (loss[0] - loss[1]) / (2 * step)
            want = float((got[0].double() * way.double()).sum())
            # roundings of out: 2^-8 of each of 8712 terms at random, over the step; curvature step^2
            noise = 2.0 ** -8 * float((out.double() * d.double()).square().sum().sqrt()) * 4 / (2 * step)
            assert abs(slope - want) <= noise + 0.02 * float((got[0].double() * way.double()).abs().sum()) * step


def test_in_place_and_given_tensors(layer):
    c = Case(layer, 50, 640, True, "feature", 0.5, F32, BF16, quant=True, backward=True)
    want = c.op.forward(c.x, c.w, **c.args())
    x = c.x.clone()
    out, scales, stats = torch.zeros((50, 640), device=DEV).to(E4M3), torch.zeros((50, 5), device=DEV), torch.zeros((50, 2), device=DEV)
    got = c.op.forward(x, c.w, stream=x, out=out, scales=scales, stats=stats, **c.args())
    assert got[0] is x and got[1] is out and got[2] is scales and got[3] is stats
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    d, ds = normal(7, 50, 640, dtype=BF16), normal(8, 50, 640)
    want = c.op.backward(d, x, c.w, stats, d_stream=ds, **c.args())
    got = c.op.backward(d, x, c.w, stats, d_stream=ds, d_residual=ds, **c.args())
    assert got[0] is ds
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    c.op.sync()


def test_no_rows_and_special_rows(layer):
    c = Case(layer, 4, 256, True, "feature", backward=True)
    none = c.x[:0]
    s, out, _, stats = c.op.forward(none, c.w, block=c.y[:0], weight_post=c.wp, gate=c.g)
    got = c.op.backward(out, s, c.w, stats, block=c.y[:0], weight_post=c.wp, gate=c.g)
    assert s.shape == (0, 256) and got[0].shape == (0, 256) and (got[2] == 0).all() and (got[3] == 0).all() and (got[4] == 0).all()
    for quant in (False, True):
        c = Case(layer, 4, 256, quant=quant)
        x, y = c.x.float(), c.y.float()
        x[0], y[0] = 0, 0                               # nothing: rms = 1 / sqrt(eps), out 0
        x[1, 3] = float("nan")                          # stays in its row
        x[2], y[2] = 0, 1e-30
        c.x, c.y = x.bfloat16(), y.bfloat16()
        s, out, scales, stats = c.op.forward(c.x, c.w, block=c.y)
        v = out.float() if not quant else out.float() * scales.repeat_interleave(128, -1)
        assert (v[0] == 0).all() and abs(float(stats[0, 0]) - c.eps ** -0.5) <= 2.0 ** -21 * c.eps ** -0.5
        assert v[1].isnan().all() and v[2:].isfinite().all()


def test_runs_are_the_same(layer):
    c = Case(layer, 2049, 1160, True, "feature", backward=True)
    s, _, _, stats = c.op.forward(c.x, c.w, **c.args())
    d = normal(7, 2049, 1160, dtype=BF16)
    first = c.op.backward(d, s, c.w, stats, **c.args())
    for _ in range(3):
        for a, b in zip(first, c.op.backward(d, s, c.w, stats, **c.args())):
            assert torch.equal(a, b)


def test_graph_and_other_stream(layer):
    """A captured forward and backward pass follow new inputs; a second stream orders by events."""
    c = Case(layer, 90, 512, True, "token", 0.5, BF16, F32, backward=True)
    d = normal(7, 90, 512, dtype=BF16)

    def both():
        s, out, _, stats = c.op.forward(c.x, c.w, **c.args())
        return (s, out, stats) + tuple(c.op.backward(d, s, c.w, stats, **c.args()))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = both()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (30, 40):
        c.x.copy_(normal(seed, 90, 512))
        c.y.copy_(normal(seed + 1, 90, 512))
        d.copy_(normal(seed + 2, 90, 512))
        graph.replay()
        got = [t.clone() for t in held]
        for a, b in zip(got, both()):
            assert torch.equal(a, b)
    c.op.sync()
