"""GPU tests of the quantised products with NaN and infinity inside rows, weights, scales and
gradients: what they reach is not finite, and everything else is bit for bit what it is
without them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def blocks(n):
    return -(-n // 128)


class Case:
    """A product of rows of a pool; dense, or segments of `each` rows with rows of nobody between them."""

    def __init__(self, layer, rows, k, n, groups, act, out=F32, backward=False):
        g = torch.Generator(device=DEV).manual_seed(rows + k)
        rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.k, self.n, self.parts, self.groups = k, n, 2 if act == "swiglu" else 1, groups
        self.each = rows // groups
        gap = 0 if groups == 1 else 3
        self.pool = rows + gap * groups
        begin = [i * (self.each + gap) for i in range(groups)]
        t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        self.at = {} if groups == 1 else dict(row_begin=t(begin), row_count=t([self.each] * groups))
        self.held = torch.zeros(self.pool, dtype=torch.bool, device=DEV)
        for b in begin:
            self.held[b:b + self.each] = True
        self.row = begin[-1] + self.each // 2                  # a row of the last group
        self.x, self.w = rand(self.pool, k).to(E4M3), rand(groups, self.parts * n, k).to(E4M3)
        self.xs = torch.rand((self.pool, blocks(k)), generator=g, device=DEV) + 0.5
        self.ws = torch.rand((groups, self.parts * blocks(n), blocks(k)), generator=g, device=DEV) + 0.5
        self.ws /= k
        self.b = rand(groups, self.parts * n)
        self.z = rand(self.pool, self.parts * n).bfloat16()
        self.dy = rand(self.pool, n).to(out)
        self.act = act
        self.op = layer.EpQuantLinearOp(layer.EpLinearConfig(groups, k, n, self.pool, out_dtype=out, activation=act, weight_grad_dtype=F32),
                                        backward=backward)

    def forward(self, **new):
        a = {"x": self.x, "xs": self.xs, "w": self.w, "ws": self.ws} | new
        out = torch.zeros((self.pool, self.n), device=DEV)
        return self.op.forward(a["x"], a["xs"], a["w"], a["ws"], bias=self.b, out=out, **self.at)

    def backward(self, **new):
        a = {"x": self.x, "xs": self.xs, "dy": self.dy, "z": self.z, "w": self.w, "ws": self.ws} | new
        dx = torch.zeros((self.pool, self.k), dtype=BF16, device=DEV)
        return self.op.backward(a["dy"], a["x"], a["xs"], a["w"], a["ws"], preact=None if self.act == "none" else a["z"], want_dbias=True,
                                dx=dx, **self.at)


def with_code(t, *at):
    t = t.clone()
    t.view(torch.uint8)[at] = NAN_CODE
    return t


def with_value(t, value, *at):
    t = t.clone()
    t[at] = value
    return t


def only(got, clean, reached, what):
    """`reached` is not finite, the rest is as it was."""
    bad = ~torch.isfinite(got)
    assert (bad == reached).all(), f"{what}: {int((bad != reached).sum())} places"
    assert torch.equal(got[~reached], clean[~reached]), what


SHAPES = [(3, 400, 40, 1), (200, 640, 333, 1), (300, 512, 256, 1), (70, 4096, 128, 1), (90, 272, 160, 3), (900, 384, 320, 3)]


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("rows,k,n,groups", SHAPES)
def test_forward(layer, rows, k, n, groups, act):
    c = Case(layer, rows, k, n, groups, act)
    clean = c.forward()
    assert torch.isfinite(clean).all()
    row = torch.zeros_like(clean, dtype=torch.bool)
    row[c.row] = True
    for at in (0, k // 2, k - 1):
        only(c.forward(x=with_code(c.x, c.row, at)), clean, row, "a code of x")
    for block in (0, blocks(k) - 1):
        only(c.forward(xs=with_value(c.xs, float("nan"), c.row, block)), clean, row, "a scale of x")
    if c.row:
        nobody = with_code(c.x, ~c.held)
        only(c.forward(x=nobody, xs=with_value(c.xs, float("nan"), ~c.held)), clean, torch.zeros_like(row), "rows of nobody")
    group = torch.zeros_like(row)
    group[c.row - c.each // 2:c.row - c.each // 2 + c.each] = True
    feature = n - 1
    for part in range(c.parts):
        reached = torch.zeros_like(row)
        reached[:, feature] = True
        only(c.forward(w=with_code(c.w, groups - 1, part * n + feature, k - 1)), clean, group & reached, "a code of W")
        block = blocks(n) - 1
        reached[:, block * 128:] = True
        ws = with_value(c.ws, float("nan"), groups - 1, part * blocks(n) + block, 0)
        only(c.forward(ws=ws), clean, group & reached, "a scale of W")
    c.op.sync()


@pytest.mark.parametrize("rows", [2, 130])
def test_a_row_quantised_with_an_infinity(layer, rows):
    """Its block's scale is infinity and stands for NaN: the row's results are, and no others."""
    k, n = 384, 200
    c = Case(layer, rows, k, n, 1, "silu")
    quant = layer.EpQuantOp(layer.EpQuantConfig(1, k, rows, dtype=F32))
    x = torch.randn((rows, k), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    q, s = quant.quantize(x)
    clean = c.forward(x=q, xs=s)
    for value in (float("inf"), -float("inf"), float("nan")):
        q, s = quant.quantize(with_value(x, value, 1, 200))
        got = c.forward(x=q, xs=s)
        assert got[1].isnan().all()
        keep = [i for i in range(rows) if i != 1]
        assert torch.equal(got[keep], clean[keep])
    c.op.sync()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("act,out", [("none", BF16), ("none", F32), ("relu", BF16), ("swiglu", BF16), ("silu", F32)])
@pytest.mark.parametrize("rows,k,n,groups", SHAPES)
def test_backward(layer, rows, k, n, groups, act, out, value):
    """A NaN or infinity in dy reaches its row of dx, and its feature's rows of dW and its db."""
    c = Case(layer, rows, k, n, groups, act, out, backward=True)
    # ReLU's slope of 0 times infinity is no number either, so that the place does not matter
    c.z[c.row] = 1.0
    clean = c.backward()
    assert all(torch.isfinite(t).all() for t in clean)
    feature, last = n // 2, groups - 1
    dx, dw, db = c.backward(dy=with_value(c.dy, value, c.row, feature))
    row = torch.zeros_like(dx, dtype=torch.bool)
    row[c.row] = True
    only(dx, clean[0], row, "dx")
    reached, of_db = torch.zeros_like(dw, dtype=torch.bool), torch.zeros_like(db, dtype=torch.bool)
    for part in range(c.parts):
        reached[last, part * n + feature] = True
        of_db[last, part * n + feature] = True
    only(dw, clean[1], reached, "dW")
    only(db, clean[2], of_db, "db")
    # a code of x reaches its column of dW alone
    dx, dw, db = c.backward(x=with_code(c.x, c.row, k - 1))
    reached = torch.zeros_like(reached)
    reached[last, :, k - 1] = True
    only(dx, clean[0], torch.zeros_like(row), "dx")
    only(dw, clean[1], reached, "dW")
    only(db, clean[2], torch.zeros_like(of_db), "db")
    c.op.sync()
