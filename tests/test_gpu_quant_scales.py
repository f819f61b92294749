"""GPU tests of quantised products whose scales' product leaves the range of f32's normal
numbers while the result does not, against 64 bits.

Tolerances. A block's sum is exact in f32; times its two scales, in an order that
leaves the range only where the result does, it is rounded three times (2^-24 each) and
added up in f32: for `terms` blocks at most (terms + 3) * 2^-24 of the sum of magnitudes.
Each of these steps may end below f32's smallest normal number, where it is off by half of
2^-149, and the largest f32 and beyond are not asked for. The activation adds 2^-20 of the
value, bf16 2^-8 (half of 2^-133 below its normal numbers)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def blocks(n):
    return -(-n // 128)


def codes(g, *shape):
    """Codes of every size, those of a few blocks zeros."""
    c = torch.randn(shape, generator=g, device=DEV) * 60
    c[..., :128] *= (torch.rand(shape[:-1], generator=g, device=DEV) < 0.7)[..., None]
    return c.to(E4M3)


def scales(g, exponent, *shape):
    """Significands of 24 bits, exponents around `exponent`."""
    e = exponent + torch.randint(-3, 4, shape, generator=g, device=DEV)
    return torch.ldexp(1 + torch.rand(shape, generator=g, device=DEV), e)


def within(got, want, tol, most, what):
    """Where the result, within its bound, is below `most`."""
    there = (want.abs() + tol) < most
    assert there.double().mean() > 0.9, what
    got = got.double()
    assert torch.isfinite(got[there]).all(), what
    off = ((got - want).abs() - tol)[there]
    assert (off <= 0).all(), f"{what}: {float(off.max())} over the bound"


# exponents of the scales of x's even rows (the odd ones have ordinary scales) and of W's
EXTREMES = [(-100, -40), (-30, -115), (-132, -10), (100, 20), (60, 60), (-145, 20), (20, -146)]


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("rows,k,n,groups", [(1, 400, 40, 1), (8, 1024, 136, 1), (200, 640, 333, 1), (300, 512, 256, 1), (70, 4096, 128, 1),
                                             (90, 272, 160, 3)])
@pytest.mark.parametrize("ex,ew", EXTREMES)
def test_forward(layer, ex, ew, rows, k, n, groups, act, out):
    g = torch.Generator(device=DEV).manual_seed(rows + k + n)
    parts = 2 if act == "swiglu" else 1
    x, w = codes(g, rows, k), codes(g, groups, parts * n, k)
    xs, ws = scales(g, ex, rows, blocks(k)), scales(g, ew, groups, parts * blocks(n), blocks(k))
    if ex + ew > 0 or act == "swiglu":
        # small sums for scales of a large product; gates that leave their up values alone
        x, w = (x.float() / 4096).to(E4M3), (w.float() / 4096).to(E4M3)
    if act == "swiglu":
        w[:, :n] = torch.ones((), device=DEV).to(E4M3)
    xs[1::2] = scales(g, 0, *xs[1::2].shape)
    each = rows // groups
    begin = torch.arange(groups, device=DEV, dtype=torch.int32) * each
    count = torch.full((groups,), each, device=DEV, dtype=torch.int32)
    at = {} if groups == 1 else dict(row_begin=begin, row_count=count)
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(groups, k, n, rows, out_dtype=out, activation=act))
    z = torch.zeros((rows, parts * n), dtype=BF16, device=DEV)
    y = op.forward(x, xs, w, ws, preact=z, **at)
    x64 = x.double() * xs.double().repeat_interleave(128, -1)[:, :k]
    row = torch.arange(parts * n, device=DEV)
    w64 = w.double() * ws.double()[:, row // n * blocks(n) + row % n // 128].repeat_interleave(128, -1)[..., :k]
    x64, kb = x64.view(groups, each, k), blocks(k)
    want_z = (x64 @ w64.transpose(1, 2)).view(rows, parts * n)
    mag = (x64.abs() @ w64.abs().transpose(1, 2)).view(rows, parts * n)
    tol_z = (kb + 3) * 2.0 ** -24 * mag + 3 * kb * 2.0 ** -150
    most = torch.finfo(BF16).max
    within(z, want_z, tol_z + 2.0 ** -8 * (want_z.abs() + tol_z) + 2.0 ** -134, most, "z")
    if act == "none":
        tol = tol_z + (2.0 ** -8 * (want_z.abs() + tol_z) + 2.0 ** -134 if out == BF16 else 0)
        within(y, want_z, tol, most, "y")
    op.sync()


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("rows,k,n", [(40, 256, 300), (300, 1040, 128)])
@pytest.mark.parametrize("ed,ew", [(-95, -40), (-20, -118), (90, 30)])
def test_input_gradient(layer, ed, ew, rows, k, n, act):
    """dx of gradients and weights whose scales' product is too small or too large."""
    g = torch.Generator(device=DEV).manual_seed(rows + n)
    x, xs = codes(g, rows, k), scales(g, 0, rows, blocks(k))
    w, ws = codes(g, 1, n, k), scales(g, ew, 1, blocks(n), blocks(k))
    if ew > 20:
        w = (w.float() / 4096).to(E4M3)
    # codes of whole numbers up to 448: quantising them again changes nothing
    q = torch.randint(-8, 9, (rows, n), generator=g, device=DEV).double()
    q[:, ::64] = 448.0
    dy = (q * 2.0 ** ed).float()
    dy[1::2] = q[1::2].float()
    z = torch.ones((rows, n), dtype=BF16, device=DEV)
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(1, k, n, rows, out_dtype=F32, activation=act), backward=True)
    dx, _, _ = op.backward(dy, x, xs, w, ws, preact=z, want_dweight=False)
    row, d = torch.arange(n, device=DEV), dy.double()
    w64 = (w.double() * ws.double()[:, row // 128].repeat_interleave(128, -1)[..., :k])[0]
    want, mag = d @ w64, d.abs() @ w64.abs()
    tol = (blocks(n) + 3) * 2.0 ** -24 * mag + 3 * blocks(n) * 2.0 ** -150
    within(dx, want, tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -134, torch.finfo(BF16).max, "dx")
    op.sync()


@pytest.mark.parametrize("rows", [3, 150])
def test_blocks_of_zeros_are_zeros_whatever_their_scales(layer, rows):
    g = torch.Generator(device=DEV).manual_seed(1)
    k, n = 512, 256
    x, w = codes(g, rows, k), codes(g, 1, n, k)
    x[:, 128:256] = 0
    xs, ws = scales(g, 0, rows, 4), scales(g, 0, 1, 2, 4)
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(1, k, n, rows, out_dtype=F32))
    want = op.forward(x, xs, w, ws)
    xs[:, 1], ws[..., 1] = 3e38, 3e38
    assert torch.equal(op.forward(x, xs, w, ws), want)
    xs[:, 1] = 0
    assert torch.equal(op.forward(x, xs, w, ws), want)
    op.sync()
