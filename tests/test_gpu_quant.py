"""GPU tests of block quantisation and of the products of block-quantised operands
against plain 64-bit implementations, at the sizes and segments where they can go
wrong.

Tolerances. Codes and scales are f32 steps rounded to nearest even: equal bit for
bit. Products: the terms of a block's sum are exact in f32, and a sum of n f32
terms, in any order and with steps that round or cut off, is off by at most
n * 2^-23 of the sum of magnitudes, scales and the sums over blocks (a few
roundings a block) included. exp and division add 2^-21 of the value. bf16 results
have one rounding more, 2^-8 of the value. dx is made of codes of dz: where dz
carries an activation's slope, its f32 value is off by 2^-20, so that a quotient
that close to the middle between two codes may take either; the bound adds a
code's step for each such term. dW's operands are bf16: 2^-8 for each of the two.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(seed, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, device=DEV).normal_(0.0, std, generator=rng(seed)).to(dtype)


def blocks(n):
    return -(-n // 128)


def bits(t):
    return t.view(torch.uint8).cpu()


# ----------------------------------------------------------------- quantiser

def plain_codes(x, each):
    """(codes as bytes, scales) of [..., M, K] in f32 steps that numpy rounds by IEEE rules."""
    v = x.float().cpu().numpy()
    M, K = v.shape[-2:]
    codes = np.zeros(v.shape, np.uint8)
    scales = np.zeros(v.shape[:-2] + (-(-M // each), blocks(K)), np.float32)
    with np.errstate(all="ignore"):
        for at in np.ndindex(scales.shape):
            lead, i, b = at[:-2], at[-2], at[-1]
            cut = lead + (slice(i * each, (i + 1) * each), slice(b * 128, (b + 1) * 128))
            part = v[cut]
            amax = np.float32(np.max(np.where(np.isnan(part), np.float32(0), np.abs(part))))
            scale = np.float32(amax / np.float32(448))
            scales[at] = scale
            q = part / scale if scale > 0 else part * np.float32(0)
            q = np.where(np.isnan(q), q, np.clip(q, -448, 448)).astype(np.float32)
            codes[cut] = torch.from_numpy(np.ascontiguousarray(q)).to(E4M3).view(torch.uint8).numpy()
    return torch.from_numpy(codes), torch.from_numpy(scales)


def same_codes(got, want):
    got, want = bits(got), want.view(torch.uint8)
    nan = (want & 0x7F) == 0x7F
    assert (((got & 0x7F) == 0x7F) == nan).all()
    assert torch.equal(got[~nan], want[~nan])


def hard_rows(rows, k, dtype, seed):
    """Rows with what goes wrong: zeros, signed zeros, tiny and large magnitudes, ties, infinity, NaN."""
    x = normal(seed, rows, k) * torch.exp(2.0 * normal(seed + 1, rows, 1))
    kinds = [lambda r: r.zero_(), lambda r: r.fill_(-0.0), lambda r: r.mul_(1e-36), lambda r: r.mul_(1e36),
             lambda r: r.copy_(torch.arange(k, device=DEV) % 449 / 16.0), lambda r: r[k // 2:k // 2 + 1].fill_(float("inf")),
             lambda r: r[-1:].fill_(float("nan")), lambda r: r.mul_(1e-44), lambda r: r[:1].fill_(3e38)]
    for i in range(rows):
        if i % 3 == 1:
            kinds[(i // 3) % len(kinds)](x[i])
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 16), (40, 16), (3, 128), (29, 144), (1, 7168), (65, 1008), (300, 2048), (2, 40000)])
def test_rows(layer, rows, k, dtype):
    op = layer.EpQuantOp(layer.EpQuantConfig(1, k, rows + 3, dtype=dtype))
    x = hard_rows(rows, k, dtype, rows + k)
    codes, scales = op.quantize(x)
    want, want_scales = plain_codes(x, 1)
    assert codes.dtype == E4M3 and scales.shape == (rows, blocks(k))
    assert torch.equal(scales.cpu().view(torch.int32), want_scales.view(torch.int32))
    # a block with an infinity stands for NaN whatever its codes
    fine = torch.isfinite(want_scales).repeat_interleave(128, -1)[:, :k]
    same_codes(codes.view(torch.uint8).cpu().masked_fill(~fine, 0), want.masked_fill(~fine, 0))
    back = op.dequantize(codes, scales)
    value = codes.float() * scales.repeat_interleave(128, -1)[:, :k]
    assert torch.equal(back.isnan(), value.isnan())
    assert torch.equal(back.nan_to_num(), value.to(dtype).nan_to_num())
    assert back.isnan().cpu()[~fine].all()
    op.sync()


@pytest.mark.parametrize("base", [False, True])
@pytest.mark.parametrize("k", [16, 272, 2048])
def test_segments_of_rows(layer, k, base):
    """Empty, tight and padded segments in any order; rows of nobody are not read and stay as they are."""
    counts, begins = [5, 0, 130, 1, 64, 300], [700, 3, 0, 130, 131, 200]
    pool, G = 720, 6
    per = 2 if base else 0
    bases = [-20, 0, 10] if base else [0, 0, 0]
    op = layer.EpQuantOp(layer.EpQuantConfig(G, k, pool, groups_per_base=per))
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    begin = [b - (bases[i // 2] if base else 0) for i, b in enumerate(begins)]
    held = torch.zeros(pool, dtype=torch.bool)
    for b, n in zip(begins, counts):
        held[b:b + n] = True
    x = normal(k, pool, k, dtype=torch.bfloat16)
    x[~held.to(DEV)] = float("nan")
    codes = torch.full((pool, k), 0x55, dtype=torch.uint8, device=DEV).view(E4M3)
    scales = torch.full((pool, blocks(k)), -7.0, device=DEV)
    op.quantize(x, row_begin=t(begin), row_count=t(counts), row_base=t(bases) if base else None, codes=codes, scales=scales)
    want, want_scales = plain_codes(x[held.to(DEV)], 1)
    assert torch.equal(bits(codes)[held], want)
    assert torch.equal(scales.cpu()[held], want_scales)
    assert (bits(codes)[~held] == 0x55).all() and (scales.cpu()[~held] == -7.0).all()
    out = torch.full((pool, k), -3.0, dtype=torch.bfloat16, device=DEV)
    op.dequantize(codes, scales, row_begin=t(begin), row_count=t(counts), row_base=t(bases) if base else None, out=out)
    value = (codes.float() * scales.repeat_interleave(128, -1)[:, :k]).bfloat16()
    assert torch.equal(out.cpu()[held], value.cpu()[held]) and (out.cpu()[~held] == -3.0).all()
    op.sync()


def test_segments_outside_the_pool_are_reported(layer):
    from combine_route_layout_gb300 import EpError
    op = layer.EpQuantOp(layer.EpQuantConfig(3, 64, 100))
    x = normal(1, 100, 64, dtype=torch.bfloat16)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    codes, scales = op.quantize(x, row_begin=t([90, -5, 10]), row_count=t([30, 3, 5]))
    want, _ = plain_codes(x, 1)
    assert torch.equal(bits(codes)[90:], want[90:]) and torch.equal(bits(codes)[10:15], want[10:15])
    with pytest.raises(EpError) as ei:
        op.sync()
    assert ei.value.status == -4
    op.sync()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g,n,k", [(1, 1, 16), (3, 127, 400), (2, 128, 128), (1, 300, 1040), (5, 129, 144)])
def test_matrices(layer, g, n, k, dtype):
    op = layer.EpQuantOp(layer.EpQuantConfig(g, k, n, block_rows=128, dtype=dtype))
    x = torch.stack([hard_rows(n, k, dtype, 7 * i + n) for i in range(g)])
    x = x.nan_to_num(nan=0.5, posinf=2.0)
    codes, scales = op.quantize(x)
    want, want_scales = plain_codes(x, 128)
    assert torch.equal(scales.cpu(), want_scales)
    same_codes(codes, want)
    each = scales.repeat_interleave(128, -1)[..., :k].repeat_interleave(128, -2)[:, :n]
    assert torch.equal(op.dequantize(codes, scales), (codes.float() * each).to(dtype))
    op.sync()


# ------------------------------------------------------------------ products

class Case:
    """Operands of a product, in 64 bits too."""

    def __init__(self, layer, counts, k, n, act="none", pad=128, out=torch.bfloat16, base=0, seed=0, backward=False, dense=False,
                 weight_grad=torch.bfloat16):
        self.counts, self.k, self.n, self.act, self.out, self.G = counts, k, n, act, out, len(counts)
        parts = 2 if act == "swiglu" else 1
        self.parts, self.nw, self.nb, self.kb = parts, parts * n, blocks(n), blocks(k)
        begins, at = [], 0
        for c in counts:
            begins.append(at)
            at += -(-c // pad) * pad if pad else c
        self.pool = max(1, at) + (0 if dense else 5)
        if dense:
            self.pool = counts[0]
        self.begins, self.dense = begins, dense
        shift = [7 * (i // base + 1) if base else 0 for i in range(self.G)]
        t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        self.at = {} if dense else {"row_begin": t([b - s for b, s in zip(begins, shift)]), "row_count": t(counts)}
        if base:
            self.at["row_base"] = t([7 * (i + 1) for i in range(-(-self.G // base))])
        self.held = torch.zeros(self.pool, dtype=torch.bool, device=DEV)
        for b, c in zip(begins, counts):
            self.held[b:b + c] = True
        x = normal(seed, self.pool, k) * torch.exp(normal(seed + 1, self.pool, 1))
        codes, self.xs = plain_codes(x, 1)
        self.x, self.xs = codes.to(DEV).view(E4M3), self.xs.to(DEV)
        w = normal(seed + 2, self.G * parts, n, k, std=k ** -0.5) * torch.exp(normal(seed + 3, self.G * parts, 1, 1))
        codes, self.ws = plain_codes(w, 128)
        self.w, self.ws = codes.view(self.G, self.nw, k).to(DEV).view(E4M3), self.ws.view(self.G, parts * self.nb, self.kb).to(DEV)
        self.b = normal(seed + 4, self.G, self.nw)
        self.r = normal(seed + 5, self.pool, n, dtype=out)
        self.op = layer.EpQuantLinearOp(layer.EpLinearConfig(self.G, k, n, self.pool, out_dtype=out, activation=act, groups_per_base=base,
                                                             weight_grad_dtype=weight_grad), backward=backward)
        self.x64 = self.x.double() * self.xs.double().repeat_interleave(128, -1)[:, :k]
        row = torch.arange(self.nw, device=DEV)
        row = row // n * self.nb + row % n // 128
        self.w64 = self.w.double() * self.ws.double()[:, row].repeat_interleave(128, -1)[..., :k]

    def rows(self):
        for g, (b, c) in enumerate(zip(self.begins, self.counts)):
            if c:
                yield g, slice(b, b + c)


def act64(act, z, n):
    if act == "swiglu":
        return z[:, :n] * torch.sigmoid(z[:, :n]) * z[:, n:]
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * torch.special.ndtr(z)}[act]()


def slope64(act, z):
    s = torch.sigmoid(z)
    return {"none": lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(), "silu": lambda: s * (1 + z * (1 - s)),
            "gelu": lambda: torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5}[act]()


def slope_size64(act, z):
    """The magnitudes that an activation's slope is the sum of (GELU: 1/2, erf / 2 and z times
    the density). For z < 0 they cancel (GELU's slope is 0 near -0.75 and almost 0 from -4
    on, SiLU's is 0 near -1.28): f32 steps are off by their 2^-20, not by the slope's."""
    s = torch.sigmoid(z)
    return {"none": lambda: torch.zeros_like(z), "relu": lambda: torch.zeros_like(z), "silu": lambda: s * (1 + z.abs() * (1 - s)),
            "gelu": lambda: 0.5 + 0.5 * torch.erf(z * 0.5 ** 0.5).abs() + z.abs() * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5}[act]()


def within(got, want, bound, what):
    assert torch.isfinite(got.double()).all(), what
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), f"{what}: {float(off.max())} over the bound"


def sum_bound(terms):
    return max(84, terms) * 2.0 ** -23


def check_forward(c, bias, residual, preact):
    y = torch.full((c.pool, c.n), -9.0, dtype=c.out, device=DEV)
    z = torch.full((c.pool, c.nw), -9.0, dtype=torch.bfloat16, device=DEV) if preact else None
    got = c.op.forward(c.x, c.xs, c.w, c.ws, bias=c.b if bias else None, residual=c.r if residual else None, out=y, preact=z, **c.at)
    assert got is y
    for g, rows in c.rows():
        x, w = c.x64[rows], c.w64[g]
        b = c.b[g].double() if bias else torch.zeros(c.nw, device=DEV, dtype=torch.float64)
        want_z = x @ w.T + b
        mag = x.abs() @ w.abs().T + b.abs()
        tol_z = sum_bound(c.k + 2 * c.kb) * mag
        if preact:
            within(z[rows], want_z, tol_z + 2.0 ** -8 * (want_z.abs() + tol_z), "z")
        want = act64(c.act, want_z, c.n)
        if c.act == "swiglu":
            # |d silu| <= 1.1, |silu(v)| <= |v|
            tol = 1.1 * tol_z[:, :c.n] * (want_z[:, c.n:].abs() + tol_z[:, c.n:]) + want_z[:, :c.n].abs() * tol_z[:, c.n:]
        else:
            tol = 1.13 * tol_z
        tol = tol + 2.0 ** -20 * want.abs()
        if residual:
            want = want + c.r[rows].double()
            tol = tol + 2.0 ** -23 * want.abs()
        if c.out == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        within(y[rows], want, tol, "y")
    assert (y[~c.held] == -9.0).all() and (z is None or (z[~c.held] == -9.0).all())
    c.op.sync()
    return y, z


SHAPES = [
    dict(counts=[1], k=16, n=1, dense=True),
    dict(counts=[2], k=4096, n=640, dense=True),
    dict(counts=[3], k=128, n=130, dense=True),
    dict(counts=[1003], k=1008, n=777, dense=True),
    dict(counts=[257], k=144, n=129, dense=True),
    dict(counts=[513], k=2064, n=256, dense=True),
    dict(counts=[64], k=7168, n=256, dense=True),
    dict(counts=[5, 0, 130, 1, 257, 0, 300, 33], k=272, n=200),
    dict(counts=[40] * 20, k=512, n=384, pad=0),
    dict(counts=[0, 0, 0], k=128, n=64),
    dict(counts=[700, 1, 0, 31], k=640, n=128, base=2),
    dict(counts=[8], k=2000, n=333, dense=True),
    dict(counts=[5], k=128 * 40, n=17, dense=True),
    dict(counts=[9], k=400, n=272, dense=True),
    dict(counts=[128, 129, 64, 0, 97, 33], k=384, n=520),
]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["none", "swiglu", "silu", "gelu", "relu"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_forward(layer, shape, act, out):
    c = Case(layer, act=act, out=out, seed=shape, **SHAPES[shape])
    check_forward(c, bias=shape % 2 == 0, residual=shape % 3 == 1, preact=shape % 3 != 2)


def code_slack(dz, off):
    """(dz' in 64 bits, what its codes' choice may leave open) of one half's columns, whose f32
    values are `off` by so much at most."""
    M, n = dz.shape
    v = torch.nn.functional.pad(dz, (0, -n % 128)).unflatten(-1, (-1, 128))
    scale = v.abs().amax(-1, keepdim=True) / 448.0
    q = torch.where(scale > 0, v / torch.where(scale > 0, scale, 1.0), 0.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3.0)
    code = torch.round(q / step) * step
    off = torch.nn.functional.pad(off, (0, -n % 128)).unflatten(-1, (-1, 128)) / torch.where(scale > 0, scale, 1.0)
    # the scale is off by its own roundings and by its block's largest value's
    near = ((q / step).abs() % 1.0 - 0.5).abs() <= (off + (2.0 ** -19 + off.amax(-1, keepdim=True) / 448.0) * q.abs()) / step
    flat = lambda t: t.flatten(-2)[:, :n]  # noqa: E731
    return flat(code * scale), flat(torch.where(near, step * scale, 0.0))


def check_backward(c, bias, seed=50):
    dy = normal(seed, c.pool, c.n, dtype=c.out) * torch.exp(normal(seed + 1, c.pool, 1)).to(c.out)
    z = normal(seed + 2, c.pool, c.nw, dtype=torch.bfloat16) * 2 if c.act != "none" else None
    outside = ~c.held
    for t in (dy, z):
        if t is not None:
            t[outside] = float("nan")
    c.xs[outside] = float("nan")
    dx = torch.full((c.pool, c.k), -9.0, dtype=torch.bfloat16, device=DEV)
    got_dx, dw, db = c.op.backward(dy, c.x, c.xs, c.w, c.ws, preact=z, want_dbias=bias, dx=dx, **c.at)
    assert got_dx is dx and (db is None) == (not bias)
    seen = set()
    for g, rows in c.rows():
        seen.add(g)
        d = dy[rows].double()
        v = None if z is None else z[rows].double()
        if c.act == "swiglu":
            gate, up = v[:, :c.n], v[:, c.n:]
            halves = [d * up * slope64("silu", gate), d * gate * torch.sigmoid(gate)]
        else:
            halves = [d if v is None else d * slope64(c.act, v)]
        if c.act == "swiglu":
            sizes = [(d * up).abs() * slope_size64("silu", gate), halves[1].abs()]
        else:
            sizes = [d.abs() * slope_size64(c.act, d if v is None else v)]
        low = [code_slack(h, 2.0 ** -20 * s) for h, s in zip(halves, sizes)]
        size = torch.cat(sizes, 1)
        dz, low, open_ = torch.cat(halves, 1), torch.cat([a for a, _ in low], 1), torch.cat([b for _, b in low], 1)
        w = c.w64[g]
        want = low @ w
        mag = low.abs() @ w.abs()
        # codes and scales of an f32 quotient: a tie in 64 bits may be none in 32, so ties count for all
        tol = (sum_bound(c.nw + 2 * c.parts * c.nb) + 2.0 ** -19) * mag + open_ @ w.abs()
        within(dx[rows], want, tol + 2.0 ** -8 * (want.abs() + tol), "dx")
        x = c.x64[rows]
        want = dz.T @ x
        mag = dz.abs().T @ x.abs()
        m = dz.shape[0]
        tol = (2 * 2.0 ** -8 + 2.0 ** -16 + sum_bound(m)) * mag + 2.0 ** -19 * size.T @ x.abs()
        if dw.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * want.abs()
        within(dw[g], want, tol, "dw")
        if bias:
            within(db[g], dz.sum(0), sum_bound(m) * dz.abs().sum(0) + 2.0 ** -19 * size.sum(0), "db")
    for g in range(c.G):
        if g not in seen:
            assert (dw[g] == 0).all() and (db is None or (db[g] == 0).all())
    assert (dx[~c.held] == -9.0).all()
    c.op.sync()


@pytest.mark.parametrize("act,out,weight_grad", [("none", torch.bfloat16, torch.bfloat16), ("swiglu", torch.bfloat16, torch.bfloat16),
                                                 ("silu", torch.float32, torch.float32), ("gelu", torch.bfloat16, torch.float32),
                                                 ("relu", torch.float32, torch.bfloat16), ("none", torch.float32, torch.float32)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_backward(layer, shape, act, out, weight_grad):
    c = Case(layer, act=act, out=out, seed=shape + 100, backward=True, weight_grad=weight_grad, **SHAPES[shape])
    check_backward(c, bias=shape % 2 == 0)


def test_scales_of_every_bf16(layer):
    """Every positive finite bf16 as a block's largest value, and f32 significands at their ends: a
    scale is the quotient by 448, rounded once."""
    every = torch.arange(1, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros((every.numel(), 16), dtype=torch.bfloat16, device=DEV)
    x[:, 5] = -every.to(DEV)
    op = layer.EpQuantOp(layer.EpQuantConfig(1, 16, x.shape[0]))
    codes, scales = op.quantize(x)
    want = every.float().numpy() / np.float32(448)
    assert torch.equal(scales.cpu()[:, 0], torch.from_numpy(want))
    assert (bits(codes)[:, 5][torch.from_numpy(want) > 0] >= 0x80 + 0x7E).all()      # -448, or -448 of a rounded-up scale
    bit = torch.cat([torch.randint(0, 1 << 23, (200000,), generator=torch.Generator().manual_seed(3)), torch.arange(0, 1 << 23, 257)])
    for exponent in (1, 40, 127, 200, 254):
        v = ((exponent << 23) | bit).to(torch.int32).view(torch.float32)
        x = torch.zeros((v.numel(), 16), device=DEV)
        x[:, 0] = v.to(DEV)
        op = layer.EpQuantOp(layer.EpQuantConfig(1, 16, x.shape[0], dtype=torch.float32))
        scales = op.quantize(x)[1].cpu()[:, 0]
        assert torch.equal(scales, torch.from_numpy(v.numpy() / np.float32(448)))
