"""GPU tests of the layer operators on inputs whose results are known exactly,
over many tiles, many rows and many launches."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def whole(gen, *shape, most=2):
    """bf16 whole numbers of -most .. most."""
    return torch.randint(-most, most + 1, shape, generator=gen, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [64, 1280])
def test_products_of_whole_numbers_are_exact(layer, out, K):
    """Sums of products of small whole numbers have no rounding before the result's own, so
    every output is known. Several tiles to a pair of SMs, of one stage or a few: the
    accumulators change hands as often as they can."""
    rows, N = 8192, 2048
    gen = torch.Generator(device=DEV).manual_seed(K)
    x, w, dy = whole(gen, rows, K), whole(gen, 1, N, K), whole(gen, rows, N).to(out)
    op = layer.EpLinearOp(layer.EpLinearConfig(1, K, N, rows, out_dtype=out, weight_grad_dtype=out), backward=True)
    y_ref = (x.double() @ w[0].double().t()).to(out)
    dx_ref = (dy.double() @ w[0].double()).to(torch.bfloat16)
    dw_ref = (dy.double().t() @ x.double()).to(out)
    for _ in range(8):
        y = op.forward(x, w)
        dx, dw, _ = op.backward(dy, x, w)
        assert torch.equal(y, y_ref) and torch.equal(dx, dx_ref)
        assert torch.equal(dw[0], dw_ref)
    op.sync()


def test_kernels_see_what_the_one_before_them_wrote(layer):
    """Chains of calls on alternating inputs, nothing waited for in between, give the bits of
    the same calls one at a time: a router's projection, router and loss, both gradients;
    and a bias' gradient whose every sum is a whole number."""
    R, T, H, E, k = 4, 128, 256, 64, 6
    gen = torch.Generator(device=DEV).manual_seed(2)
    gate = layer.EpLinearOp(layer.EpLinearConfig(1, H, E, R * T, out_dtype=torch.float32,
                                                 weight_grad_dtype=torch.float32), backward=True)
    router = layer.EpRouterOp(layer.EpRouterConfig(R, T, E, k, score_func="sigmoid", seq_len=32))
    w = torch.randn((1, E, H), generator=gen, device=DEV).mul_(H ** -0.5).bfloat16()
    xs = [torch.randn((R * T, H), generator=gen, device=DEV).bfloat16() for _ in range(2)]
    dws = torch.randn((R, T, k), generator=gen, device=DEV)

    def chain(x, wait):
        def done():
            if wait:
                torch.cuda.synchronize()
        logits = gate.forward(x, w).view(R, T, E)
        done()
        weights, indices, counts, loss = router.forward(logits, balance=True)
        done()
        d = router.backward(logits, indices, d_weights=dws, counts=counts, d_loss=loss)
        done()
        dx, dw, db = gate.backward(d.view(R * T, E), x, w, want_dbias=True)
        done()
        return logits, weights, indices, counts, loss, d, dx, dw, db

    want = [chain(x, True) for x in xs]
    got = [chain(xs[i % 2], False) for i in range(40)]
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i % 2]))
    gate.sync()
    router.sync()

    rows, N = 4096, 520
    op = layer.EpLinearOp(layer.EpLinearConfig(1, 64, N, rows), backward=True)
    x, w = whole(gen, rows, 64), whole(gen, 1, N, 64)
    dys = [whole(gen, rows, N) for _ in range(2)]
    refs = [dy.double().sum(0).float() for dy in dys]
    out = [op.backward(dys[i % 2], x, w, want_dx=False, want_dweight=False, want_dbias=True)[2] for i in range(40)]
    for i, db in enumerate(out):
        assert torch.equal(db[0], refs[i % 2])
    op.sync()


# 129/128 and 252/128: their product is 1.98413, a little less than 254 times bf16's spacing in [1, 2)
ONE, TWO = 129 / 128, 252 / 128


def test_bias_gradient_of_many_rows_is_exact(layer):
    """Counts of 16,777,216 rows: whole sums below 2^24 in every step."""
    rows = 1 << 24
    op = layer.EpLinearOp(layer.EpLinearConfig(1, 8, 8, rows), backward=True)
    x = torch.zeros((rows, 8), dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros((rows, 8), dtype=torch.bfloat16, device=DEV)
    dy[::3] = 1.0
    w = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device=DEV)
    db = op.backward(dy, x, w, want_dx=False, want_dweight=False, want_dbias=True)[2]
    op.sync()
    assert (db == -(-rows // 3)).all()


@pytest.mark.parametrize("what", ["dweight", "dweight of a segment", "forward", "dx"])
def test_long_contractions_round_once(layer, what):
    """Contractions of 2^21 to 2^24 equal terms of one sign. The sum's f32 error is bounded by
    the sums that it is made of: 2^15 terms at a time in the tensor core, 2^11 steps that each
    cut off less than 2^-22 of the sum so far, and up to 2^9 f32 additions: a little over 2^-11
    altogether. The true sum lies 0.03 of a spacing from a bf16 value and rounding turns to the
    next one 2^-9.1 of it away: the result has to be that value."""
    bf = torch.bfloat16
    one, two = (torch.tensor(v, dtype=bf, device=DEV) for v in (ONE, TWO))

    def check(got, terms):
        want = torch.tensor(terms * ONE * TWO, dtype=torch.float64).to(bf)
        assert terms < 1 << 21 or abs(float(want) / (terms * ONE * TWO) - 1) < 2.0 ** -12
        assert (got.float() == float(want)).all(), (float(got.float().min()), float(got.float().max()), float(want))

    if what == "dweight":                      # cut into parts, each of many sums
        rows = 1 << 24
        op = layer.EpLinearOp(layer.EpLinearConfig(1, 8, 8, rows), backward=True)
        x, dy = one.expand(rows, 8).contiguous(), two.expand(rows, 8).contiguous()
        dw = op.backward(dy, x, torch.zeros((1, 8, 8), dtype=bf, device=DEV), want_dx=False)[1]
        check(dw, rows)
    elif what == "dweight of a segment":       # too many tiles for parts; short and empty ones beside it
        counts = [5 * i % 97 for i in range(40)]
        counts[7] = 1 << 21
        begins = [sum(counts[:i]) for i in range(40)]
        rows = sum(counts)
        op = layer.EpLinearOp(layer.EpLinearConfig(40, 8, 8, rows), backward=True)
        x, dy = one.expand(rows, 8).contiguous(), two.expand(rows, 8).contiguous()
        at = {"row_begin": torch.tensor(begins, dtype=torch.int32, device=DEV),
              "row_count": torch.tensor(counts, dtype=torch.int32, device=DEV)}
        dw = op.backward(dy, x, torch.zeros((40, 8, 8), dtype=bf, device=DEV), want_dx=False, **at)[1]
        for g in (7, 6, 39):
            check(dw[g], counts[g])
        assert (dw[0] == 0).all()
    elif what == "forward":
        K = 1 << 22
        op = layer.EpLinearOp(layer.EpLinearConfig(1, K, 8, 5))
        check(op.forward(one.expand(5, K).contiguous(), two.expand(1, 8, K).contiguous()), K)
    else:
        N = 1 << 22
        op = layer.EpLinearOp(layer.EpLinearConfig(1, 8, N, 5), backward=True)
        dx = op.backward(one.expand(5, N).contiguous(), torch.zeros((5, 8), dtype=bf, device=DEV),
                         two.expand(1, N, 8).contiguous(), want_dweight=False)[0]
        check(dx, N)
    op.sync()


# groups, K, N, counts, dweight dtype: contractions long enough to be cut, beside others that are not
@pytest.mark.parametrize("c", [(3, 72, 40, [0, 3200, 17], torch.float32), (2, 512, 129, [700, 4000], torch.float32),
                               (4, 64, 96, [5003, 1, 64, 3073], torch.bfloat16), (3, 136, 200, [3136, 0, 6271], torch.bfloat16)])
def test_weight_gradient_cut_into_parts_over_uneven_segments(layer, c):
    """Whole numbers: every sum is exact below 2^24. Rows outside the segments hold NaN."""
    G, K, N, counts, dt = c
    gen = torch.Generator(device=DEV).manual_seed(G)
    begins = [sum(-(-n // 128) * 128 for n in counts[:i]) for i in range(G)]
    rows = begins[-1] + counts[-1] + 70
    x, dy = whole(gen, rows, K), whole(gen, rows, N)
    held = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for b, n in zip(begins, counts):
        held[b:b + n] = True
    x[~held] = float("nan")
    dy[~held] = float("nan")
    w = torch.zeros((G, N, K), dtype=torch.bfloat16, device=DEV)
    at = {"row_begin": torch.tensor(begins, dtype=torch.int32, device=DEV),
          "row_count": torch.tensor(counts, dtype=torch.int32, device=DEV)}
    op = layer.EpLinearOp(layer.EpLinearConfig(G, K, N, rows, weight_grad_dtype=dt), backward=True)
    for _ in range(3):
        _, dw, db = op.backward(dy, x, w, want_dx=False, want_dbias=True, **at)
        for g, (b, n) in enumerate(zip(begins, counts)):
            assert torch.equal(dw[g], (dy[b:b + n].double().t() @ x[b:b + n].double()).to(dt))
            assert torch.equal(db[g], dy[b:b + n].double().sum(0).float())
    op.sync()


def test_all_of_a_large_segment(layer):
    """270,000 rows of 8,192, nearly all of them in one segment: its weight and bias gradients
    whole, its first and last rows and some between them of everything else."""
    rows, K, N = 270000, 64, 8192
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(0, 3, (rows, K), generator=gen, device=DEV).to(torch.bfloat16)
    w = whole(gen, 2, N, K)
    counts = [rows - 300, 300]
    at = {"row_begin": torch.tensor([0, counts[0]], dtype=torch.int32, device=DEV),
          "row_count": torch.tensor(counts, dtype=torch.int32, device=DEV)}
    op = layer.EpLinearOp(layer.EpLinearConfig(2, K, N, rows, activation="relu"), backward=True)
    z = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    y = op.forward(x, w, preact=z, **at)
    dx, dw, db = op.backward(torch.ones_like(z), x, w, z, want_dbias=True, **at)
    op.sync()
    some = torch.cat([torch.arange(0, 300), torch.arange(150000, 150300), torch.arange(counts[0] - 300, counts[0])]).to(DEV)
    ref = x[some].double() @ w[0].double().t()
    assert torch.equal(z[some].double(), ref) and torch.equal(y[some].double(), ref.clamp(min=0))
    assert torch.equal(dx[some], ((ref > 0).double() @ w[0].double()).bfloat16())
    want_w = torch.zeros((N, K), dtype=torch.float64, device=DEV)
    want_b = torch.zeros(N, dtype=torch.float64, device=DEV)
    for a in range(0, counts[0], 10000):
        b = min(a + 10000, counts[0])
        on = (x[a:b].float() @ w[0].float().t() > 0).double()    # whole numbers: exact
        want_w += on.t() @ x[a:b].double()
        want_b += on.sum(0)
    assert torch.equal(dw[0], want_w.bfloat16()) and torch.equal(db[0], want_b.float())
