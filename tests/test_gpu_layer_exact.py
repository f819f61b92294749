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
