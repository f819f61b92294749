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
