"""GPU tests of products whose segments overlap: forward passes compute such rows for each of
their groups, refuse what has more tiles than they can number, and the quantised backward
pass reports overlapping segments that need more scratch than there is."""
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


def int32s(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def refused(op):
    from combine_route_layout_gb300 import EpError
    with pytest.raises(EpError) as ei:
        op.sync()
    assert ei.value.status == -4
    op.sync()


def test_more_tiles_than_an_int32_numbers(layer):
    """1024 groups that all have all of 2^29 rows: 2^31 tiles. Nothing is computed."""
    G, pool = 1024, 1 << 29
    at = dict(row_begin=int32s([0] * G), row_count=int32s([pool] * G))
    y = torch.full((pool, 1), -7.0, dtype=BF16, device=DEV)
    x = torch.zeros((pool, 16), dtype=torch.uint8, device=DEV).view(E4M3)
    xs = torch.ones((pool, 1), device=DEV)
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(G, 16, 1, pool))
    op.forward(x, xs, torch.zeros((G, 1, 16), device=DEV).to(E4M3), torch.ones((G, 1, 1), device=DEV), out=y, **at)
    refused(op)
    assert bool((y[::4097] == -7).all()) and bool((y[-300:] == -7).all())
    del xs
    x = x.view(BF16)
    op = layer.EpLinearOp(layer.EpLinearConfig(G, 8, 1, pool))
    op.forward(x, torch.zeros((G, 1, 8), dtype=BF16, device=DEV), out=y, **at)
    refused(op)
    assert bool((y[::4097] == -7).all()) and bool((y[-300:] == -7).all())


def test_same_rows_in_two_groups_of_a_forward_pass(layer):
    """Groups with the same weights: whichever comes last, their rows are right."""
    k, n, pool = 256, 160, 500
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-2, 3, (pool, k), generator=g, device=DEV).float()
    w = torch.randint(-2, 3, (1, n, k), generator=g, device=DEV).float()
    at = dict(row_begin=int32s([0, 100, 300]), row_count=int32s([400, 150, 200]))
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(3, k, n, pool, out_dtype=F32))
    y = op.forward(x.to(E4M3), torch.ones((pool, 2), device=DEV), w.to(E4M3).expand(3, n, k).contiguous(), torch.ones((3, 2, 2), device=DEV), **at)
    assert torch.equal(y.double(), x.double() @ w[0].double().t())
    op.sync()


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_overlapping_segments_of_a_backward_pass_are_reported(layer, act):
    """Three groups that each have the whole pool of 640 rows need 30 blocks of 64 rows; the scratch
    of the quantised backward pass has 13."""
    k, n, pool, G = 128, 64, 640, 3
    parts = 2 if act == "swiglu" else 1
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(G, k, n, pool, activation=act), backward=True)
    dy = torch.ones((pool, n), dtype=BF16, device=DEV)
    z = torch.ones((pool, parts * n), dtype=BF16, device=DEV)
    x, xs = torch.ones((pool, k), device=DEV).to(E4M3), torch.ones((pool, 1), device=DEV)
    w, ws = torch.ones((G, parts * n, k), device=DEV).to(E4M3), torch.ones((G, parts, 1), device=DEV)
    op.backward(dy, x, xs, w, ws, preact=z, want_dbias=True, row_begin=int32s([0] * G), row_count=int32s([pool] * G))
    refused(op)
    # and the operator is as good as before
    _, _, db = op.backward(dy, x, xs, w, ws, preact=None if act == "none" else z, want_dbias=True,
                           row_begin=int32s([0, 640, 0]), row_count=int32s([640, 0, 0]))
    op.sync()
    assert (db[0] != 0).all() and (db[1:] == 0).all()
