"""GPU tests of what the layer operators' handles keep from call to call: error
bits and tickets, in captured graphs."""
import math

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


def reported(op):
    from combine_route_layout_gb300 import ep
    with pytest.raises(ep.EpError) as ei:
        op.sync()
    return ei.value.status


def captured(calls):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    return g


def test_a_later_captured_call_keeps_the_error_of_an_earlier_one(layer):
    """Calls of a handle that has never run, two in one graph: the first one's error is
    still there after the second, which does not look at what was wrong."""
    from combine_route_layout_gb300 import ep
    E, k = 16, 2
    l = torch.randn((1, 4, E), device=DEV)
    one = torch.ones((), device=DEV)
    bad = torch.zeros((1, 4, k), dtype=torch.int32, device=DEV)
    bad[0, 1, 0] = E

    op = layer.EpRouterOp(layer.EpRouterConfig(1, 4, E, k))

    def loss_and_gradient():
        counts, _ = op.balance_loss(l, bad)
        op.backward(l, counts=counts, d_loss=one)

    g = captured(loss_and_gradient)
    g.replay()
    assert reported(op) == ep.EP_ERR_INVALID_INDEX
    op.sync()
    g.replay()
    assert reported(op) == ep.EP_ERR_INVALID_INDEX

    op2 = layer.EpRouterOp(layer.EpRouterConfig(1, 4, E, k, score_func="sigmoid"))
    bias = torch.zeros(E, device=DEV)
    bias[3] = math.nan

    def route_and_gradient():
        _, indices = op2.forward(l, bias)
        op2.backward(l, indices, d_weights=torch.ones((1, 4, k), device=DEV))

    g2 = captured(route_and_gradient)
    g2.replay()
    assert reported(op2) == ep.EP_ERR_INVALID_ARG

    lin = layer.EpLinearOp(layer.EpLinearConfig(2, 16, 8, 10))
    x = torch.zeros((10, 16), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((2, 8, 16), dtype=torch.bfloat16, device=DEV)
    begin = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    long, fine = (torch.tensor(c, dtype=torch.int32, device=DEV) for c in ([4, 6], [4, 4]))

    def two_products():
        lin.forward(x, w, row_begin=begin, row_count=long)
        lin.forward(x, w, row_begin=begin, row_count=fine)

    g3 = captured(two_products)
    g3.replay()
    assert reported(lin) == ep.EP_ERR_INVALID_INDEX


def test_later_replays_and_eager_calls_keep_an_unreported_error(layer):
    from combine_route_layout_gb300 import ep
    l = torch.zeros((1, 4, 8), device=DEV)
    for later in ("replay", "eager"):
        op = layer.EpRouterOp(layer.EpRouterConfig(1, 4, 8, 2))
        g = captured(lambda: op.forward(l))
        l[0, 2, 3] = math.nan
        g.replay()
        l[0, 2, 3] = 0.0
        if later == "replay":
            g.replay()
        else:
            op.forward(l)
        assert reported(op) == ep.EP_ERR_INVALID_ARG
        op.sync()
        g.replay()
        op.sync()


def test_calls_of_several_captures_start_from_a_cleared_header(layer):
    """A workspace full of other data, a first call captured twice, the second capture run
    alone: no error is made up and split contractions join."""
    cfg = layer.EpLinearConfig(1, 4096, 96, 40)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((40, 4096), generator=gen, device=DEV).bfloat16()
    w = torch.randn((1, 96, 4096), generator=gen, device=DEV).bfloat16()
    want = layer.EpLinearOp(cfg).forward(x, w)
    op = layer.EpLinearOp(cfg)
    op.workspace.fill_(0x5A)
    out = [torch.zeros_like(want) for _ in range(2)]
    graphs = [captured(lambda i=i: (op.forward(x, w, out=out[i]), op.forward(x, w, out=out[i]))) for i in range(2)]
    graphs[1].replay()
    op.sync()
    assert torch.equal(out[1], want) and (out[0] == 0).all()
    graphs[0].replay()
    op.sync()
    assert torch.equal(out[0], want)


def test_after_a_timeout_replays_start_with_fresh_tickets(layer):
    """What a wait that gave up leaves behind (its error bit, tickets that were taken) is written
    into the workspace by hand: the report clears it for a graph that was captured before, which
    holds no clearing of its own."""
    from combine_route_layout_gb300 import ep
    cfg = layer.EpLinearConfig(1, 3648, 96, 40)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((40, 3648), generator=gen, device=DEV).bfloat16()
    w = torch.randn((1, 96, 3648), generator=gen, device=DEV).bfloat16()
    x2 = torch.randn((40, 3648), generator=gen, device=DEV).bfloat16()
    op = layer.EpLinearOp(cfg)
    wants = [op.forward(v, w) for v in (x2, x)]
    op.sync()
    out = torch.zeros_like(wants[0])
    g = captured(lambda: op.forward(x, w, out=out))
    header = op.workspace[:1024].view(torch.int32)
    header[0] = 2                                # kErrLinearTimeout
    header[64:64 + 160] = 7                      # tickets: seven of the eight parts of each tile are in
    assert reported(op) == ep.EP_ERR_TIMEOUT
    assert (header[64:] == 0).all()
    other = x.clone()
    for i in range(4):                           # another input each time: a part that is not waited for shows
        x.copy_((x2, other)[i % 2])
        out.fill_(7.0)
        g.replay()
        assert torch.equal(out, wants[i % 2])
    op.sync()
