"""GPU tests of what the layer operators' handles keep from call to call: error
bits and tickets, in captured graphs."""
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
