"""GPU tests of the router's groups of experts where masks leave few of them."""
import itertools
import math

import pytest
import torch

from test_gpu_layer import plain_route, router_math

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


# experts, groups: a group is 1, 2, 4 or 8 lanes, or not a whole run of lanes
@pytest.mark.parametrize("E,groups", [(32, 32), (64, 32), (128, 32), (64, 16), (256, 16), (64, 8), (256, 8), (128, 4), (60, 6), (30, 3),
                                      (1000, 20), (1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_with_fewer_open_groups_than_it_may_take(layer, E, groups, score):
    """Rows whose masks leave none, one, two or three groups open, the first, the last and others
    among them, while topk_groups may stay: every open expert can be chosen."""
    size, k = E // groups, min(4, E // groups * 2)
    stay = min(groups, max(2, groups // 2, -(-k // size)))
    sets = [()] + [s for n in (1, 2, 3) for s in itertools.combinations(sorted({0, 1, groups // 2, groups - 1}), min(n, groups))]
    gen = torch.Generator().manual_seed(E + groups)
    l = torch.randn((1, len(sets), E), generator=gen)
    for t, s in enumerate(sets):
        shut = torch.tensor([e // size not in s for e in range(E)])
        l[0, t, shut] = -math.inf
    l = l.to(DEV)
    cfg = layer.EpRouterConfig(1, len(sets), E, k, score_func=score, num_groups=groups, topk_groups=stay)
    op = layer.EpRouterOp(cfg)
    weights, indices, counts, loss = op.forward(l, balance=True)
    op.sync()
    want = plain_route(cfg, l, None, [len(sets)])
    assert torch.equal(indices.cpu(), want)
    w, ls, ct, _ = router_math(cfg, l.double().cpu(), want, [len(sets)])
    # a weight is a quotient of a sum of at most 4 terms, each off by a few 2^-24
    assert (weights.double().cpu() - w).abs().max() <= 16 * 2.0 ** -24
    assert torch.equal(counts.cpu().long(), ct)
    # a mean of at most 15 rows' quotients, each over up to 1024 terms that decay quickly
    assert abs(float(loss) - float(ls)) <= 84 * 2.0 ** -23 * max(1.0, float(ls))


def test_sigmoid_rows_at_the_end_of_their_range(layer):
    """Rows whose scores are the last ones above f32's underflow: the loss of the call that
    selects, the loss of given indices and the gradient agree with the formula. A score of
    2^-128 has 21 bits, so a probability is off by a few 2^-21, the others' steps by less."""
    E, k = 32, 4
    gen = torch.Generator().manual_seed(7)
    l = -87.4 - 1.3 * torch.rand((1, 9, E), generator=gen)
    l[0, 3, 5:] = -math.inf
    l[0, 4] = torch.randn(E, generator=gen)
    l = l.to(DEV)
    op = layer.EpRouterOp(layer.EpRouterConfig(1, 9, E, k, score_func="sigmoid"))
    w, idx, counts, loss = op.forward(l, balance=True)
    counts2, loss2 = op.balance_loss(l, idx)
    d = op.backward(l, counts=counts, d_loss=torch.ones((), device=DEV))
    op.sync()
    x = l.double().requires_grad_(True)
    p = torch.sigmoid(x) / torch.sigmoid(x).sum(-1, keepdim=True)
    want = (counts[0].double() * E / (k * 9) * p.sum((0, 1)) / 9).sum()
    (grad,) = torch.autograd.grad(want, x)
    assert torch.equal(counts, counts2)
    for got in (loss, loss2):
        assert abs(float(got) - float(want.detach())) <= 2.0 ** -18 * float(want.detach())
    assert (d.double() - torch.nan_to_num(grad)).abs().max() <= 2.0 ** -18 * grad.nan_to_num().abs().max()
