"""Router and product handles without a GPU: configs, workspaces and arguments
are checked before any launch, and the layer module refuses tensors that do not
fit. No address here is dereferenced."""
import pytest
import torch

FAKE = 1 << 40


@pytest.fixture(scope="module")
def ep():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import ep as mod
    return mod


def router(ep, **kw):
    c = ep.ep_router_config()
    base = dict(world_size=8, max_num_inp_token_per_rank=128, num_experts=256, num_experts_per_token=8,
                logits_dtype=ep.EP_DTYPE_FP32, score_func=ep.EP_SCORE_SIGMOID, num_groups=8, topk_groups=4,
                normalize_weights=1, seq_len=0, route_scale=2.5, balance_coef=0.01)
    base.update(kw)
    for k, v in base.items():
        setattr(c, k, v)
    return c


def linear(ep, **kw):
    c = ep.ep_linear_config()
    base = dict(max_rows=1000, num_groups=4, groups_per_base=2, in_features=64, out_features=33,
                out_dtype=ep.EP_DTYPE_BF16, weight_grad_dtype=ep.EP_DTYPE_BF16, activation=ep.EP_ACT_SWIGLU, backward=1)
    base.update(kw)
    for k, v in base.items():
        setattr(c, k, v)
    return c


def refused(ep, status, call):
    with pytest.raises(ep.EpError) as ei:
        call()
    assert ei.value.status == status
    assert ep.ep_last_error()


@pytest.mark.parametrize("bad", [dict(world_size=0), dict(world_size=33), dict(max_num_inp_token_per_rank=0), dict(num_experts=0),
                                 dict(num_experts=1025), dict(num_experts_per_token=0), dict(num_experts_per_token=33),
                                 dict(num_experts=4, num_groups=1, topk_groups=1), dict(logits_dtype=2), dict(score_func=2),
                                 dict(num_groups=0), dict(num_groups=7), dict(num_groups=64), dict(topk_groups=0), dict(topk_groups=9),
                                 dict(num_groups=32, topk_groups=1, num_experts_per_token=9), dict(route_scale=0.0),
                                 dict(route_scale=float("nan")), dict(route_scale=float("inf")), dict(balance_coef=-1.0),
                                 dict(balance_coef=float("nan")), dict(seq_len=-1), dict(max_num_inp_token_per_rank=2 ** 31 - 1)])
def test_router_config_refused(ep, bad):
    c = router(ep, **bad)
    assert ep.ep_router_workspace_size(c) == 0
    refused(ep, ep.EP_ERR_INVALID_ARG, lambda: ep.ep_router_create(c, FAKE, 1 << 40))


def test_router_workspace_and_arguments(ep):
    c = router(ep)
    n = ep.ep_router_workspace_size(c)
    assert n >= 2 * 16 * 256 * 4                    # sums of 16 chunks of rows
    refused(ep, ep.EP_ERR_WORKSPACE, lambda: ep.ep_router_create(c, FAKE, n - 1))
    refused(ep, ep.EP_ERR_WORKSPACE, lambda: ep.ep_router_create(c, FAKE + 16, n))
    refused(ep, ep.EP_ERR_WORKSPACE, lambda: ep.ep_router_create(c, None, n))
    h = ep.ep_router_create(c, FAKE, n)
    bad = ep.EP_ERR_INVALID_ARG
    try:
        refused(ep, bad, lambda: ep.ep_router_forward(h, None, None, None, FAKE, FAKE, None, None, None))
        refused(ep, bad, lambda: ep.ep_router_forward(h, FAKE + 2, None, None, FAKE, FAKE, None, None, None))
        refused(ep, bad, lambda: ep.ep_router_forward(h, FAKE, None, None, None, FAKE, None, None, None))
        refused(ep, bad, lambda: ep.ep_router_forward(h, FAKE, None, None, FAKE, None, None, None, None))
        refused(ep, bad, lambda: ep.ep_router_forward(h, FAKE, None, None, FAKE, FAKE, FAKE, None, None))
        refused(ep, bad, lambda: ep.ep_router_forward(h, FAKE, None, [0] * 7 + [129], FAKE, FAKE, None, None, None))
        refused(ep, bad, lambda: ep.ep_router_forward(h, FAKE, None, [-1] + [0] * 7, FAKE, FAKE, None, None, None))
        refused(ep, bad, lambda: ep.ep_router_balance_loss(h, FAKE, None, None, FAKE, FAKE, None))
        refused(ep, bad, lambda: ep.ep_router_balance_loss(h, FAKE, FAKE, None, None, FAKE, None))
        refused(ep, bad, lambda: ep.ep_router_backward(h, FAKE, FAKE, None, None, None, None, FAKE, None))
        refused(ep, bad, lambda: ep.ep_router_backward(h, FAKE, None, None, FAKE, None, None, FAKE, None))
        refused(ep, bad, lambda: ep.ep_router_backward(h, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, None))
        refused(ep, bad, lambda: ep.ep_router_backward(h, FAKE, FAKE, None, FAKE, None, None, None, None))
        refused(ep, bad, lambda: ep.ep_router_backward(h, FAKE, FAKE, None, FAKE, None, None, FAKE + 1, None))
    finally:
        ep.ep_router_destroy(h)
    refused(ep, bad, lambda: ep.ep_router_forward(None, FAKE, None, None, FAKE, FAKE, None, None, None))
    s = router(ep, score_func=ep.EP_SCORE_SOFTMAX)
    h = ep.ep_router_create(s, FAKE, ep.ep_router_workspace_size(s))
    try:
        refused(ep, ep.EP_ERR_UNSUPPORTED, lambda: ep.ep_router_forward(h, FAKE, FAKE, None, FAKE, FAKE, None, None, None))
    finally:
        ep.ep_router_destroy(h)
        ep.ep_router_destroy(None)


@pytest.mark.parametrize("bad", [dict(num_groups=0), dict(num_groups=1025), dict(groups_per_base=-1), dict(in_features=0),
                                 dict(in_features=60), dict(out_features=0), dict(max_rows=0), dict(max_rows=2 ** 31), dict(out_dtype=2),
                                 dict(weight_grad_dtype=3), dict(activation=5), dict(activation=-1)])
def test_linear_config_refused(ep, bad):
    c = linear(ep, **bad)
    assert ep.ep_linear_workspace_size(c) == 0
    refused(ep, ep.EP_ERR_INVALID_ARG, lambda: ep.ep_linear_create(c, FAKE, 1 << 40))


def test_linear_workspace_and_arguments(ep):
    c = linear(ep)
    n = ep.ep_linear_workspace_size(c)
    assert n >= 1000 * 66 * 2                      # dz
    assert ep.ep_linear_workspace_size(linear(ep, backward=0)) < n
    refused(ep, ep.EP_ERR_WORKSPACE, lambda: ep.ep_linear_create(c, FAKE, n - 1))
    refused(ep, ep.EP_ERR_WORKSPACE, lambda: ep.ep_linear_create(c, FAKE + 128, n))
    bad = ep.EP_ERR_INVALID_ARG
    F = FAKE

    def forward(h, x=F, w=F, bias=None, res=None, b=F, c=F, base=None, rows=0, y=F, z=None):
        return lambda: ep.ep_linear_forward(h, x, w, bias, res, b, c, base, rows, y, z, None)

    def backward(h, dy=F, x=F, w=F, z=F, b=F, c=F, base=None, rows=0, dx=F, dw=F, db=F):
        return lambda: ep.ep_linear_backward(h, dy, x, w, z, b, c, base, rows, dx, dw, db, None)

    h = ep.ep_linear_create(c, FAKE, n)
    try:
        for call in (forward(h, x=None), forward(h, x=F + 8), forward(h, w=F + 2), forward(h, y=None), forward(h, y=F + 1),
                     forward(h, b=None), forward(h, c=None), forward(h, b=None, c=None), forward(h, bias=F + 2), forward(h, z=F + 1),
                     forward(h, res=F + 1), forward(None)):
            refused(ep, bad, call)
        for call in (backward(h, dy=None), backward(h, dy=F + 1), backward(h, z=None), backward(h, dx=None, dw=None, db=None),
                     backward(h, dx=F + 1), backward(h, dw=F + 1), backward(h, db=F + 2), backward(h, x=None)):
            refused(ep, bad, call)
    finally:
        ep.ep_linear_destroy(h)
    d = linear(ep, num_groups=1, groups_per_base=0, backward=0)
    h = ep.ep_linear_create(d, FAKE, ep.ep_linear_workspace_size(d))
    try:
        for call in (forward(h, b=None, c=None, rows=-1), forward(h, b=None, c=None, rows=1001), forward(h, base=F)):
            refused(ep, bad, call)
        refused(ep, ep.EP_ERR_STATE, backward(h))
    finally:
        ep.ep_linear_destroy(h)
        ep.ep_linear_destroy(None)


def test_misaligned_addresses_refused(ep):
    c = router(ep)
    h = ep.ep_router_create(c, FAKE, ep.ep_router_workspace_size(c))
    bad = ep.EP_ERR_INVALID_ARG
    try:
        for at in (2, 4, 5, 6, 7):               # bias, indices, weights, counts, loss
            args = [h, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, None]
            args[at] = FAKE + 2
            refused(ep, bad, lambda: ep.ep_router_forward(*args))
        for at in (2, 4, 5):                     # indices, counts, loss
            args = [h, FAKE, FAKE, None, FAKE, FAKE, None]
            args[at] = FAKE + 1
            refused(ep, bad, lambda: ep.ep_router_balance_loss(*args))
        for at in (2, 4, 5, 6, 7):               # indices, d_weights, counts, d_loss, d_logits
            args = [h, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, None]
            args[at] = FAKE + 2
            refused(ep, bad, lambda: ep.ep_router_backward(*args))
    finally:
        ep.ep_router_destroy(h)
    c = linear(ep)
    h = ep.ep_linear_create(c, FAKE, ep.ep_linear_workspace_size(c))
    try:
        for at in (5, 6, 7):                     # row_begin, row_count, row_base
            args = [h, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, 0, FAKE, None, None]
            args[at] = FAKE + 2
            refused(ep, bad, lambda: ep.ep_linear_forward(*args))
    finally:
        ep.ep_linear_destroy(h)


def test_layer_refuses_tensors_that_do_not_fit(ep):
    from combine_route_layout_gb300 import EpError, EpLinearConfig, EpLinearOp, EpRouterConfig, EpRouterOp
    op = EpRouterOp(EpRouterConfig(2, 4, 16, 2), device="cpu")       # nothing is launched
    good = torch.zeros((2, 4, 16))
    idx = torch.zeros((2, 4, 2), dtype=torch.int32)
    for call in (lambda: op.forward(good[:, :3]), lambda: op.forward(good.bfloat16()),
                 lambda: op.forward(good.transpose(0, 1).contiguous().transpose(0, 1)), lambda: op.forward(None),
                 lambda: op.forward(good, bias=torch.zeros(15)), lambda: op.forward(good, num_tokens=[1]),
                 lambda: op.balance_loss(good, idx.long()), lambda: op.backward(good, None, d_weights=torch.zeros((2, 4, 2))),
                 lambda: op.backward(good, idx, counts=torch.zeros((1, 16), dtype=torch.int32))):
        with pytest.raises(EpError):
            call()
    for kw in (dict(score_func="tanh"), dict(logits_dtype=torch.float16)):
        with pytest.raises(EpError):
            EpRouterOp(EpRouterConfig(2, 4, 16, 2, **kw), device="cpu")
    op = EpLinearOp(EpLinearConfig(2, 16, 8, 30, activation="swiglu"), device="cpu", backward=True)
    bf = torch.bfloat16
    x, w = torch.zeros((30, 16), dtype=bf), torch.zeros((2, 16, 16), dtype=bf)
    seg = dict(row_begin=torch.zeros(2, dtype=torch.int32), row_count=torch.zeros(2, dtype=torch.int32))
    for call in (lambda: op.forward(x, w[:, :8], **seg), lambda: op.forward(x.float(), w, **seg), lambda: op.forward(x[:20], w, **seg),
                 lambda: op.forward(x, w, bias=torch.zeros((2, 8)), **seg), lambda: op.forward(x, w, residual=torch.zeros((30, 16), dtype=bf), **seg),
                 lambda: op.forward(x, w, row_begin=torch.zeros(2), row_count=seg["row_count"]),
                 lambda: op.forward(x, w, row_base=torch.zeros(1, dtype=torch.int32), **seg), lambda: op.forward(x, w),
                 lambda: op.backward(torch.zeros((30, 8), dtype=bf), x, w, None, **seg),
                 lambda: op.backward(torch.zeros((30, 16), dtype=bf), x, w, torch.zeros((30, 16), dtype=bf), **seg)):
        with pytest.raises(EpError):
            call()
    with pytest.raises(EpError):
        EpLinearOp(EpLinearConfig(2, 16, 8, 30, activation="tanh"), device="cpu")
