"""Handles of the quantiser, of the products of quantised operands and of the norms
without a GPU: configs, workspaces and arguments are checked before any launch, and
the layer module refuses tensors that do not fit. No address here is dereferenced."""
import pytest
import torch

FAKE = 1 << 40


@pytest.fixture(scope="module")
def ep():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import ep as mod
    return mod


def filled(c, base, more):
    for k, v in {**base, **more}.items():
        setattr(c, k, v)
    return c


def quant(ep, **kw):
    return filled(ep.ep_quant_config(), dict(max_rows=1000, num_groups=4, groups_per_base=2, features=272, block_rows=1, dtype=ep.EP_DTYPE_BF16), kw)


def linear(ep, **kw):
    return filled(ep.ep_linear_config(), dict(max_rows=1000, num_groups=4, groups_per_base=2, in_features=64, out_features=33,
                                              out_dtype=ep.EP_DTYPE_BF16, weight_grad_dtype=ep.EP_DTYPE_BF16, activation=ep.EP_ACT_SWIGLU,
                                              backward=1), kw)


def norm(ep, **kw):
    return filled(ep.ep_norm_config(), dict(max_rows=1000, hidden_dim=136, stream_dtype=ep.EP_DTYPE_BF16, block_dtype=ep.EP_DTYPE_FP32,
                                            quant_type=ep.EP_QUANT_NONE, post_norm=1, gate=ep.EP_GATE_FEATURE, backward=1, eps=1e-6,
                                            residual_scale=0.5), kw)


def refused(ep, status, call):
    with pytest.raises(ep.EpError) as ei:
        call()
    assert ei.value.status == status
    assert ep.ep_last_error()


@pytest.mark.parametrize("bad", [dict(max_rows=0), dict(max_rows=2 ** 31), dict(num_groups=0), dict(num_groups=1025), dict(groups_per_base=-1),
                                 dict(features=0), dict(features=8), dict(features=24), dict(features=2 ** 23), dict(block_rows=0),
                                 dict(block_rows=64), dict(dtype=2), dict(block_rows=128, num_groups=2049),
                                 dict(block_rows=128, num_groups=2048, max_rows=2 ** 21), dict(block_rows=128, num_groups=2000, max_rows=2 ** 20, features=2 ** 22)])
def test_quant_config_refused(ep, bad):
    c = quant(ep, **bad)
    assert ep.ep_quant_workspace_size(c) == 0
    refused(ep, ep.EP_ERR_INVALID_ARG, lambda: ep.ep_quant_create(c, FAKE, 1 << 40))


@pytest.mark.parametrize("bad", [dict(in_features=8), dict(in_features=72), dict(in_features=0), dict(out_features=0), dict(num_groups=0),
                                 dict(max_rows=0), dict(out_dtype=2), dict(weight_grad_dtype=3), dict(activation=5)])
def test_qlinear_config_refused(ep, bad):
    c = linear(ep, **bad)
    assert ep.ep_qlinear_workspace_size(c) == 0
    refused(ep, ep.EP_ERR_INVALID_ARG, lambda: ep.ep_qlinear_create(c, FAKE, 1 << 40))


@pytest.mark.parametrize("bad", [dict(max_rows=0), dict(max_rows=2 ** 31), dict(hidden_dim=0), dict(hidden_dim=12), dict(hidden_dim=16392),
                                 dict(stream_dtype=2), dict(block_dtype=3), dict(quant_type=2), dict(gate=3), dict(gate=-1), dict(eps=0.0),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(residual_scale=float("nan")),
                                 dict(residual_scale=float("inf"))])
def test_norm_config_refused(ep, bad):
    c = norm(ep, **bad)
    assert ep.ep_norm_workspace_size(c) == 0
    refused(ep, ep.EP_ERR_INVALID_ARG, lambda: ep.ep_norm_create(c, FAKE, 1 << 40))


@pytest.mark.parametrize("kind", ["quant", "qlinear", "norm"])
def test_workspaces(ep, kind):
    c = {"quant": quant, "qlinear": linear, "norm": norm}[kind](ep)
    size, create, destroy = (getattr(ep, f"ep_{kind}_{f}") for f in ("workspace_size", "create", "destroy"))
    n = size(c)
    assert n > 0
    for at, have in ((None, n), (FAKE + 128, n), (FAKE, n - 1)):
        refused(ep, ep.EP_ERR_WORKSPACE, lambda: create(c, at, have))
    destroy(create(c, FAKE, n))
    destroy(None)
    refused(ep, ep.EP_ERR_INVALID_ARG, lambda: getattr(ep, f"ep_{kind}_sync")(None, None))


def test_backward_scratch_is_reserved(ep):
    # dz and x in bf16, dz's codes and scales
    assert ep.ep_qlinear_workspace_size(linear(ep)) - ep.ep_qlinear_workspace_size(linear(ep, backward=0)) >= \
        1000 * (66 * 2 + 64 * 2 + 256 + 8)
    assert ep.ep_norm_workspace_size(norm(ep)) >= ep.ep_norm_workspace_size(norm(ep, backward=0)) + 152 * 3 * 136 * 4


def test_quant_arguments(ep):
    bad, F = ep.EP_ERR_INVALID_ARG, FAKE

    def call(h, x=F, b=F, c=F, base=None, n=0, codes=F, scales=F):
        return (lambda: ep.ep_quantize(h, x, b, c, base, n, codes, scales, None),
                lambda: ep.ep_dequantize(h, codes, scales, b, c, base, n, x, None))

    c = quant(ep)
    h = ep.ep_quant_create(c, F, ep.ep_quant_workspace_size(c))
    try:
        for kw in (dict(x=None), dict(x=F + 8), dict(codes=None), dict(codes=F + 4), dict(scales=None), dict(scales=F + 2), dict(b=None),
                   dict(c=None), dict(b=None, c=None), dict(b=F + 1), dict(c=F + 2), dict(base=F + 2), dict(b=None, c=None, base=F)):
            for f in call(h, **kw):
                refused(ep, bad, f)
        for f in call(None):
            refused(ep, bad, f)
    finally:
        ep.ep_quant_destroy(h)
    c = quant(ep, num_groups=1, groups_per_base=0)
    h = ep.ep_quant_create(c, F, ep.ep_quant_workspace_size(c))
    try:
        for kw in (dict(b=None, c=None, n=-1), dict(b=None, c=None, n=1001), dict(base=F)):
            for f in call(h, **kw):
                refused(ep, bad, f)
    finally:
        ep.ep_quant_destroy(h)
    c = quant(ep, block_rows=128)
    h = ep.ep_quant_create(c, F, ep.ep_quant_workspace_size(c))
    try:
        for kw in (dict(n=1000), dict(b=None, c=None, n=999), dict(b=None, c=None, base=F, n=1000)):
            for f in call(h, **kw):
                refused(ep, bad, f)
    finally:
        ep.ep_quant_destroy(h)


def test_qlinear_arguments(ep):
    bad, F = ep.EP_ERR_INVALID_ARG, FAKE

    def forward(h, x=F, xs=F, w=F, ws=F, bias=None, res=None, b=F, c=F, base=None, rows=0, y=F, z=None):
        return lambda: ep.ep_qlinear_forward(h, x, xs, w, ws, bias, res, b, c, base, rows, y, z, None)

    def backward(h, dy=F, x=F, xs=F, w=F, ws=F, z=F, b=F, c=F, base=None, rows=0, dx=F, dw=F, db=F):
        return lambda: ep.ep_qlinear_backward(h, dy, x, xs, w, ws, z, b, c, base, rows, dx, dw, db, None)

    c = linear(ep)
    h = ep.ep_qlinear_create(c, F, ep.ep_qlinear_workspace_size(c))
    try:
        for kw in (dict(x=None), dict(x=F + 8), dict(xs=None), dict(xs=F + 2), dict(w=None), dict(w=F + 4), dict(ws=None), dict(ws=F + 1),
                   dict(b=None), dict(c=None), dict(b=None, c=None), dict(b=F + 2), dict(base=F + 2)):
            refused(ep, bad, forward(h, **kw))
            refused(ep, bad, backward(h, **kw))
        for kw in (dict(y=None), dict(y=F + 1), dict(bias=F + 2), dict(res=F + 1), dict(z=F + 1)):
            refused(ep, bad, forward(h, **kw))
        for kw in (dict(dy=None), dict(dy=F + 1), dict(z=None), dict(z=F + 1), dict(dx=None, dw=None, db=None), dict(dx=F + 1), dict(dw=F + 1),
                   dict(db=F + 2)):
            refused(ep, bad, backward(h, **kw))
        refused(ep, bad, forward(None))
        refused(ep, bad, backward(None))
    finally:
        ep.ep_qlinear_destroy(h)
    c = linear(ep, num_groups=1, groups_per_base=0, backward=0)
    h = ep.ep_qlinear_create(c, F, ep.ep_qlinear_workspace_size(c))
    try:
        for kw in (dict(b=None, c=None, rows=-1), dict(b=None, c=None, rows=1001), dict(base=F)):
            refused(ep, bad, forward(h, **kw))
        refused(ep, ep.EP_ERR_STATE, backward(h))
    finally:
        ep.ep_qlinear_destroy(h)


def test_norm_arguments(ep):
    bad, F = ep.EP_ERR_INVALID_ARG, FAKE

    def forward(h, x=F, y=F, g=F, wp=F, w=F, n=10, s=F, o=F, sc=None, st=F):
        return lambda: ep.ep_norm_forward(h, x, y, g, wp, w, n, s, o, sc, st, None)

    def backward(h, d=F, ds=F, x=F, y=F, g=F, wp=F, w=F, st=F, n=10, dx=F, dy=F, dw=F, dp=F, dg=F):
        return lambda: ep.ep_norm_backward(h, d, ds, x, y, g, wp, w, st, n, dx, dy, dw, dp, dg, None)

    c = norm(ep)
    h = ep.ep_norm_create(c, F, ep.ep_norm_workspace_size(c))
    try:
        for kw in (dict(y=None), dict(y=F + 8), dict(g=None), dict(g=F + 4), dict(wp=None), dict(wp=F + 4), dict(w=None), dict(w=F + 8),
                   dict(n=-1), dict(n=1001), dict(st=F + 2)):
            refused(ep, bad, forward(h, **kw))
            refused(ep, bad, backward(h, **kw))
        for kw in (dict(x=None), dict(x=F + 2), dict(s=None), dict(s=F + 8), dict(o=None), dict(o=F + 8), dict(sc=F)):
            refused(ep, bad, forward(h, **kw))
        for kw in (dict(d=None), dict(d=F + 8), dict(ds=F + 8), dict(x=None), dict(st=None), dict(dx=None), dict(dx=F + 8), dict(dy=None),
                   dict(dy=F + 8), dict(dw=None), dict(dw=F + 2), dict(dp=None), dict(dp=F + 2), dict(dg=None), dict(dg=F + 2)):
            refused(ep, bad, backward(h, **kw))
        refused(ep, bad, forward(None))
        refused(ep, bad, backward(None))
    finally:
        ep.ep_norm_destroy(h)
    c = norm(ep, backward=0, quant_type=ep.EP_QUANT_FP8_E4M3_BLOCK128, gate=ep.EP_GATE_NONE, post_norm=0)
    h = ep.ep_norm_create(c, F, ep.ep_norm_workspace_size(c))
    try:
        for kw in (dict(g=None, wp=None), dict(g=F, wp=None, sc=F), dict(g=None, wp=F, sc=F), dict(g=None, wp=None, sc=F + 2),
                   dict(y=None, g=None, wp=None, sc=F)):
            refused(ep, bad, forward(h, **kw))
        refused(ep, ep.EP_ERR_STATE, backward(h, g=None, wp=None))
    finally:
        ep.ep_norm_destroy(h)


def test_layer_refuses_tensors_that_do_not_fit(ep):
    from combine_route_layout_gb300 import EpError, EpLinearConfig, EpNormConfig, EpNormOp, EpQuantConfig, EpQuantLinearOp, EpQuantOp
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    z = lambda *shape, t=torch.float32: torch.zeros(shape).to(t)  # noqa: E731
    seg = dict(row_begin=z(2, t=torch.int32), row_count=z(2, t=torch.int32))
    calls = []
    op = EpQuantOp(EpQuantConfig(2, 144, 30), device="cpu")
    x = z(30, 144, t=bf)
    calls += [lambda: op.quantize(x), lambda: op.quantize(x.float(), **seg), lambda: op.quantize(x[:20], **seg), lambda: op.quantize(x[:, :128], **seg),
              lambda: op.quantize(x, codes=z(30, 144), **seg), lambda: op.quantize(x, scales=z(30, 1), **seg),
              lambda: op.quantize(x, row_base=z(1, t=torch.int32), **seg), lambda: op.dequantize(z(30, 144, t=f8), z(30, 1), **seg),
              lambda: op.dequantize(z(30, 144), z(30, 2), **seg), lambda: op.dequantize(z(30, 144, t=f8), z(30, 2), out=x.float(), **seg)]
    op2 = EpQuantOp(EpQuantConfig(2, 144, 30, block_rows=128), device="cpu")
    m = z(2, 30, 144, t=bf)
    calls += [lambda: op2.quantize(m[:1]), lambda: op2.quantize(m.float()), lambda: op2.quantize(m, **seg), lambda: op2.quantize(m, num_rows=30),
              lambda: op2.quantize(m, scales=z(2, 2, 2)), lambda: op2.quantize(None)]
    lin = EpQuantLinearOp(EpLinearConfig(2, 144, 40, 30, activation="swiglu"), device="cpu", backward=True)
    a, s, w, ws = z(30, 144, t=f8), z(30, 2), z(2, 80, 144, t=f8), z(2, 2, 2)
    dy, pre = z(30, 40, t=bf), z(30, 80, t=bf)
    calls += [lambda: lin.forward(a.to(bf), s, w, ws, **seg), lambda: lin.forward(a, s[:, :1], w, ws, **seg), lambda: lin.forward(a, s, w.to(bf), ws, **seg),
              lambda: lin.forward(a, s, w, ws[:, :1], **seg), lambda: lin.forward(a, s, w, ws), lambda: lin.forward(a, s, w, ws, bias=z(2, 40), **seg),
              lambda: lin.forward(a, s, w, ws, preact=dy, **seg), lambda: lin.forward(a, s, w, ws, out=pre, **seg), lambda: lin.forward(a, None, w, ws, **seg),
              lambda: lin.backward(dy, a, s, w, ws, **seg), lambda: lin.backward(pre, a, s, w, ws, preact=pre, **seg),
              lambda: lin.backward(dy, a, s, w, ws, preact=pre, dx=a, **seg)]
    no = EpNormOp(EpNormConfig(144, 30, post_norm=True, gate="token", block_dtype=torch.float32), device="cpu", backward=True)
    r, y, v, t, st = z(30, 144, t=bf), z(30, 144), z(144), z(30), z(30, 2)
    good = dict(block=y, weight_post=v, gate=t)
    calls += [lambda: no.forward(r.float(), v, **good), lambda: no.forward(z(31, 144, t=bf), v, **good), lambda: no.forward(r[:, :136], v, **good),
              lambda: no.forward(r, v, block=r, weight_post=v, gate=t), lambda: no.forward(r, v, block=y, weight_post=v),
              lambda: no.forward(r, v, block=y, gate=t), lambda: no.forward(r, v, block=y, weight_post=v, gate=v), lambda: no.forward(r, v, gate=t),
              lambda: no.forward(r, v, weight_post=v), lambda: no.forward(r, v, scales=z(30, 2), **good), lambda: no.forward(r, v, stream=r.clone()),
              lambda: no.forward(r, v[:136], **good), lambda: no.forward(None, v), lambda: no.backward(r, r, v, st[:20], **good),
              lambda: no.backward(y, r, v, st, **good), lambda: no.backward(r, r, v, st, d_stream=y, **good),
              lambda: no.backward(r, r, v, st, d_residual=y, **good), lambda: no.backward(r, r, v, None, **good)]
    for call in calls:
        with pytest.raises(EpError):
            call()
    for bad in (lambda: EpQuantOp(EpQuantConfig(1, 144, 30, dtype=torch.float16), device="cpu"), lambda: EpQuantOp(EpQuantConfig(1, 144, 30, 2), device="cpu"),
                lambda: EpNormOp(EpNormConfig(144, 30, gate="row"), device="cpu"), lambda: EpNormOp(EpNormConfig(144, 30, quant_type="fp4"), device="cpu"),
                lambda: EpQuantLinearOp(EpLinearConfig(1, 72, 8, 30), device="cpu")):
        with pytest.raises(EpError):
            bad()


def test_calls_are_refused_while_another_device_is_current(ep, monkeypatch):
    from combine_route_layout_gb300 import EpError, EpLinearConfig, EpNormConfig, EpNormOp, EpQuantConfig, EpQuantLinearOp, EpQuantOp
    from combine_route_layout_gb300 import layer

    def no_stream(device):
        raise AssertionError("asked for a stream of another device")

    monkeypatch.setattr(layer, "_raw_stream", no_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    z = lambda *shape, t=torch.float32: torch.zeros(shape).to(t)  # noqa: E731
    q = EpQuantOp(EpQuantConfig(1, 16, 4), device="cpu")
    lin = EpQuantLinearOp(EpLinearConfig(1, 16, 8, 4), device="cpu", backward=True)
    no = EpNormOp(EpNormConfig(16, 4), device="cpu", backward=True)
    x, s, w, ws = z(4, 16, t=f8), z(4, 1), z(1, 8, 16, t=f8), z(1, 1, 1)
    for call in (lambda: q.quantize(z(4, 16, t=bf)), lambda: q.dequantize(x, s), q.sync, lambda: lin.forward(x, s, w, ws),
                 lambda: lin.backward(z(4, 8, t=bf), x, s, w, ws), lin.sync, lambda: no.forward(z(4, 16, t=bf), z(16)),
                 lambda: no.backward(z(4, 16, t=bf), z(4, 16, t=bf), z(16), z(4, 2)), no.sync):
        with pytest.raises(EpError) as ei:
            call()
        assert ei.value.status == ep.EP_ERR_INVALID_ARG and "current" in str(ei.value)
