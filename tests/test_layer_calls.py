"""What the layer module does around a call, without a GPU: which device the call
goes to, what it keeps of its arguments. Nothing is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def test_calls_are_refused_while_another_device_is_current(layer, monkeypatch):
    """The stream is that of the operator's device, the launch would go to the current one."""
    from combine_route_layout_gb300 import EpError
    from combine_route_layout_gb300.ep import EP_ERR_INVALID_ARG

    def no_stream(device):
        raise AssertionError("asked for a stream of another device")

    monkeypatch.setattr(layer, "_raw_stream", no_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    router = layer.EpRouterOp(layer.EpRouterConfig(1, 4, 16, 2), device="cpu")
    logits = torch.zeros((1, 4, 16))
    idx = torch.zeros((1, 4, 2), dtype=torch.int32)
    counts = torch.zeros((1, 16), dtype=torch.int32)
    linear = layer.EpLinearOp(layer.EpLinearConfig(1, 16, 8, 4), device="cpu", backward=True)
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    w = torch.zeros((1, 8, 16), dtype=torch.bfloat16)
    dy = torch.zeros((4, 8), dtype=torch.bfloat16)
    for call in (lambda: router.forward(logits), lambda: router.forward(logits, balance=True),
                 lambda: router.balance_loss(logits, idx), lambda: router.sync(),
                 lambda: router.backward(logits, counts=counts, d_loss=torch.ones(())),
                 lambda: linear.forward(x, w), lambda: linear.backward(dy, x, w), lambda: linear.sync()):
        with pytest.raises(EpError) as ei:
            call()
        assert ei.value.status == EP_ERR_INVALID_ARG and "current" in str(ei.value)


def test_token_counts_are_kept_whole(layer, monkeypatch):
    """Counts and the C array that they became are replaced together: whoever asks for the same
    counts between the two steps gets an array of these counts."""
    op = layer.EpRouterOp(layer.EpRouterConfig(2, 4, 16, 2), device="cpu")
    op._tokens([1, 2])
    convert, seen = layer.ep._i32_array, []

    def interrupted(values):
        if len(seen) < 1:
            seen.append(None)
            seen.append(list(op._tokens([3, 4])))    # another thread, just now
        return convert(values)

    monkeypatch.setattr(layer.ep, "_i32_array", interrupted)
    assert list(op._tokens([3, 4])) == [3, 4]
    assert seen[1] == [3, 4]
    assert list(op._tokens([1, 2])) == [1, 2]
