"""GPU tests of the norms at the ends of f32's range: rows of infinities, rows whose mean of
squares passes f32, rows of zeros with the smallest eps; and rows of whole numbers, whose
sums are exact, with one piece of eight elements that is not zero, at every place.

Tolerances. Sums of small whole numbers are exact in any order; the mean is rounded once
(its factor 1 / H is rounded too) and eps added, 3 * 2^-24 of it, of which the root keeps
half; the root is rounded once: 2.5 * 2^-24 of the rms, 2^-22 for all of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def layer():
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import layer as mod
    return mod


def values(out, scales):
    return out.float() if scales is None else out.float() * scales.repeat_interleave(128, -1)[:, :out.shape[1]]


@pytest.mark.parametrize("rows,h", [(3, 256), (700, 256), (5, 1000), (2, 7168), (401, 9000), (1, 16384)])
@pytest.mark.parametrize("eps", [1e-38, 1e-40, 1e-44])
@pytest.mark.parametrize("post", [False, True])
def test_rows_of_zeros_with_the_smallest_eps(layer, eps, rows, h, post):
    """rms is 1 / sqrt(eps), up to 1e22, and a row of zeros has n = 0: t = d_stream + rms v, d_block
    with post norm rms' (du w_post), every number in it far below f32's largest."""
    op = layer.EpNormOp(layer.EpNormConfig(h, rows, eps=eps, post_norm=post, stream_dtype=F32, block_dtype=F32), backward=True)
    x = torch.zeros((rows, h), device=DEV)
    w = torch.ones(h, device=DEV)
    wp = torch.ones(h, device=DEV) if post else None
    s, out, _, stats = op.forward(x, w, block=x, weight_post=wp)
    assert (s == 0).all() and (out == 0).all()
    rms = float(torch.tensor(eps, dtype=F32).double()) ** -0.5
    assert ((stats[:, 0].double() / rms - 1).abs() <= 2.0 ** -22).all()
    d = torch.full((rows, h), 2.0 ** -20, dtype=BF16, device=DEV)
    got = op.backward(d, s, w, stats, block=x, weight_post=wp)
    want = rms * 2.0 ** -20
    assert ((got[0].double() / want - 1).abs() <= 2.0 ** -21).all()
    want *= rms if post else 1
    if want < 3e38:
        assert ((got[1].double() / want - 1).abs() <= 2.0 ** -20).all()
    assert (got[2] == 0).all() and (got[3] is None or (got[3] == 0).all())
    op.sync()


@pytest.mark.parametrize("rows,h", [(1, 8), (9, 520), (3, 7168), (500, 7168), (2, 16384), (400, 16384)])
@pytest.mark.parametrize("stream,block", [(BF16, BF16), (F32, F32)])
def test_every_piece_of_a_row_counts(layer, rows, h, stream, block):
    """Row i is zeros but for the pieces of eight at i, i + rows, ...: one each over h / 8 rows, the
    last one among them where there are fewer."""
    pieces = h // 8
    x = torch.zeros((rows, pieces, 8), device=DEV)
    at = torch.arange(rows, device=DEV) if rows < pieces else torch.arange(rows, device=DEV) % pieces
    at[-1] = pieces - 1
    number = torch.tensor([1.0, 2, 3, -4, 5, 6, 7, 8], device=DEV)
    x[torch.arange(rows, device=DEV), at] = number
    x = x.view(rows, h)
    for post in (False, True):
        op = layer.EpNormOp(layer.EpNormConfig(h, rows, eps=1e-6, post_norm=post, stream_dtype=stream, block_dtype=block), backward=True)
        w = torch.ones(h, device=DEV)
        wp = torch.ones(h, device=DEV) if post else None
        zero = torch.zeros((rows, h), dtype=stream, device=DEV)
        want = (204.0 / h + 1e-6) ** -0.5
        _, _, _, stats = op.forward(x.to(stream), w)
        assert ((stats[:, 0].double() / want - 1).abs() <= 2.0 ** -22).all()
        s, out, _, stats = op.forward(zero, w, block=x.to(block), weight_post=wp)
        if post:
            assert ((stats[:, 1].double() / want - 1).abs() <= 2.0 ** -22).all()
        # backward: v n sums to rms 204 / h, of a stream of x and out's gradient x; exact products, one mean
        d = x.to(BF16)
        stats = torch.full((rows, 2), 0.5, device=DEV)     # given numbers: n is x / 2
        got = op.backward(d, x.to(stream), w, stats, block=x.to(block), weight_post=wp)
        mean = 204.0 / 2 / h
        t = 0.5 * (x.double() - x.double() / 2 * mean)
        # t is rounded to the stream's type: at most 2^-8 of the sum of its two terms' magnitudes (of
        # |t| alone, which with 8 features and a mean of 12.75 is 2.7 |x|), 2^-21 for f32's few steps
        step = 2.0 ** -8 if stream == BF16 else 2.0 ** -21
        assert ((got[0].double() - t).abs() <= step * x.double().abs() / 2 * (1 + mean / 2)).all()
        terms = (x.double() * x.double() / 2).sum(0)
        assert torch.equal(got[2].double(), terms)
        op.sync()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("rows,h", [(4, 256), (700, 1000), (4, 7168), (330, 16384)])
def test_infinities_and_a_mean_beyond_f32(layer, rows, h, quant):
    """A mean of squares beyond f32 gives rms 0 and a row of zeros; an infinity in it a NaN in its
    own place (infinity times 0). Neighbours are what they are alone."""
    op = layer.EpNormOp(layer.EpNormConfig(h, rows, quant_type="fp8_e4m3_block128" if quant else "none"))
    g = torch.Generator(device=DEV).manual_seed(h)
    x = torch.randn((rows, h), generator=g, device=DEV).bfloat16()
    w = torch.ones(h, device=DEV)
    _, plain, plain_scales, plain_stats = op.forward(x, w)
    hard = x.clone()
    hard[1, h // 2] = float("inf")
    hard[2] = 1e30
    _, out, scales, stats = op.forward(hard, w)
    keep = [i for i in range(rows) if i not in (1, 2)]
    assert torch.equal(out[keep].view(torch.uint8), plain[keep].view(torch.uint8)) and torch.equal(stats[keep], plain_stats[keep])
    assert stats[1, 0] == 0 and stats[2, 0] == 0
    v = values(out, scales)
    assert (v[2] == 0).all()
    assert v[1, h // 2].isnan() and (v[1, :h // 2] == 0).all() and (v[1, h // 2 + 1:] == 0).all()
    op.sync()
