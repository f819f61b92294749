"""GPU tests of the quantiser's and the quantised products' runs: whole numbers that
come out exact over many tiles and parts, the same bits every time, graphs, streams,
host threads, errors, pools beyond 2^31 elements, and a layer of all of them: FP8
dispatch, both experts' products, the quantiser between them, combine and the norms
around it."""
import threading

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


def blocks(n):
    return -(-n // 128)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def codes(seed, *shape, top=2):
    """Small whole numbers as codes."""
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device=DEV).float().to(E4M3)


def powers(seed, *shape):
    return torch.exp2(torch.randint(-1, 3, shape, generator=gen(seed), device=DEV).float())


def int32s(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def segments(counts, pad=128):
    begins, at = [], 0
    for c in counts:
        begins.append(at)
        at += -(-c // pad) * pad if pad else c
    return begins, max(at, 1)


def values(q, s):
    return q.float() * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def weight_values(w, ws, n):
    g, nw, k = w.shape
    row = torch.arange(nw, device=DEV)
    row = row // n * blocks(n) + row % n // 128
    return values(w, ws[:, row])


@pytest.mark.parametrize("counts,k,n,act", [
    ([4096], 1024, 1536, "none"),                      # several tiles a pair
    ([513], 8192, 300, "none"),                        # contractions in parts
    ([100, 0, 257, 31, 128, 129, 700, 64, 1, 5] * 4, 640, 520, "none"),
    ([300] * 40, 256, 1000, "relu"),
    ([17] * 200, 384, 640, "none"),                    # few rows, more tiles than pairs
    ([33, 1, 90], 7168, 128, "none"),                  # few rows, parts
])
def test_whole_numbers_are_exact(layer, counts, k, n, act):
    """Codes of -2..2 and scales of 1/2..4 give terms that are multiples of 1/4, at most 64 of
    them: sums below 2^22 in f32 are exact in any order."""
    torch.backends.cuda.matmul.allow_tf32 = False
    dense = len(counts) == 1
    begins, pool = segments(counts)
    pool = counts[0] if dense else pool
    G = len(counts)
    x, xs = codes(1, pool, k), powers(2, pool, blocks(k))
    w, ws = codes(3, G, n, k), powers(4, G, blocks(n), blocks(k))
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(G, k, n, pool, out_dtype=F32, activation=act), backward=True)
    at = {} if dense else dict(row_begin=int32s(begins), row_count=int32s(counts))
    xv, wv = values(x, xs), weight_values(w, ws, n)
    # small whole numbers with a power of two: dz' is dz, whose largest is 448 of a block's scale
    dy = torch.randint(-2, 3, (pool, n), generator=gen(5), device=DEV).float()
    dy[:, ::64] = 448.0 / 64
    for turn in range(3):
        y = torch.full((pool, n), -7.0, device=DEV)
        op.forward(x, xs, w, ws, out=y, **at)
        for g, (b, c) in enumerate(zip(begins, counts)):
            want = xv[b:b + c] @ wv[g].t()
            assert torch.equal(y[b:b + c], want.clamp(min=0) if act == "relu" else want), (turn, g)
        if act == "none":
            dx = torch.full((pool, k), -7.0, dtype=BF16, device=DEV)
            op.backward(dy, x, xs, w, ws, dx=dx, want_dweight=False, **at)
            for g, (b, c) in enumerate(zip(begins, counts)):
                assert torch.equal(dx[b:b + c], (dy[b:b + c] @ wv[g]).bfloat16()), (turn, g)
    op.sync()


def test_runs_are_the_same(layer):
    counts = [700, 33, 0, 128, 300]
    begins, pool = segments(counts)
    g = gen(1)
    x = torch.randn((pool, 4096), generator=g, device=DEV).to(E4M3)
    xs, ws = (torch.rand(s, generator=g, device=DEV) for s in ((pool, 32), (5, 8, 32)))
    w = torch.randn((5, 1000, 4096), generator=g, device=DEV).to(E4M3)
    z = torch.randn((pool, 1000), generator=g, device=DEV).bfloat16()
    dy = torch.randn((pool, 500), generator=g, device=DEV).bfloat16()
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(5, 4096, 500, pool, activation="swiglu"), backward=True)
    at = dict(row_begin=int32s(begins), row_count=int32s(counts))
    held = torch.cat([torch.arange(b, b + c, device=DEV) for b, c in zip(begins, counts)])

    def run():
        y = op.forward(x, xs, w, ws, **at)
        dx, dw, db = op.backward(dy, x, xs, w, ws, preact=z, want_dbias=True, **at)
        return y[held], dx[held], dw, db

    first = run()
    for _ in range(4):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)
    op.sync()


def test_graph_follows_new_rows_and_counts(layer):
    """Quantise, two products and a backward pass, captured once on handles that have not run, and
    replayed with new rows, counts and weights."""
    G, k, n, pool = 4, 512, 384, 600
    rows = layer.EpQuantOp(layer.EpQuantConfig(G, k, pool))
    mid = layer.EpQuantOp(layer.EpQuantConfig(G, n, pool))
    up = layer.EpQuantLinearOp(layer.EpLinearConfig(G, k, n, pool, activation="swiglu"), backward=True)
    down = layer.EpQuantLinearOp(layer.EpLinearConfig(G, n, k, pool))
    x = torch.zeros((pool, k), dtype=BF16, device=DEV)
    dy = torch.zeros((pool, n), dtype=BF16, device=DEV)
    w1, s1 = torch.zeros((G, 2 * n, k), device=DEV).to(E4M3), torch.zeros((G, 2 * blocks(n), blocks(k)), device=DEV)
    w2, s2 = torch.zeros((G, k, n), device=DEV).to(E4M3), torch.zeros((G, blocks(k), blocks(n)), device=DEV)
    begin, count = int32s([0] * G), int32s([0] * G)
    at = dict(row_begin=begin, row_count=count)
    buffers = [torch.zeros((pool, c), dtype=BF16, device=DEV) for c in (n, 2 * n, k, k)]

    def run():
        h, z, y, dx = buffers
        q, s = rows.quantize(x, **at)
        up.forward(q, s, w1, s1, out=h, preact=z, **at)
        hq, hs = mid.quantize(h, **at)
        down.forward(hq, hs, w2, s2, out=y, **at)
        _, dw, db = up.backward(dy, q, s, w1, s1, preact=z, want_dbias=True, dx=dx, **at)
        return dw, db

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = run()
    for seed, counts in ((1, [100, 30, 0, 129]), (2, [0, 0, 0, 0]), (3, [1, 256, 128, 5])):
        g = gen(seed)
        begins, _ = segments(counts)
        begin.copy_(int32s(begins))
        count.copy_(int32s(counts))
        for t in (x, dy):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        for t in (w1, w2):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV).to(E4M3))
        for t in (s1, s2):
            t.copy_(torch.rand(t.shape, generator=g, device=DEV))
        for t in buffers:
            t.fill_(-1)
        graph.replay()
        got = [t.clone() for t in buffers] + [t.clone() for t in held]
        for t in buffers:
            t.fill_(-1)
        want = [*buffers, *run()]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for op in (rows, mid, up, down):
        op.sync()


def test_two_streams_and_their_own_operators(layer):
    """Two products at once, each with an operator of its own."""
    torch.backends.cuda.matmul.allow_tf32 = False
    made = []
    for i, (m, k, n) in enumerate([(700, 1024, 512), (90, 4096, 300)]):
        x, xs = codes(10 + i, m, k), powers(20 + i, m, blocks(k))
        w, ws = codes(30 + i, 1, n, k), powers(40 + i, 1, blocks(n), blocks(k))
        made.append((layer.EpQuantLinearOp(layer.EpLinearConfig(1, k, n, m, out_dtype=F32)), x, xs, w, ws,
                     values(x, xs) @ weight_values(w, ws, n)[0].t(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for op, x, xs, w, ws, _, st in made:
            with torch.cuda.stream(st):
                got.append(op.forward(x, xs, w, ws))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, made[i % 2][5])
    for op, *_ in made:
        op.sync()


def test_host_threads_with_operators_of_their_own(layer):
    errors = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                m, k, n = 200 + 77 * i, 256 * (i + 1), 128 * (i + 2)
                op = layer.EpQuantLinearOp(layer.EpLinearConfig(1, k, n, m, out_dtype=F32))
                quant = layer.EpQuantOp(layer.EpQuantConfig(1, k, m, dtype=F32))
                x = codes(i, m, k).float()
                x[:, ::128] = 7.0                       # scales of 1/64
                w, ws = codes(50 + i, 1, n, k), powers(60 + i, 1, blocks(n), blocks(k))
                q, s = quant.quantize(x)
                want = x @ weight_values(w, ws, n)[0].t()
                for _ in range(10):
                    if not torch.equal(op.forward(q, s, w, ws), want):
                        errors.append(i)
                op.sync()
                quant.sync()
        except Exception as e:  # noqa: BLE001
            errors.append((i, e))

    torch.backends.cuda.matmul.allow_tf32 = False
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


def test_segments_outside_the_pool_are_cut_and_reported(layer):
    from combine_route_layout_gb300 import EpError
    x, xs = codes(1, 200, 128), powers(2, 200, 1)
    w, ws = codes(3, 3, 64, 128), powers(4, 3, 1, 1)
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(3, 128, 64, 200, out_dtype=F32), backward=True)
    y = torch.full((200, 64), -7.0, device=DEV)
    op.forward(x, xs, w, ws, out=y, row_begin=int32s([150, -3, 10]), row_count=int32s([100, 5, 20]))
    v, wv = values(x, xs), weight_values(w, ws, 64)
    assert torch.equal(y[150:], v[150:] @ wv[0].t()) and torch.equal(y[10:30], v[10:30] @ wv[2].t())
    assert (y[:10] == -7).all() and (y[30:150] == -7).all()
    with pytest.raises(EpError) as ei:
        op.sync()
    assert ei.value.status == -4
    op.sync()


def test_pools_beyond_32_bits(layer):
    """The last rows of pools of more than 2^31 elements."""
    k, pool = 4096, 540_000
    x = torch.zeros((pool, k), dtype=BF16, device=DEV)
    x[-70:] = torch.randn((70, k), generator=gen(1), device=DEV).bfloat16()
    quant = layer.EpQuantOp(layer.EpQuantConfig(1, k, pool))
    begin, count = int32s([pool - 70]), int32s([70])
    q, s = quant.quantize(x, row_begin=begin, row_count=count)
    small = layer.EpQuantOp(layer.EpQuantConfig(1, k, 70))
    want_q, want_s = small.quantize(x[-70:].contiguous())
    assert torch.equal(q[-70:].view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s[-70:], want_s)
    back = quant.dequantize(q, s, row_begin=begin, row_count=count, out=x)
    assert torch.equal(back[-70:], small.dequantize(want_q, want_s))
    w, ws = codes(2, 1, k, k), powers(3, 1, 32, 32)
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(1, k, k, pool), backward=True)
    one = layer.EpQuantLinearOp(layer.EpLinearConfig(1, k, k, 70), backward=True)
    at = dict(row_begin=begin, row_count=count)
    op.forward(q, s, w, ws, out=x, **at)
    want = one.forward(want_q, want_s, w, ws)
    assert torch.equal(x[-70:], want)
    dy = x
    dx, _, _ = op.backward(dy, q, s, w, ws, want_dweight=False, **at)
    assert torch.equal(dx[-70:], one.backward(want, want_q, want_s, w, ws, want_dweight=False)[0])
    norm = layer.EpNormOp(layer.EpNormConfig(k, pool))
    weight = torch.ones(k, device=DEV)
    _, out, _, _ = norm.forward(dx, weight, block=dy)
    # a row's sum of 4096 squares, in an order that goes by the number of rows, is off by
    # 4096 * 2^-23 at most, the rest by a few 2^-24, and out is rounded to bf16
    v = dx[-70:].double() + dy[-70:].double()
    v = v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    assert ((out[-70:].double() - v).abs() <= (2.0 ** -8 + 4096 * 2.0 ** -23 + 2.0 ** -20) * v.abs()).all()
    for o in (quant, op, norm):
        o.sync()


@pytest.mark.parametrize("tokens", [1, 40])
def test_layer_of_fp8_dispatch_products_combine_and_norms(layer, tokens):
    """norm -> FP8 dispatch -> up (SwiGLU) -> quantise -> down -> weighted combine -> residual, gate and
    norms, each step against 64 bits from what the step before gave."""
    from combine_route_layout_gb300 import EpDispatchCombineConfig, EpDispatchCombineOp
    R, H, I, Er, topk = 4, 512, 256, 4, 3
    E, n = R * Er, R * tokens
    g = gen(tokens)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    stream = rand(n, H).bfloat16()
    norm = layer.EpNormOp(layer.EpNormConfig(H, n, gate="token", post_norm=True, residual_scale=0.5, block_dtype=F32))
    w_in, w_post, w_out, gate = 1 + 0.1 * rand(H), 1 + 0.1 * rand(H), 1 + 0.1 * rand(H), torch.sigmoid(rand(n))
    _, x, _, _ = norm.forward(stream, w_in)
    weights = torch.rand((R, tokens, topk), generator=g, device=DEV)
    idx = torch.rand((R, tokens, E), generator=g, device=DEV).argsort(-1)[..., :topk].to(torch.int32).contiguous()
    idx[0, 0, 1] = -1
    cfg = EpDispatchCombineConfig(BF16, R, H, 0, 4, 4, tokens, Er, topk, standard_moe=True, quant_type="fp8_e4m3_block128",
                                  combine_out_dtype=F32, weighted_combine=True)
    ex = EpDispatchCombineOp(cfg)
    packed = ex.dispatch_standard_moe(x.view(R, tokens, H), weights, None, idx)
    rows, scales = packed["packed_recv_x"], packed["packed_recv_scales"]
    pool = rows.shape[0]
    at = dict(row_begin=packed["expert_offset"], row_count=packed["packed_recv_count"], row_base=packed["rank_base"])
    wq = layer.EpQuantOp(layer.EpQuantConfig(2 * E, H, I, block_rows=128))
    up_w, up_s = wq.quantize((rand(2 * E, I, H) * H ** -0.5).bfloat16())
    wq2 = layer.EpQuantOp(layer.EpQuantConfig(E, I, H, block_rows=128))
    down_w, down_s = wq2.quantize((rand(E, H, I) * I ** -0.5).bfloat16())
    up_w, up_s = up_w.view(E, 2 * I, H), up_s.view(E, 2 * blocks(I), blocks(H))
    up = layer.EpQuantLinearOp(layer.EpLinearConfig(E, H, I, pool, activation="swiglu", groups_per_base=Er))
    down = layer.EpQuantLinearOp(layer.EpLinearConfig(E, I, H, pool, groups_per_base=Er))
    mid = layer.EpQuantOp(layer.EpQuantConfig(E, I, pool, groups_per_base=Er))
    h = torch.zeros((pool, I), dtype=BF16, device=DEV)
    y = torch.zeros((pool, H), dtype=BF16, device=DEV)
    up.forward(rows, scales, up_w, up_s, out=h, **at)
    hq, hs = mid.quantize(h, **at)
    down.forward(hq, hs, down_w, down_s, out=y, **at)
    out = ex.combine_standard_moe(y, weights, idx, call_reset=True)
    s2, nxt, _, _ = norm.forward(stream, w_out, block=out.view(n, H), weight_post=w_post, gate=gate)
    # 64 bits, from the rows that dispatch gave
    begin = (at["row_base"].view(-1, 1) + at["row_begin"].view(R, Er)).view(-1)
    rms = lambda v: (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    near = lambda a, b, rel: float((a.double() - b).norm()) <= rel * float(b.norm())  # noqa: E731
    assert near(x, stream.double() * rms(stream.double()) * w_in.double(), 2.0 ** -8)
    uw, dw = weight_values(up_w, up_s, I).double(), weight_values(down_w, down_s, H).double()
    seen = 0
    for e in range(E):
        b, c = int(begin[e]), int(at["row_count"].view(-1)[e])
        seen += c
        if not c:
            continue
        z = values(rows[b:b + c], scales[b:b + c]).double() @ uw[e].t()
        assert near(h[b:b + c], z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:], 2.0 ** -8)
        assert near(y[b:b + c], values(hq[b:b + c], hs[b:b + c]).double() @ dw[e].t(), 2.0 ** -8)
        # a code is off by half a step at most, 2^-4 of the value
        assert near(values(hq[b:b + c], hs[b:b + c]), h[b:b + c].double(), 2.0 ** -4)
    assert seen == int((idx >= 0).sum())
    o = out.view(n, H).double()
    want = stream.double() + 0.5 * gate.double()[:, None] * o * rms(o) * w_post.double()
    assert near(s2, want, 2.0 ** -8) and near(nxt, want * rms(want) * w_out.double(), 2.0 ** -8)
    for op in (norm, ex, wq, wq2, up, down, mid):
        op.sync()


def test_the_most_groups(layer):
    """1024 experts with 0 to 3 rows each, tight segments."""
    torch.backends.cuda.matmul.allow_tf32 = False
    G, k, n = 1024, 256, 144
    counts = [(7 * g) % 4 for g in range(G)]
    begins, pool = segments(counts, pad=0)
    at = dict(row_begin=int32s(begins), row_count=int32s(counts))
    w, ws = codes(3, G, n, k), powers(4, G, blocks(n), blocks(k))
    x = torch.randint(-2, 3, (pool, k), generator=gen(5), device=DEV).float()
    x[:, ::128] = 7.0                                  # scales of 1/64
    quant = layer.EpQuantOp(layer.EpQuantConfig(G, k, pool, dtype=F32))
    q, s = quant.quantize(x, **at)
    assert torch.equal(values(q, s), x)
    op = layer.EpQuantLinearOp(layer.EpLinearConfig(G, k, n, pool, out_dtype=F32, weight_grad_dtype=F32), backward=True)
    y = op.forward(q, s, w, ws, **at)
    wv = weight_values(w, ws, n)
    of = torch.repeat_interleave(torch.arange(G, device=DEV), int32s(counts).long())
    want = torch.bmm(wv[of], x[:, :, None])[..., 0]
    assert torch.equal(y, want)
    dy = torch.randint(-2, 3, (pool, n), generator=gen(6), device=DEV).float()
    dy[:, ::64] = 7.0
    dx, dw, db = op.backward(dy, q, s, w, ws, want_dbias=True, **at)
    assert torch.equal(dx, torch.bmm(dy[:, None], wv[of])[:, 0].bfloat16())
    assert torch.equal(dw, torch.zeros((G, n, k), device=DEV).index_add_(0, of, dy[:, :, None] * x[:, None]))
    assert torch.equal(db, torch.zeros((G, n), device=DEV).index_add_(0, of, dy))
    op.sync()
    quant.sync()


def test_part_of_the_rows_and_residual_in_place(layer):
    """num_rows leaves the rows behind it alone; y may be the residual."""
    torch.backends.cuda.matmul.allow_tf32 = False
    for rows, m, n in ((300, 211, 160), (300, 211, 333), (20, 7, 160), (64, 40, 128)):
        k = 4096 if rows == 64 else 512
        x, xs = codes(1, rows, k), powers(2, rows, blocks(k))
        w, ws = codes(3, 1, n, k), powers(4, 1, blocks(n), blocks(k))
        op = layer.EpQuantLinearOp(layer.EpLinearConfig(1, k, n, rows, out_dtype=F32))
        r = torch.randint(-9, 10, (rows, n), generator=gen(7), device=DEV).float()
        want = r.clone()
        want[:m] += (values(x, xs) @ weight_values(w, ws, n)[0].t())[:m]
        assert op.forward(x, xs, w, ws, residual=r, out=r, num_rows=m) is r
        assert torch.equal(r, want)
        quant = layer.EpQuantOp(layer.EpQuantConfig(1, n, rows, dtype=F32)) if n % 16 == 0 else None
        if quant:
            q, s = torch.full((rows, n), 3, dtype=torch.uint8, device=DEV).view(E4M3), torch.full((rows, blocks(n)), -1.0, device=DEV)
            quant.quantize(want, num_rows=m, codes=q, scales=s)
            assert (q[m:].view(torch.uint8) == 3).all() and (s[m:] == -1).all() and (s[:m] > 0).all()
        op.sync()
