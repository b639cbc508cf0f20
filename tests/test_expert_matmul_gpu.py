"""The experts' products in 8 bits against plain implementations in 64 bits.

Quantized values and scales are equal to the definition's, bit for bit.  A product's
terms are exact in 32 bits (8 significant bits, and the scales behind the sum): each
addition, and each of the two multiplications by scales a block, is off by a step of
32 bits at most, of the sum of the terms' magnitudes.
"""
import math

import pytest
import torch

import segmented_top_selection_amd as st

pytestmark = pytest.mark.gpu

DEV = "cuda"
F8 = torch.float8_e4m3fn
STEP = 2.0 ** -23  # of 32 bits
EIGHT = 7 * 2.0 ** -13


def inner(terms, t):
    """How far a sum of so many terms is off before it is rounded to t, of its magnitudes."""
    steps = (terms + 3 * ((terms + 127) // 128)) * STEP
    return steps if t == torch.float32 else steps + EIGHT
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def blocks_of(n):
    return -(-n // 128)


def plain_quantize(x, rows=1):
    """x (..., rows, width) by blocks of rows x 128: (8 bits, scales)."""
    *lead, m, w = x.shape
    mb, wb = -(-m // rows), blocks_of(w)
    f = torch.zeros(*lead, mb * rows, wb * 128, device=x.device)
    f[..., :m, :w] = x.float()
    f = f.unflatten(-1, (wb, 128)).unflatten(-3, (mb, rows))  # ..., mb, rows, wb, 128
    most = f.abs().amax((-1, -3)).clamp(min=2.0 ** -96)
    # Quotients of 32 bits, rounded once: by way of 64 bits, which are wide enough for that
    # (torch multiplies by a number's reciprocal).
    inverse, scale = (448.0 / most.double()).float(), (most.double() / 448.0).float()
    q = (f * inverse[..., :, None, :, None]).to(F8).flatten(-2, -1).flatten(-3, -2)
    return q[..., :m, :w], scale


def values(q, scales, rows=1):
    s = scales.double().repeat_interleave(rows, -2)[..., :q.shape[-2], :]
    return q.double() * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def same_bits(a, b):
    bits = {1: torch.uint8, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.view(bits), b.view(bits))


def edges(g, *shape, dtype=torch.float32):
    """Values of many sizes: zeros, blocks of nothing else, subnormals, the largest."""
    x = randn(g, *shape, dtype=torch.float32)
    x = x * torch.exp2(torch.randint(-12, 13, shape, generator=g, device=DEV).float())
    x = torch.where(torch.rand(*shape, generator=g, device=DEV) < 0.1, -0.0, x).to(dtype)
    if x.shape[-2] > 4:
        x[..., 1, :] = 0.0
        x[..., 2, :] = torch.finfo(dtype).max
        x[..., 3, :] = torch.finfo(dtype).smallest_normal / 4
    return x


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("rows,width", [(0, 5), (1, 1), (1, 128), (3, 127), (17, 129), (33, 1001),
                                        (300, 64), (7, 4096), (1000, 260)])
def test_quantize_rows(rows, width, dtype):
    x = edges(gen(rows + width), rows, width, dtype=dtype)
    q, s = st.quantize_rows(x)
    torch.cuda.synchronize()
    assert q.dtype == F8 and q.shape == x.shape and s.shape == (rows, blocks_of(width))
    want_q, want_s = plain_quantize(x)
    assert same_bits(q, want_q) and same_bits(s, want_s)


def test_quantize_rows_layouts():
    g = gen(1)
    wide = edges(g, 40, 700, dtype=torch.bfloat16)
    for x in (wide[:, 3:400], wide[::3], wide.t(), wide[5:6, 1:2].expand(6, 1)):
        q, s = st.quantize_rows(x)
        want_q, want_s = plain_quantize(x)
        assert same_bits(q, want_q) and same_bits(s, want_s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = st.quantize_rows(wide, stream=side)
    torch.cuda.synchronize()
    assert same_bits(q, plain_quantize(wide)[0])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_what_is_not_finite_marks_its_block(bad):
    x = randn(gen(2), 3, 300)
    x[1, 200] = bad
    v = values(*st.quantize_rows(x))
    assert bool(v[1, 128:256].isnan().all()) and bool(v[1, :128].isfinite().all())
    assert bool(v[[0, 2]].isfinite().all()) and bool(v[1, 256:].isfinite().all())


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (129, 127), (5, 1001), (3, 130, 260),
                                   (0, 5, 7), (4, 0, 9), (2, 300, 1)])
def test_quantize_blocks(shape, dtype):
    x = edges(gen(sum(shape)), *shape, dtype=dtype)
    q, s = st.quantize_blocks(x)
    torch.cuda.synchronize()
    assert q.dtype == F8 and q.shape == x.shape
    assert s.shape == (*shape[:-2], blocks_of(shape[-2]), blocks_of(shape[-1]))
    if x.numel():
        want_q, want_s = plain_quantize(x, 128)
        assert same_bits(q, want_q) and same_bits(s, want_s)


def test_quantize_blocks_layouts():
    wide = edges(gen(3), 4, 150, 400, dtype=torch.float16)
    for x in (wide[:, 3:140, 5:300], wide[::2], wide.transpose(1, 2), wide[1], wide[0].t()):
        q, s = st.quantize_blocks(x)
        want_q, want_s = plain_quantize(x, 128)
        assert same_bits(q, want_q) and same_bits(s, want_s)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("tokens,k,experts,width,dropped", [
    (1, 2, 8, 256, 0.0), (37, 3, 5, 1001, 0.2), (200, 8, 16, 128, 0.0), (5, 1, 3, 7, 0.5),
    (64, 4, 4, 515, 1.0), (0, 2, 4, 64, 0.0)])
def test_dispatch_quantized(tokens, k, experts, width, dropped, dtype):
    g = gen(tokens + width)
    x = edges(g, tokens, width, dtype=dtype)
    ids = torch.randint(0, experts, (tokens, k), generator=g, device=DEV)
    ids[torch.rand(tokens, k, generator=g, device=DEV) < dropped] = -1
    _, position, offsets = st.sort_ids(ids, experts)
    q, s = st.dispatch_quantized(x, position, offsets)
    rows = st.dispatch(x, position, offsets)
    want_q, want_s = st.quantize_rows(rows)
    kept = int(offsets[-1])
    assert q.shape == rows.shape and same_bits(q, want_q) and same_bits(s[:kept], want_s[:kept])
    assert bool((s[kept:] == 0).all())
    q, s = st.dispatch_quantized(x, position)  # all kept
    want_q, want_s = st.quantize_rows(st.dispatch(x, position))
    assert same_bits(q, want_q) and same_bits(s, want_s)


# --------------------------------------------------------------------------
def offsets_of(counts):
    return torch.tensor([0, *counts], device=DEV).cumsum(0)


def plain_product(rows, row_scales, weights, weight_scales, offsets):
    """(the product, the sum of its terms' magnitudes)."""
    x, off = values(rows, row_scales), offsets.tolist()
    out = torch.zeros(rows.shape[0], weights.shape[1], dtype=torch.float64, device=DEV)
    size = torch.zeros_like(out)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        w = values(weights[e], weight_scales[e], 128).t().contiguous()
        out[a:b], size[a:b] = x[a:b] @ w, x[a:b].abs() @ w.abs()
    return out, size


def half_step(t, exact):
    return torch.finfo(t).eps / 2 * exact.abs() + (2.0 ** -25 if t == torch.float16 else 2.0 ** -149)


def close(got, want, inner):
    bound = half_step(got.dtype, want.abs() + inner) + inner
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((err <= bound).all()), f"off by {float((err / bound).max()):.3g} of the bound"


def check_product(rows, row_scales, weights, weight_scales, offsets, **kw):
    out = st.expert_matmul(rows, row_scales, weights, weight_scales, offsets, **kw)
    torch.cuda.synchronize()
    want, size = plain_product(rows, row_scales, weights, weight_scales, offsets)
    assert out.shape == want.shape
    close(out, want, inner(rows.shape[1], out.dtype) * size)
    return out


def operands(g, rows, experts, width, depth):
    x = st.quantize_rows(randn(g, rows, depth))
    w = st.quantize_blocks(randn(g, experts, width, depth, scale=depth ** -0.5))
    return (*x, *w)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("counts,width,depth", [
    ([1], 1, 1), ([1], 128, 128), ([16], 16, 256), ([17], 130, 127), ([128], 256, 384),
    ([129, 0, 3], 257, 130), ([0, 0, 0, 5], 64, 1001), ([300, 1, 260], 200, 260), ([2] * 70, 40, 515),
    ([1000], 515, 1024), ([31, 33, 64, 65, 100, 127], 333, 4096), ([0, 0], 9, 9), ([600, 500], 640, 512)])
def test_expert_matmul(counts, width, depth, dtype):
    g = gen(sum(counts) + width + depth)
    check_product(*operands(g, sum(counts), len(counts), width, depth), offsets_of(counts), dtype=dtype)


def test_expert_matmul_rounding_of_large_and_small():
    # Scales far apart between blocks, rows and experts.
    g = gen(1)
    x = randn(g, 200, 700) * torch.exp2(torch.randint(-20, 21, (200, 1), generator=g, device=DEV).float())
    x = x * torch.exp2(torch.randint(-6, 7, (1, 700), generator=g, device=DEV).float())
    w = randn(g, 3, 300, 700) * torch.exp2(torch.arange(3, device=DEV).float() * 9 - 9)[:, None, None]
    check_product(*st.quantize_rows(x), *st.quantize_blocks(w), offsets_of([70, 0, 130]),
                  dtype=torch.float32)


def test_rows_behind_the_last_expert():
    g = gen(4)
    rows, rs, w, ws = operands(g, 300, 2, 100, 256)
    off = torch.tensor([0, 40, 170], device=DEV)
    out = torch.full((302, 110), 7.0, device=DEV, dtype=torch.float16)
    rs[170:] = math.nan  # not looked at
    view = out[1:301, 5:105]
    got = st.expert_matmul(rows, rs, w, ws, off, out=view)
    want, size = plain_product(rows[:170], rs[:170], w, ws, off)
    assert got is view
    close(view[:170], want, inner(256, view.dtype) * size)
    assert bool((view[170:] == 0).all())
    for rest in (out[:1], out[301:], out[:, :5], out[:, 105:]):
        assert bool((rest == 7).all())
    # None at all.
    st.expert_matmul(rows, rs, w, ws, torch.zeros(3, dtype=torch.int64, device=DEV), out=view)
    assert bool((view == 0).all())


def test_first_rows_belong_to_nobody():
    g = gen(5)
    rows, rs, w, ws = operands(g, 90, 2, 64, 128)
    out = torch.full((90, 64), 3.0, device=DEV)
    st.expert_matmul(rows, rs, w, ws, torch.tensor([20, 50, 90], device=DEV), out=out)
    assert bool((out[:20] == 3).all())
    want, size = plain_product(rows, rs, w, ws, torch.tensor([20, 50, 90], device=DEV))
    close(out[20:], want[20:], inner(128, out.dtype) * size[20:])


@pytest.mark.parametrize("depth", [100, 256])
def test_layouts_of_operands(depth):
    g = gen(6)
    rows, rs, w, ws = operands(g, 70, 3, 96, depth)
    off = offsets_of([30, 0, 40])
    want = st.expert_matmul(rows, rs, w, ws, off)
    # Dense rows (100 bytes apart: copied), rows of wider ones, transposed, scales as views.
    same = lambda *a: torch.equal(st.expert_matmul(*a, off), want)  # noqa: E731
    dense, dense_w = rows.contiguous(), w.contiguous()
    assert same(dense, rs, dense_w, ws)
    wide = torch.zeros(70, 512, device=DEV).to(F8)
    wide[:, 16:16 + depth] = rows
    wide[:, 16 + depth:] = torch.full((), math.nan, device=DEV).to(F8)  # behind the row: anything
    assert same(wide[:, 16:16 + depth], rs, w, ws)
    odd = torch.zeros(70, 512, device=DEV).to(F8)
    odd[:, 3:3 + depth] = rows
    assert same(odd[:, 3:3 + depth], rs, w, ws)
    assert same(rows.t().contiguous().t(), rs.t().contiguous().t(), w, ws)
    assert same(rows, rs, w.transpose(1, 2).contiguous().transpose(1, 2), ws)
    spaced = torch.zeros(6, 96, 512, device=DEV).to(F8)
    spaced[::2, :, :depth] = w
    assert same(rows, rs, spaced[::2, :, :depth], ws)


def test_what_is_not_finite_stays_in_its_row():
    g = gen(7)
    x = randn(g, 60, 300)
    x[11, 7], x[40, 299] = math.nan, math.inf
    w, ws = st.quantize_blocks(randn(g, 2, 70, 300))
    out = st.expert_matmul(*st.quantize_rows(x), w, ws, offsets_of([25, 35]))
    assert bool(out[[11, 40]].isnan().all())
    out[[11, 40]] = 0
    assert bool(out.isfinite().all())


def test_expert_matmul_on_a_stream_and_in_a_graph():
    g = gen(8)
    x = randn(g, 100, 256, dtype=torch.bfloat16)
    w, ws = st.quantize_blocks(randn(g, 8, 192, 256))
    ids = torch.randint(-1, 8, (100, 2), generator=g, device=DEV)
    _, position, offsets = st.sort_ids(ids, 8)

    def run(**kw):
        q, s = st.dispatch_quantized(x, position, offsets, **kw)
        return st.expert_matmul(q, s, w, ws, offsets, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(on_side, run())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
        dw = st.expert_matmul_dweights(out, st.dispatch(x, position, offsets), offsets)
    for _ in range(3):
        x.copy_(randn(g, 100, 256, dtype=torch.bfloat16))
        ids = torch.randint(-1, 8, (100, 2), generator=g, device=DEV)
        for old, new in zip((position, offsets), st.sort_ids(ids, 8)[1:]):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run())
        assert torch.equal(dw, st.expert_matmul_dweights(run(), st.dispatch(x, position, offsets), offsets))


def test_rows_gradient_by_the_transposed_weights():
    g = gen(9)
    rows, rs, w, ws = operands(g, 150, 3, 200, 330)
    off = offsets_of([50, 37, 63])
    dq, ds = st.quantize_rows(randn(g, 150, 200, dtype=torch.bfloat16))
    wt, wts = w.transpose(1, 2).contiguous(), ws.transpose(1, 2).contiguous()
    dx = check_product(dq, ds, wt, wts, off, dtype=torch.float32)
    # <dx, x> = <dout, out>: both are the same sum.
    out, _ = plain_product(rows, rs, w, ws, off)
    a = (dx.double() * values(rows, rs)).sum()
    b = (values(dq, ds) * out).sum()
    size = (values(dq, ds).abs() * plain_product(rows, rs, w, ws, off)[1]).sum()
    assert float((a - b).abs()) <= (inner(200, dx.dtype) + 2 * STEP) * float(size)


# --------------------------------------------------------------------------
def plain_dweights(dout, rows, offsets):
    off = offsets.tolist()
    out = torch.zeros(len(off) - 1, dout.shape[1], rows.shape[1], dtype=torch.float64, device=DEV)
    size = torch.zeros_like(out)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if b > a:
            d, x = (values(*plain_quantize(t[a:b].t())) for t in (dout, rows))
            out[e], size[e] = d @ x.t().contiguous(), d.abs() @ x.abs().t().contiguous()
    return out, size


def inner_of(offsets, size, t):
    return inner(offsets.diff().clamp(min=0), t)[:, None, None] * size


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("counts,width,depth", [
    ([1], 1, 1), ([128], 128, 128), ([129, 0, 3], 130, 257), ([0, 0], 5, 9), ([300, 1, 260], 200, 72),
    ([2] * 70, 40, 33), ([1000], 333, 515), ([127, 128, 129], 64, 1001), ([], 3, 4)])
def test_dweights(counts, width, depth, dtype):
    counts = counts or [0]
    g = gen(sum(counts) + width)
    n = sum(counts)
    dout, rows = randn(g, n, width, dtype=dtype, scale=0.01), randn(g, n, depth, dtype=dtype)
    off = offsets_of(counts)
    want, size = plain_dweights(dout, rows, off)
    for out_type in {dtype, torch.float32}:
        got = st.expert_matmul_dweights(dout, rows, off, dtype=out_type)
        torch.cuda.synchronize()
        assert got.dtype == out_type and got.shape == want.shape
        close(got, want, inner_of(off, size, out_type))


def test_dweights_layouts_and_accumulation():
    g = gen(1)
    wide = randn(g, 200, 300, dtype=torch.bfloat16)
    dout, rows = wide[:, 3:70], randn(g, 200, 150, dtype=torch.bfloat16).t().contiguous().t()
    off = torch.tensor([10, 60, 60, 150], device=DEV)  # rows before the first and behind the last
    wide[150:] = math.nan
    want, size = plain_dweights(dout, rows, off)
    out = randn(g, 5, 80, 160)
    before = out.clone()
    view = out[1:4, 2:69, 7:157]
    got = st.expert_matmul_dweights(dout, rows, off, out=view, accumulate=True)
    assert got is view
    off_by = inner_of(off, size, torch.float32)
    close(view, want + before[1:4, 2:69, 7:157].double(), off_by + half_step(torch.float32, want.abs() + off_by))
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[1:4, 2:69, 7:157] = False
    assert torch.equal(out[rest], before[rest])
    assert torch.equal(out[2, 2:69, 7:157], before[2, 2:69, 7:157])  # an expert without rows
    st.expert_matmul_dweights(dout, rows, off, out=view)
    close(view, want, off_by)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = st.expert_matmul_dweights(dout, rows, off, dtype=torch.float32, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(again, view)


def test_dweights_against_differences():
    # The product is linear in the weights: with values that 8 bits hold, the difference
    # of two losses is the gradient times the step.
    g = gen(3)
    x = torch.randint(-8, 9, (40, 64), generator=g, device=DEV).float()
    dout = torch.randint(-8, 9, (40, 32), generator=g, device=DEV).float()
    x[::10], dout[::10] = 7, 7  # each block's largest: scales of 8 / 448 or 7 / 448
    off = offsets_of([15, 25])
    d = st.expert_matmul_dweights(dout, x, off, dtype=torch.float32)
    step = torch.randint(-1, 2, (2, 32, 64), generator=g, device=DEV).float()
    loss = sum(((x[a:b].double() @ step[e].double().t()) * dout[a:b].double()).sum()
               for e, (a, b) in enumerate(((0, 15), (15, 40))))
    got = (d.double() * step.double()).sum()
    # Quantizing an integer up to 8 is off by 2^-4 of it at most, on either side.
    size = sum((x[a:b].abs().double().t() @ dout[a:b].abs().double()).sum() for a, b in ((0, 15), (15, 40)))
    assert float((got - loss).abs()) <= float((2 * 2.0 ** -4 + 2.0 ** -8) * size)


# --------------------------------------------------------------------------
def test_a_layer_from_logits_to_tokens_and_back():
    """The operators together: a layer of experts, and its gradients by the same calls."""
    g = gen(12)
    tokens, k, experts, width, hidden = 90, 2, 6, 160, 224
    h = randn(g, tokens, width)
    logits = randn(g, tokens, experts)
    up, down = randn(g, experts, hidden, width) / width ** 0.5, randn(g, experts, width, hidden) / hidden ** 0.5
    weights, ids = st.route(logits, k, scoring="sigmoid", bias=torch.zeros(experts, device=DEV))
    _, position, offsets = st.sort_ids(ids, experts)
    up8, down8 = st.quantize_blocks(up), st.quantize_blocks(down)
    rows8 = st.dispatch_quantized(h, position, offsets)
    mid = torch.relu(st.expert_matmul(*rows8, *up8, offsets, dtype=torch.float32))
    mid8 = st.quantize_rows(mid)
    y = st.expert_matmul(*mid8, *down8, offsets, dtype=torch.float32)
    out = st.combine(y, position, offsets, weights)

    # The same in 64 bits, on the values that the 8 bits stand for.
    off = offsets.tolist()
    x64, up64, down64 = values(*rows8), values(*up8, 128), values(*down8, 128)
    mid64 = torch.zeros(tokens * k, hidden, dtype=torch.float64, device=DEV)
    y64 = torch.zeros(tokens * k, width, dtype=torch.float64, device=DEV)
    for e in range(experts):
        a, b = off[e], off[e + 1]
        mid64[a:b] = (x64[a:b] @ up64[e].t().contiguous()).relu()
        y64[a:b] = values(*mid8)[a:b] @ down64[e].t().contiguous()
    want = (y64[position.long()] * weights.double()[:, :, None]).sum(1)
    assert float((mid.double() - mid64).abs().max()) <= inner(width, mid.dtype) * float((x64.abs().amax() * up64.abs().amax()) * width)
    assert float((out.double() - want).abs().max()) <= (inner(hidden, out.dtype) + 4 * STEP) * float(values(*mid8).abs().amax() * down64.abs().amax() * hidden)

    dout = randn(g, tokens, width)
    dy, dweights = st.combine_backward(dout, y, position, offsets, weights)
    dlogits = st.route_backward(dweights, logits, ids, scoring="sigmoid")
    ddown = st.expert_matmul_dweights(dy, mid, offsets)
    down_t = [t.transpose(1, 2).contiguous() for t in down8]
    dmid = st.expert_matmul(*st.quantize_rows(dy), *down_t, offsets, dtype=torch.float32) * (mid > 0)
    dup = st.expert_matmul_dweights(dmid, st.dispatch(h, position, offsets), offsets)
    up_t = [t.transpose(1, 2).contiguous() for t in up8]
    drows = st.expert_matmul(*st.quantize_rows(dmid), *up_t, offsets, dtype=torch.float32)
    dh = st.dispatch_backward(drows, position, offsets)
    # Against automatic differentiation of the layer in 64 bits: 8 bits are off by 2^-4
    # of a value at most, a product of two by twice that, in sums of mixed signs.
    leaves = [t.double().requires_grad_() for t in (h, logits, up, down)]
    h2, logits2, up2, down2 = leaves
    p = torch.sigmoid(logits2).gather(1, ids.long())
    w2 = p / p.sum(1, keepdim=True)
    rows2 = h2.repeat_interleave(k, 0)
    each = ids.view(-1).long()
    mid2 = torch.relu((up2[each] * rows2[:, None, :]).sum(2))
    y2 = (down2[each] * mid2[:, None, :]).sum(2)
    ((y2.view(tokens, k, width) * w2[:, :, None]).sum(1) * dout.double()).sum().backward()
    for got, leaf in ((dh, h2), (dlogits, logits2), (dup, up2), (ddown, down2)):
        far = float((got.double() - leaf.grad).norm() / leaf.grad.norm())
        assert far <= 4 * 2 * 2.0 ** -4, far


def test_refusals():
    g = gen(13)
    rows, rs, w, ws = operands(g, 20, 2, 32, 256)
    off = offsets_of([5, 15])
    value = [dict(rs=rs[:, :1]), dict(rs=rs[:19]), dict(ws=ws[:1]), dict(w=w[:, :, :128]), dict(off=off[:2]),
             dict(w=w[0]), dict(rows=rows[0]), dict(rows=rows.cpu()), dict(off=off.cpu()),
             dict(out=torch.empty(20, 31, device=DEV)), dict(out=torch.empty(32, 20, device=DEV).t())]
    wrong = [dict(rows=rows.float()), dict(w=w.float()), dict(rs=rs.double()), dict(off=off.int()),
             dict(dtype=torch.float64), dict(dtype=F8), dict(out=torch.empty(20, 32, device=DEV), dtype=torch.float16)]
    for error, cases in ((ValueError, value), (TypeError, wrong)):
        for c in cases:
            a = dict(rows=rows, rs=rs, w=w, ws=ws, off=off, dtype=None, out=None)
            a.update(c)
            with pytest.raises(error):
                st.expert_matmul(a["rows"], a["rs"], a["w"], a["ws"], a["off"], dtype=a["dtype"], out=a["out"])
    x = randn(g, 20, 40)
    for bad, error in ((x.double(), TypeError), (x[0], ValueError), (x.cpu(), ValueError), (x[:, :0], ValueError)):
        with pytest.raises(error):
            st.quantize_rows(bad)
        with pytest.raises(error):
            st.quantize_blocks(bad)
    position = torch.zeros(19, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        st.dispatch_quantized(x, position)
    with pytest.raises(TypeError):
        st.dispatch_quantized(x, None)
    d = randn(g, 20, 30)
    for a, kw, error in (((d[:19], x, off), {}, ValueError), ((d, x, off[:1]), {}, ValueError),
                         ((d, x.half(), off), {}, TypeError), ((d, x, off), dict(dtype=torch.float16), TypeError),
                         ((d, x, off), dict(accumulate=True), ValueError),
                         ((d, x, off), dict(out=torch.empty(2, 30, 41, device=DEV)), ValueError),
                         ((d, x, off), dict(out=torch.empty(2, 40, 30, device=DEV).transpose(1, 2)), ValueError),
                         ((d, x, off), dict(out=torch.empty(1, 30, 40, device=DEV).expand(2, 30, 40)), ValueError)):
        with pytest.raises(error):
            st.expert_matmul_dweights(*a, **kw)
