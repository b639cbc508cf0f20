"""The operators of routing, the experts' products and verified drafts at sizes that
choose between their kernels' forms, and several calls of them at once.

What is compared, and how far it may be off, is that of the operators' own tests.
"""
import pytest
import torch

import segmented_top_selection_amd as st
import test_expert_matmul_gpu as products
import test_route_gpu as routing
import test_verify_drafts_gpu as drafts

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES, NAMES = products.TYPES, products.NAMES


def shared(g, rows, experts):
    """Rows of `experts` experts, some with none, some with many."""
    liked = torch.randn(experts, generator=g, device=DEV)
    liked[::7] = -9.0
    ids = torch.multinomial(torch.softmax(liked, 0), rows, replacement=True, generator=g)
    return torch.bincount(ids, minlength=experts).tolist()


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("rows,experts,width,depth", [
    (200, 40, 300, 129), (200, 40, 515, 260), (200, 40, 1000, 640),     # few rows an expert
    (800, 40, 200, 384), (800, 40, 300, 1001), (800, 40, 777, 515),     # twice as many
    (1000, 8, 500, 520), (1000, 8, 800, 515), (1000, 8, 1500, 130),     # few large tiles
    (640, 8, 300, 129), (640, 8, 1000, 515), (640, 8, 1900, 260),       # fewer rows of them
    (300, 2, 257, 400), (500, 3, 900, 200),                             # very few
    (1500, 20, 1000, 515),                                              # some
    (5000, 70, 700, 390),                                               # many
    (3000, 2, 5200, 330), (3000, 2, 5200, 128)])                        # of many rows an expert
def test_expert_matmul_forms(rows, experts, width, depth, dtype):
    g = products.gen(rows + experts + width)
    counts = shared(g, rows, experts) if experts > 2 else [1777, rows - 1777]
    products.check_product(*products.operands(g, rows, experts, width, depth),
                           products.offsets_of(counts), dtype=dtype)


def test_expert_matmul_many_large_tiles():
    g = products.gen(1)
    products.check_product(*products.operands(g, 9000, 3, 7300, 140),
                           products.offsets_of([4001, 2303, 2696]), dtype=torch.bfloat16)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("rows,experts,width,depth", [
    (900, 5, 130, 200), (2850, 1, 719, 1123),                     # few tiles
    (3000, 70, 300, 400), (5000, 3, 1300, 1100), (60, 64, 257, 300)])  # many
def test_dweights_forms(rows, experts, width, depth, dtype):
    g = products.gen(rows + width)
    off = products.offsets_of(shared(g, rows, experts) if experts > 1 else [rows])
    dout = products.randn(g, rows, width, dtype=dtype, scale=0.1)
    x = products.randn(g, rows, depth, dtype=dtype)
    want, size = products.plain_dweights(dout, x, off)
    for out_type in {dtype, torch.float32}:
        inner = products.inner_of(off, size, out_type)
        got = st.expert_matmul_dweights(dout, x, off, dtype=out_type)
        products.close(got, want, inner)
        before = products.randn(g, *want.shape, dtype=out_type)
        out = before.clone()
        st.expert_matmul_dweights(dout, x, off, out=out, accumulate=True)
        both = want + before.double()
        products.close(out, both, inner + products.STEP / 2 * (both.abs() + inner))


@pytest.mark.parametrize("accumulate", [False, True])
def test_dweights_large_tiles(accumulate):
    g = products.gen(2)
    counts = [1000, 0, 385, 1, 128, 1114, 700, 33, 640, 500]
    n, off = sum(counts), products.offsets_of(counts)
    dout = products.randn(g, n, 2000, dtype=torch.bfloat16, scale=0.1)
    rows = products.randn(g, n, 3300, dtype=torch.bfloat16)
    want, size = products.plain_dweights(dout, rows, off)
    inner = products.inner_of(off, size, torch.bfloat16)
    del size
    out = products.randn(g, 10, 2000, 3300, dtype=torch.bfloat16)
    if accumulate:
        want += out.double()
        # The sum's rounding to 32 bits.
        inner += products.STEP / 2 * (want.abs() + inner)
    st.expert_matmul_dweights(dout, rows, off, out=out, accumulate=accumulate)
    products.close(out, want, inner)


@pytest.mark.parametrize("lengths,vocab,dtype", [([1], 5_000_011, torch.float16),
                                                 ([2, 0, 3, 1] * 10, 70001, torch.bfloat16),
                                                 ([1, 0], 300_007, torch.float32)])
def test_verify_large(lengths, vocab, dtype):
    drafts.check(drafts.inputs(drafts.gen(vocab), lengths, vocab, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=NAMES.get)
@pytest.mark.parametrize("size,temperature", [(1e17, 1.0), (1e30, 1.0), (-1e30, 0.7), (3e37, 2.0), (10.0, 1e-18),
                                              (10.0, 1e-40), (1.0, 1e-290), (1e-42, 1e-290), (1e30, 1e-300)])
def test_verify_logits_far_past_their_temperature(size, temperature, dtype, monkeypatch):
    # max / temperature is past 2^52: all is on the largest logits, of which there are several.
    # The quotient itself may overflow, a difference's to nothing but the infinity that it stands for.
    plain = drafts.distribution
    monkeypatch.setattr(drafts, "distribution", lambda x, t: plain((x.double() - x.double().max()) / t, 1.0))
    g = drafts.gen(21)
    s = drafts.inputs(g, [3, 0, 2, 1], 2500, dtype, temperature=temperature)
    for name in ("target", "draft"):
        x = torch.randint(0, 40, s[name].shape, generator=g, device=DEV).float()
        s[name] = ((1.0 + x / 64) * size).to(dtype)
    # All but the last row of the first request: nothing but the lowest number.
    s["target"][:3] = torch.finfo(dtype).min
    s["tokens"] = torch.where(torch.arange(6, device=DEV) % 2 == 0, s["draft"].float().argmax(1), s["tokens"])
    drafts.check(s)


@pytest.mark.parametrize("experts,k", [(64, 8), (160, 6), (256, 8), (1000, 3)])
def test_route_where_32_bits_settle_nothing(experts, k):
    # All of a token's scores within a few steps of 32 bits, in every token of a wave.
    g = routing.gen(experts)
    x = 0.5 + torch.randint(0, 40, (37, experts), generator=g, device=DEV).float() * 2.0 ** -24
    bias = torch.randint(0, 2, (experts,), generator=g, device=DEV).float() * 2.0 ** -26
    routing.check(x, k, scoring="sigmoid", bias=bias)


def test_calls_on_two_streams_at_once():
    g = products.gen(5)
    off = products.offsets_of([150, 0, 250])
    streams = [torch.cuda.Stream() for _ in range(2)]
    d = [products.randn(g, 400, 520, dtype=torch.bfloat16) for _ in range(2)]
    x = [products.randn(g, 400, 300, dtype=torch.bfloat16) for _ in range(2)]
    s = [drafts.inputs(drafts.gen(i), [3, 1, 0, 2], 20011, torch.bfloat16) for i in range(2)]

    def calls(i, **kw):
        got = [st.expert_matmul_dweights(d[i], x[i], off, **kw)]
        got += st.verify_drafts(s[i]["target"], s[i]["tokens"], s[i]["offsets"], s[i]["accept"],
                                s[i]["sample"], draft_logits=s[i]["draft"], temperature=0.8, **kw)
        got += st.route(x[i], 8, **kw)
        q, scales = st.quantize_rows(d[i], **kw)
        return got + [q.view(torch.uint8), scales]
    want = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    for stream in streams:
        stream.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(calls(i, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i], strict=True))


def test_two_graphs_in_turn():
    g = products.gen(6)
    off = products.offsets_of([90, 110])
    d, x = products.randn(g, 200, 260, dtype=torch.float16), products.randn(g, 200, 140, dtype=torch.float16)
    s = drafts.inputs(drafts.gen(9), [2, 1], 9001, torch.float16)

    def verify():
        return st.verify_drafts(s["target"], s["tokens"], s["offsets"], s["accept"], s["sample"],
                                draft_logits=s["draft"])

    def gradient():
        return st.expert_matmul_dweights(d, x, off)
    verify(), gradient()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        tokens, counts = verify()
        one = gradient()
    with torch.cuda.graph(graphs[1]):
        two = gradient()
        again, _ = verify()
    for i in range(3):
        d.copy_(products.randn(g, 200, 260, dtype=torch.float16))
        s["target"].copy_(products.randn(g, *s["target"].shape, dtype=torch.float16, scale=3.0))
        for graph in (graphs[i % 2], graphs[1 - i % 2], graphs[0]):
            graph.replay()
        torch.cuda.synchronize()
        want, want_counts = verify()
        assert torch.equal(tokens, want) and torch.equal(again, want) and torch.equal(counts, want_counts)
        assert torch.equal(one, gradient()) and torch.equal(two, one)


def far(memory, like, *strides):
    """A copy of `like` in `memory`, its neighbours so many elements apart."""
    t = memory[:memory.numel() // 16 * 16].view(like.dtype).as_strided(like.shape, strides)
    t.copy_(like)
    return t


def test_places_past_32_bits():
    g = products.gen(7)
    memory = torch.empty(9 << 30, dtype=torch.uint8, device=DEV)
    # Matrices 4.5 GiB apart: weights, and their gradient.
    rows, rs, w, ws = products.operands(g, 60, 2, 130, 256)
    off = products.offsets_of([25, 35])
    want = st.expert_matmul(rows, rs, w, ws, off)
    assert torch.equal(st.expert_matmul(rows, rs, far(memory, w, 9 << 29, 256, 1), ws, off), want)
    d, x = products.randn(g, 60, 130, dtype=torch.bfloat16), products.randn(g, 60, 70, dtype=torch.bfloat16)
    want = st.expert_matmul_dweights(d, x, off)
    out = far(memory, want, 9 << 28, 80, 1).zero_()
    assert torch.equal(st.expert_matmul_dweights(d, x, off, out=out), want)
    q, s = st.quantize_blocks(far(memory, w.float().bfloat16(), 9 << 28, 256, 1))
    want_q, want_s = st.quantize_blocks(w.float().bfloat16())
    assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
    # Rows 4.5 GiB or 300 MiB apart: results, inputs, logits.
    want = st.expert_matmul(*(t[:2] for t in (rows, rs)), w, ws, products.offsets_of([1, 1]))
    out = far(memory, want, 9 << 28, 1).zero_()
    st.expert_matmul(*(t[:2] for t in (rows, rs)), w, ws, products.offsets_of([1, 1]), out=out)
    assert torch.equal(out, want)
    wide = far(memory, x[:30], 150 << 20, 1)
    for got, want in zip(st.quantize_rows(wide), st.quantize_rows(x[:30])):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(st.expert_matmul_dweights(d[:30], wide, off.clamp(max=30)),
                       st.expert_matmul_dweights(d[:30], x[:30], off.clamp(max=30)))
    want = st.route(x[:30], 4)
    got = st.route(wide, 4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dw = products.randn(g, 30, 4)
    assert torch.equal(st.route_backward(dw, wide, want[1]), st.route_backward(dw, x[:30], want[1]))
    s = drafts.inputs(g, [3, 2], 5000, torch.bfloat16)
    s["target"] = far(memory, s["target"], 9 << 26, 1)
    drafts.check(s)
