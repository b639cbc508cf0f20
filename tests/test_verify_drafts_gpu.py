"""Verified drafts against a plain implementation in 64 bits.

All results are whole numbers and have to be equal.  The kernels' powers are 7e-11 off
at most; a random uniform number is nearer than that to one of the borders of a row of
10^5 tokens once in 10^5 calls.
"""
import math

import pytest
import torch

import segmented_top_selection_amd as st

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def distribution(x, temperature):
    """A row's probabilities in 64 bits, or None."""
    x = x.double().cpu()
    if bool((x.isnan() | (x == math.inf)).any()) or bool((x == -math.inf).all()):
        return None
    if temperature == 0:
        p = torch.zeros_like(x)
        p[int((x == x.max()).nonzero()[0])] = 1.0
        return p
    return torch.softmax(x / temperature, 0)


def plain(target, tokens, offsets, accept, sample, draft, temperature):
    off, V = offsets.tolist(), target.shape[1]
    requests = len(off) - 1
    out = torch.full((tokens.numel() + requests,), -1, dtype=torch.int64)
    counts = []
    ids = tokens.tolist()
    for r in range(requests):
        t = float(temperature[r]) if isinstance(temperature, torch.Tensor) else temperature
        stood, rest, known = 0, None, True
        for i in range(off[r], off[r + 1]):
            p = distribution(target[i + r], t)
            if draft is not None and t > 0:
                q = distribution(draft[i], t)
            else:
                q = torch.zeros(V, dtype=torch.float64)
                if 0 <= ids[i] < V:
                    q[ids[i]] = 1.0
            if p is None or q is None:
                known = False
                break
            if 0 <= ids[i] < V and float(accept[i].double()) * float(q[ids[i]]) < float(p[ids[i]]):
                out[i + r] = ids[i]
                stood += 1
                continue
            rest = (p - q).clamp(min=0)
            if float(rest.sum()) == 0:
                rest = p
            break
        else:
            rest = distribution(target[off[r + 1] + r], t)
            known = rest is not None
        if known:
            c = rest.cumsum(0)
            above = (c > float(sample[r].double()) * float(c[-1])).nonzero()
            out[off[r] + r + stood] = int(above[0]) if above.numel() else int((rest > 0).nonzero()[-1])
        counts.append(stood + known)
    return out, torch.tensor(counts, dtype=torch.int32)


def inputs(g, lengths, vocab, dtype, drafted=True, near=0.8, ids=torch.int64, temperature=1.0):
    D, R = sum(lengths), len(lengths)
    offsets = torch.tensor([0, *lengths], device=DEV).cumsum(0)
    target = (3 * torch.randn(D + R, vocab, generator=g, device=DEV)).to(dtype)
    row = torch.tensor([i + r for r in range(R) for i in range(sum(lengths[:r]), sum(lengths[:r + 1]))],
                       dtype=torch.int64, device=DEV)
    draft = (target[row].float() + near * torch.randn(D, vocab, generator=g, device=DEV)).to(dtype)
    z = draft.float() / max(temperature, 0.1)
    tokens = (z - torch.empty_like(z).exponential_(generator=g).log()).argmax(1) if D else row
    return dict(target=target, tokens=tokens.to(ids), offsets=offsets,
                accept=torch.rand(D, generator=g, device=DEV), sample=torch.rand(R, generator=g, device=DEV),
                draft=draft if drafted else None, temperature=temperature)


def check(s, **kw):
    tokens, counts = st.verify_drafts(s["target"], s["tokens"], s["offsets"], s["accept"], s["sample"],
                                      draft_logits=s["draft"], temperature=s["temperature"], **kw)
    torch.cuda.synchronize()
    want, want_counts = plain(s["target"], s["tokens"], s["offsets"], s["accept"], s["sample"],
                              s["draft"], s["temperature"])
    assert tokens.dtype == s["tokens"].dtype and counts.dtype == torch.int32
    assert torch.equal(counts.cpu(), want_counts), (counts.tolist(), want_counts.tolist())
    assert torch.equal(tokens.long().cpu(), want), (tokens.tolist(), want.tolist())
    return tokens, counts


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("lengths,vocab", [([0], 1), ([1], 1), ([3], 2), ([4], 1000), ([0, 5, 0, 2], 4097),
                                           ([7, 1, 3], 32003), ([0, 0, 0], 333), ([300], 65), ([2], 131072),
                                           ([1] * 70, 129), ([260, 0, 1], 17)])
def test_verify(lengths, vocab, drafted, dtype):
    g = gen(sum(lengths) + vocab)
    check(inputs(g, lengths, vocab, dtype, drafted, ids=torch.int32 if drafted else torch.int64))


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("requests,vocab", [(40, 12000), (60, 16400), (130, 8200), (130, 20000), (300, 8191),
                                            (300, 16385), (600, 1025)])
def test_rows_drawn_from_in_larger_parts(requests, vocab, dtype):
    # The more requests, the fewer workgroups share a row.
    g = gen(requests + vocab)
    check(inputs(g, [r % 3 % 2 for r in range(requests)], vocab, dtype))


@pytest.mark.parametrize("temperature", [0.0, 0.05, 0.7, 1.0, 30.0])
@pytest.mark.parametrize("drafted", [False, True])
def test_temperatures(temperature, drafted):
    g = gen(4)
    for dtype in TYPES:
        check(inputs(g, [3, 0, 6, 2], 5000, dtype, drafted, temperature=temperature))


def test_a_temperature_for_each_request():
    g = gen(5)
    s = inputs(g, [3, 0, 6, 2, 4, 0], 3000, torch.bfloat16)
    s["temperature"] = torch.tensor([0.0, 1.0, 0.5, 0.0, 2.0, 0.0], device=DEV)
    s["tokens"][9:11] = s["target"][12:14].float().argmax(1)  # greedy ones that stand
    check(s)


@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.5])
def test_borders_that_34_bits_would_miss(temperature):
    # Two tokens, and uniform numbers nearer than 3e-11 to the first one's probability.  In 64
    # bits a power is 1e-13 off at most, and so is a probability p0 (the largest power is exact up
    # to that too): p0 (1 - p0) 2e-13 <= 5e-14, and some 2^-52.
    n = 1 << 22
    x = 5 * torch.randn(n, generator=gen(15), device=DEV)
    p = 1 / (1 + torch.exp(x.double() / temperature))
    u = p.float()
    away = (p - u.double()).abs()
    at = ((away > 2e-13) & (away < 3e-11) & (u < 1)).nonzero()[:, 0]
    assert at.numel() > 500
    x, p, u = x[at], p[at], u[at]
    target = torch.stack([torch.zeros_like(x), x], 1)
    n = at.numel()
    none = torch.zeros(0, device=DEV)
    zeros = torch.zeros(n + 1, dtype=torch.int64, device=DEV)
    tokens, _ = st.verify_drafts(target, zeros[:0], zeros, none, u, temperature=temperature)
    assert torch.equal(tokens, (p <= u.double()).long())
    # A certain draft of the first token stands if u < p.
    _, counts = st.verify_drafts(target.repeat_interleave(2, 0), zeros[:n], torch.arange(n + 1, device=DEV), u, u,
                                 temperature=temperature)
    assert torch.equal(counts == 2, u.double() < p)


def test_all_stand_and_none_stands():
    g = gen(6)
    for near in (0.0, 8.0):  # the draft is the target; it is far from it
        for drafted in (True, False):
            s = inputs(g, [5, 3, 8], 2000, torch.float32, drafted, near=near)
            for u in (0.0, 0.999999):
                s["accept"].fill_(u)
                _, counts = check(s)
                if near == 0.0 and drafted:
                    assert counts.tolist() == [6, 4, 9]  # p = q: u < 1 always stands


def test_ends_of_the_uniform_numbers():
    g = gen(7)
    s = inputs(g, [2, 2, 0, 0], 700, torch.float32)
    s["target"][:, :3] = -math.inf
    s["target"][:, 690:] = -math.inf
    s["accept"].fill_(1.0 - 2.0 ** -24)
    for u in (0.0, 1.0 - 2.0 ** -24):
        s["sample"].fill_(u)
        check(s)
    s["sample"].fill_(1.0)  # outside: the last token that can be
    tokens, _ = check(s)
    assert int(tokens[-1]) == 689


def test_greedy_ties_and_lowest_index():
    x = torch.zeros(5, 9000, device=DEV, dtype=torch.float16)
    x[:, 4500] = 2
    x[:, 8999] = 2
    s = dict(target=x, tokens=torch.tensor([4500, 4500, 8999], device=DEV), offsets=torch.tensor([0, 2, 3], device=DEV),
             accept=torch.zeros(3, device=DEV), sample=torch.zeros(2, device=DEV), draft=None, temperature=0.0)
    tokens, counts = check(s)
    assert tokens.tolist() == [4500, 4500, 4500, 4500, -1] and counts.tolist() == [3, 1]


def test_tokens_ruled_out_and_outside():
    g = gen(8)
    for drafted in (False, True):
        s = inputs(g, [4, 4, 4], 500, torch.float32, drafted)
        s["target"][torch.rand(15, 500, generator=g, device=DEV) < 0.9] = -math.inf
        if drafted:
            s["draft"][torch.rand(12, 500, generator=g, device=DEV) < 0.9] = -math.inf
        s["tokens"][1], s["tokens"][4] = -1, 500
        check(s)
        # p only where q is all: the residual is nothing, and p itself is drawn from.
        s["target"][:] = -math.inf
        s["target"][:, 77] = 1.0
        if drafted:
            s["draft"][:] = s["target"][:12]
        s["tokens"][:] = 76
        tokens, counts = check(s)
        assert counts.tolist() == [1, 1, 1] and tokens[[0, 5, 10]].tolist() == [77, 77, 77]


def test_rows_without_a_distribution():
    g = gen(9)
    for bad in (math.nan, math.inf, None):
        for temperature in (1.0, 0.0):
            for drafted in (False, True):
                s = inputs(g, [3, 2, 0, 1, 2], 6000, torch.float32, drafted, near=0.0, temperature=temperature)
                s["accept"].zero_()
                for row in (1, 6, 7):  # a draft's row, a row behind the drafts, one that has no drafts
                    if bad is None:
                        s["target"][row] = -math.inf
                    else:
                        s["target"][row, 5999] = bad
                if drafted:
                    s["draft"][6, 17] = math.nan
                check(s)


def test_large_and_small_logits():
    g = gen(10)
    s = inputs(g, [3, 3], 4000, torch.float32)
    s["target"] *= 1e4
    s["draft"] *= 1e4
    check(s)
    s = inputs(g, [3, 3], 4000, torch.float32)
    s["target"] = s["target"] * 1e-3 + 3e4
    s["draft"] = s["draft"] * 1e-3 - 3e4
    check(s)
    s["target"][:, ::2] = torch.finfo(torch.float32).min
    check(s)


def test_layouts_streams_and_the_same_twice():
    g = gen(11)
    s = inputs(g, [4, 0, 3], 3000, torch.bfloat16)
    wide = torch.zeros(10, 3100, device=DEV, dtype=torch.bfloat16)
    wide[:, 7:3007] = s["target"]
    a = check(s)
    s["target"] = wide[:, 7:3007]
    s["draft"] = s["draft"].t().contiguous().t()
    b = check(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = check(s, stream=side)
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_graph():
    g = gen(12)
    s = inputs(g, [4, 0, 3, 7], 9000, torch.bfloat16)
    run = lambda: st.verify_drafts(s["target"], s["tokens"], s["offsets"], s["accept"], s["sample"],  # noqa: E731
                                   draft_logits=s["draft"])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, counts = run()
    for _ in range(4):
        for name, v in inputs(g, [4, 0, 3, 7], 9000, torch.bfloat16).items():
            if isinstance(v, torch.Tensor):
                s[name].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert torch.equal(tokens, want[0]) and torch.equal(counts, want[1])


def test_frequencies():
    """The tokens that come first are distributed as the target, whatever the draft."""
    g = gen(13)
    n, vocab = 40000, 6
    target = torch.randn(1, vocab, generator=g, device=DEV).repeat(2 * n, 1)
    draft = torch.randn(1, vocab, generator=g, device=DEV).repeat(n, 1)
    drawn = torch.multinomial(torch.softmax(draft[:1].double(), 1), n, replacement=True, generator=g)[0]
    tokens, _ = st.verify_drafts(target, drawn, torch.arange(n + 1, device=DEV),
                                 torch.rand(n, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV),
                                 draft_logits=draft)
    share = torch.bincount(tokens[::2], minlength=vocab).double() / n
    p = torch.softmax(target[0].double(), 0)
    # Six standard deviations of a share of n draws.
    assert bool(((share - p).abs() <= 6 * (p * (1 - p) / n).sqrt()).all())


def test_no_requests_and_refusals():
    empty = torch.zeros(0, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    tokens, counts = st.verify_drafts(torch.zeros(0, 5, device=DEV), none, torch.zeros(1, dtype=torch.int64, device=DEV),
                                      empty, empty)
    assert tokens.numel() == counts.numel() == 0
    s = inputs(gen(14), [2, 1], 50, torch.float32)
    value = [dict(target=s["target"][:4]), dict(tokens=s["tokens"][:2]), dict(offsets=s["offsets"][:2]),
             dict(accept=s["accept"][:2]), dict(sample=s["sample"][:1]), dict(draft=s["draft"][:2]),
             dict(draft=s["draft"][:, :49]), dict(temperature=-1.0), dict(temperature=math.inf),
             dict(temperature=math.nan), dict(temperature=torch.ones(3, device=DEV)), dict(target=s["target"].cpu()),
             dict(tokens=s["tokens"].cpu()), dict(tokens=s["tokens"][None])]
    wrong = [dict(target=s["target"].double()), dict(tokens=s["tokens"].float()), dict(offsets=s["offsets"].int()),
             dict(accept=s["accept"].double()), dict(sample=s["sample"].half()), dict(draft=s["draft"].half()),
             dict(temperature=torch.ones(2, device=DEV, dtype=torch.float64)), dict(temperature="1")]
    for error, cases in ((ValueError, value), (TypeError, wrong)):
        for c in cases:
            a = dict(s, **c)
            with pytest.raises(error):
                st.verify_drafts(a["target"], a["tokens"], a["offsets"], a["accept"], a["sample"],
                                 draft_logits=a["draft"], temperature=a["temperature"])
