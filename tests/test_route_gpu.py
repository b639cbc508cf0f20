"""The router's selection and its gradient against a plain implementation in 64 bits.

Weights are rounded once to 32 bits.  Where the softmax is over all experts and scores
are compared as logits, its sum is made of exponentials in 32 bits: each is off by two
steps and by the rounding of its exponent, up to 16 of them are added up in 32 bits.
"""
import math

import pytest
import torch

import segmented_top_selection_amd as st

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24  # half a step of 32 bits
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def logits_of(g, tokens, experts, dtype, ruled=0.0):
    x = 1.5 * torch.randn(tokens, experts, generator=g, device=DEV)
    if ruled:
        x = torch.where(torch.rand(tokens, experts, generator=g, device=DEV) < ruled, -math.inf, x)
    return x.to(dtype)


def scores_of(x, scoring):
    x = x.double()
    if scoring == "sigmoid":
        return torch.sigmoid(x)
    return torch.softmax(x, 1).nan_to_num(0.0)


def plain_choice(x, k, scoring, bias, groups, kept, best):
    """The experts chosen, one token after the other, on the host."""
    score = scores_of(x, scoring).cpu()
    if bias is not None:
        score = score + bias.double().cpu()
    score = torch.where(x.cpu() == -math.inf, -math.inf, score)
    size = score.shape[1] // groups
    out = []
    for row in score.tolist():
        values = []
        for g in range(groups):
            top = sorted((v for v in row[g * size:(g + 1) * size] if v > -math.inf), reverse=True)
            values.append(sum(top[:best]) if top else -math.inf)
        stay = sorted(range(groups), key=lambda g: (-values[g], g))[:kept]
        free = [e for e, v in enumerate(row) if v > -math.inf and e // size in stay]
        free.sort(key=lambda e: (-row[e], e))
        out.append((free + [-1] * k)[:k])
    return torch.tensor(out, dtype=torch.int32, device=x.device).reshape(-1, k)


def plain_weights(x, experts, scoring, renormalize, scale):
    none = experts < 0
    at = experts.clamp(min=0).long()
    if scoring == "sigmoid":
        # By logarithms where they are renormalized: sigmoids may underflow.
        log = torch.nn.functional.logsigmoid(x.double()).gather(1, at)
    else:
        log = torch.log_softmax(x.double(), 1).gather(1, at)
    log = torch.where(none, -math.inf, log)
    w = (torch.softmax(log, 1) if renormalize else log.exp()).nan_to_num(0.0)
    return torch.where(none, 0.0, w * scale)


def spread(x):
    """How far the exponents of a softmax are from zero on average, by probability."""
    x = x.double()
    d = (x.amax(1, keepdim=True) - x).nan_to_num(0.0, 0.0)
    return (torch.softmax(x, 1).nan_to_num(0.0) * d).sum(1, keepdim=True)


def check(x, k, *, scoring="softmax", bias=None, groups=1, kept=None, best=2, renormalize=True,
          scale=1.0, **kw):
    kept = groups if kept is None else kept
    w, e = st.route(x, k, scoring=scoring, bias=bias, groups=groups, kept_groups=kept,
                    group_best=best, renormalize=renormalize, scale=scale, **kw)
    torch.cuda.synchronize()
    assert w.dtype == torch.float32 and e.dtype == torch.int32
    assert w.shape == e.shape == (x.shape[0], k)
    assert torch.equal(e, plain_choice(x, k, scoring, bias, groups, kept, best))
    want = plain_weights(x, e, scoring, renormalize, scale)
    off = 1.01 + (0.0 if renormalize or scoring == "sigmoid" else 20.0 + spread(x))
    assert bool(((w.double() - want).abs() <= off * U * want.abs() + 2.0 ** -149).all())
    return w, e


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("experts,k", [(1, 1), (2, 2), (8, 2), (60, 6), (64, 8), (65, 8), (128, 8),
                                       (200, 64), (256, 8), (257, 3), (512, 16), (1000, 10),
                                       (1024, 64)])
def test_route(experts, k, biased, scoring, dtype):
    g = gen(experts + k)
    x = logits_of(g, 37, experts, dtype)
    bias = 0.1 * torch.randn(experts, generator=g, device=DEV) if biased else None
    for renormalize in (False, True):
        check(x, k, scoring=scoring, bias=bias, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("experts,groups,kept,k", [(256, 8, 4, 8), (64, 4, 1, 8), (60, 4, 2, 6),
                                                   (60, 60, 7, 7), (64, 64, 9, 9), (200, 5, 2, 33),
                                                   (1024, 16, 3, 20), (1000, 40, 3, 20), (24, 3, 3, 5),
                                                   (960, 15, 14, 64), (8, 4, 2, 4)])
def test_groups(experts, groups, kept, k, best, scoring):
    g = gen(experts + groups + kept)
    for dtype, biased in ((torch.float32, True), (torch.bfloat16, False)):
        x = logits_of(g, 33, experts, dtype)
        bias = 0.1 * torch.randn(experts, generator=g, device=DEV) if biased else None
        check(x, k, scoring=scoring, bias=bias, groups=groups, kept=kept, best=best)


@pytest.mark.parametrize("tokens", [0, 1, 3, 4, 5, 63, 1000])
def test_tokens(tokens):
    g = gen(tokens)
    check(logits_of(g, tokens, 64, torch.float32), 8)
    check(logits_of(g, tokens, 300, torch.float16), 8)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_experts_ruled_out(groups, kept, scoring):
    g = gen(5)
    x = logits_of(g, 300, 40, torch.float32, ruled=0.8)
    x[7] = -math.inf
    x[8, 1:] = -math.inf
    bias = 0.2 * torch.randn(40, generator=g, device=DEV)
    for b in (None, bias):
        for renormalize in (False, True):
            w, e = check(x, 8, scoring=scoring, bias=b, groups=groups, kept=kept,
                         renormalize=renormalize)
            assert bool((e[7] == -1).all()) and bool((w[7] == 0).all())
    assert e[8].tolist() == [0 if x[8, 0] > -math.inf else -1] + [-1] * 7
    # By the bias, for all tokens.
    bias[3:] = -math.inf
    _, e = st.route(torch.zeros(5, 40, device=DEV), 6, bias=bias, scoring=scoring)
    assert bool((e[:, 3:] == -1).all()) and bool((e[:, :3].sort(1).values == torch.arange(3, device=DEV)).all())


def test_ties_go_to_the_lower_index():
    x = torch.zeros(9, 96, device=DEV, dtype=torch.bfloat16)
    for kw in (dict(), dict(bias=torch.full((96,), 0.25, device=DEV)), dict(scoring="sigmoid"),
               dict(groups=6, kept=2), dict(groups=6, kept=2, best=1, scoring="sigmoid")):
        _, e = check(x, 20, **kw)
        assert e[0].tolist() == list(range(20))
    # Coarse logits: many equal ones, and biases of a few steps.
    g = gen(8)
    x = torch.randint(-3, 4, (200, 128), generator=g, device=DEV).half()
    bias = torch.randint(-2, 3, (128,), generator=g, device=DEV) * 0.001
    check(x, 8)
    check(x, 8, bias=bias, scoring="sigmoid")
    check(x, 8, bias=bias, scoring="sigmoid", groups=8, kept=3)


def test_neighbours_that_32_bits_would_swap():
    # Scores that differ by 1e-9: equal in 32 bits, of which the lower index would be taken.
    x = torch.zeros(64, 64, device=DEV)
    bias = torch.zeros(64, device=DEV)
    at = torch.arange(64, device=DEV)
    x[at, at] = 4e-9  # the sigmoid's slope is a quarter
    for scoring in ("sigmoid", "softmax"):
        w, e = check(x, 2, scoring=scoring, bias=bias)
        assert e[:, 0].tolist() == list(range(64))


def test_far_logits():
    lowest = torch.finfo(torch.float32).min
    x = torch.tensor([[lowest] * 8, [1e38, lowest, 0, 1, 2, 3, 4, 5], [-200.0 - i for i in range(8)],
                      [800.0 + i for i in range(8)], [0, 0, 0, 0, lowest, lowest, lowest, lowest]], device=DEV)
    for kw in (dict(), dict(renormalize=False), dict(scoring="sigmoid"),
               dict(scoring="sigmoid", renormalize=False)):
        w, got = st.route(x, 5, **kw)
        assert bool(torch.isfinite(w).all())
        # By the logits: probabilities this far apart underflow in 64 bits too.
        e = x.sort(dim=1, descending=True, stable=True).indices[:, :5].int()
        assert torch.equal(got, e)
        want = plain_weights(x, e, kw.get("scoring", "softmax"), kw.get("renormalize", True), 1.0)
        off = (22.0 + spread(x)) * U
        assert bool(((w.double() - want).abs() <= off * want + 2.0 ** -126).all())


# Ranges of scores that no finite factor spreads over the keys' whole numbers, and some above.
@pytest.mark.parametrize("size", [1e-45, 1e-42, 1.2e-38, 1e-36, 1e-33, 1e-31, 1e-29, 1e-20, 1e-9])
@pytest.mark.parametrize("experts", [60, 64, 256, 512, 1000])
def test_logits_that_lie_close_together(experts, size):
    g = gen(experts)
    rows = [torch.randint(-1000, 1001, (9, experts), generator=g, device=DEV) * size,  # far and near
            torch.randint(-4, 5, (9, experts), generator=g, device=DEV) * size,        # equal ones
            torch.zeros(9, experts, device=DEV), torch.zeros(2, experts, device=DEV)]
    rows[2][torch.arange(9), torch.arange(9) * 6] = size  # one above the others, and below
    rows[3][0, -1], rows[3][1, 3] = size, -size
    rows.append(logits_of(g, 9, experts, torch.float32))  # in the same waves
    x = torch.cat(rows)[torch.randperm(38, generator=g, device=DEV)]
    want = x.cpu().double().sort(dim=1, descending=True, stable=True).indices.int()
    for k in (1, 8, 60):
        for scoring in ("softmax", "sigmoid"):
            w, e = st.route(x, k, scoring=scoring)
            assert torch.equal(e.cpu(), want[:, :k])
            plain = plain_weights(x, e, scoring, True, 1.0)
            assert bool(((w.double() - plain).abs() <= 1.01 * U * plain).all())
    # One expert ruled out: none of the others is.
    x[:, 5] = -math.inf
    _, e = st.route(x, 59)
    assert torch.equal(e.cpu(), x.cpu().double().sort(dim=1, descending=True, stable=True).indices[:, :59].int())


@pytest.mark.parametrize("experts,groups,kept", [(60, 1, 1), (64, 1, 1), (256, 8, 3), (200, 5, 2), (512, 1, 1)])
def test_sigmoids_that_lie_close_together(experts, groups, kept):
    g = gen(experts + 1)
    x = -88 + 16 * torch.rand(30, experts, generator=g, device=DEV)
    x[:5] = -104 + torch.rand(5, experts, generator=g, device=DEV)  # nothing in 32 bits
    for bias in (torch.zeros(experts, device=DEV), 1e-40 * torch.randn(experts, generator=g, device=DEV)):
        for k in (1, 8, 32):
            check(x, k, scoring="sigmoid", bias=bias, groups=groups, kept=kept)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("experts", [16, 240, 1024])
def test_groups_of_nan(experts, dtype):
    # A NaN is the lowest score that is not ruled out, and so are two: its group has experts left.
    size, none, nan = experts // 4, -math.inf, math.nan
    x = torch.full((6, 4, size), none)
    x[0, 1] = x[0, 3] = nan                    # two groups of NaN next to two that are ruled out
    x[1, 3] = nan
    x[2, 2, 1] = nan                           # one NaN alone
    x[3, 0], x[3, 2, :2] = nan, torch.tensor([nan, -3.0])  # a number and a NaN before two NaN
    x[4, 0], x[4, 1], x[4, 3] = nan, -9.0, 2.0
    x[5, 1:3] = nan
    first = [[size, size + 1], [3 * size, 3 * size + 1], [2 * size + 1, -1],
             [2 * size + 1, 2 * size], [3 * size, 3 * size + 1], [size, size + 1]]
    x = x.view(6, experts).to(DEV, dtype)
    for bias in (None, torch.zeros(experts, device=DEV)):
        for best in (1, 2):
            _, e = st.route(x, 2, scoring="sigmoid", bias=bias, groups=4, kept_groups=1, group_best=best)
            assert e.tolist() == first
            _, e = st.route(x, 2, scoring="sigmoid", bias=bias, groups=4, kept_groups=3, group_best=best)
            assert bool((e[:, 0] >= 0).all()) and bool((e[[0, 1, 3, 4, 5], 1] >= 0).all())


def test_groups_of_biases_whose_sums_leave_32_bits():
    x = torch.randn(9, 32, generator=gen(21), device=DEV)
    far = [[3e38, 3e38, 0, 0], [3.2e38, 3.1e38, 0, 0], [0, 0, 0, 0], [3.3e38, 0, 1, 2],
           [-3.1e38, -3.2e38, -3.3e38, -3.4e38], [-3e38] * 4, [-math.inf] * 4, [-3.05e38, -math.inf, 0, 0]]
    # Apart from each other, so that nothing but the groups' sums is in doubt.
    above = [[3e38 - 1e36 * i, 2e38 + 1.1e37 * (i % 3) + 2e35 * i, 1e38 - 1e36 * i, 1e37 - 1e36 * i]
             for i in range(8)]
    below = [[-1.8e38 - 1e36 * i, -2e38 - 1.1e37 * (i % 3) - 2e35 * i, -3e38 - 1e36 * i, -3.2e38 - 1e36 * i]
             for i in range(7)] + [[0, -1e37, -2e37, -3e37]]
    order = torch.randperm(8, generator=gen(22), device=DEV).tolist()
    for groups in (far, far[::-1], [far[i] for i in order], far[4:7] * 2 + far[4:6], far[4:7][::-1] * 2 + far[4:6],
                   above, above[::-1], below, below[::-1], [below[i] for i in order]):
        bias = torch.tensor(groups, device=DEV).view(32)
        for kept in (1, 2, 3):
            for scoring in ("sigmoid", "softmax"):
                check(x, 4 * kept, scoring=scoring, bias=bias, groups=8, kept=kept)
                check(x, 4, scoring=scoring, bias=bias, groups=8, kept=kept, best=1)


def test_groups_by_an_infinite_logit():
    most = torch.finfo(torch.float32).max
    x = torch.tensor([[most, 0, 1, 2, math.inf, 3, 4, 5, -most, -1, -2, -3]], device=DEV)
    for kept, want in ((1, [4, 7, 6, 5]), (2, [4, 0, 7, 6])):
        _, e = st.route(x, 4, scoring="sigmoid", groups=3, kept_groups=kept, group_best=1)
        assert e[0].tolist() == want
    # The same by a bias, where sums of two are compared.
    bias = x[0].clone()
    for best in (1, 2):
        _, e = st.route(torch.zeros_like(x), 4, bias=bias, scoring="sigmoid", groups=3, kept_groups=1, group_best=best)
        assert e[0].tolist() == [4, 7, 6, 5]


def test_nan_and_inf():
    x = torch.randn(6, 32, generator=gen(1), device=DEV)
    x[0, 3], x[1, 0], x[2, 5] = math.nan, math.inf, math.nan
    for bias in (None, torch.zeros(32, device=DEV)):
        for renormalize in (False, True):
            w, e = st.route(x, 4, bias=bias, renormalize=renormalize)
            assert bool(w[:3].isnan().all()) and not bool(w[3:].isnan().any())
            assert bool(((e >= 0) & (e < 32)).all())
            w, e = st.route(x, 4, bias=bias, renormalize=renormalize, scoring="sigmoid")
            assert not bool(w.isnan().any()) and e[1, 0] == 0
            assert bool(((e >= 0) & (e < 32)).all())
    d = st.route_backward(torch.ones(6, 4, device=DEV), x, e, renormalize=False)
    assert bool(d[0].isnan().all()) and not bool(d[3:].isnan().any())


def test_strides_and_streams():
    g = gen(3)
    wide = logits_of(g, 50, 200, torch.bfloat16)
    check(wide[:, 3:100], 5)
    check(wide.t()[:64].t(), 5)
    check(wide[:1, 7:8].expand(9, 1), 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(wide[:, 1:65], 5, stream=side)


# --------------------------------------------------------------------------
def plain_gradient(dw, x, e, scoring, renormalize, scale):
    """(the gradient, the magnitudes whose sum it is), in 64 bits."""
    none = (e < 0) | (e >= x.shape[1])
    at = torch.where(none, 0, e).long()
    g = torch.where(none, 0.0, dw.double() * scale)
    x = x.double()
    p = torch.softmax(x, 1).nan_to_num(0.0) if scoring == "softmax" else torch.sigmoid(x)
    own = torch.where(none, 0.0, p.gather(1, at))
    if scoring == "softmax" and not renormalize:
        common = p * (own * g).sum(1, keepdim=True)
        direct = torch.zeros_like(p).scatter_add_(1, at, own * g)
        size = p * (own * g).abs().sum(1, keepdim=True) + direct.abs()
        return direct - common, size
    d = torch.where(none, 0.0, g)
    if renormalize:
        u = plain_weights(x, torch.where(none, -1, e), scoring, True, 1.0)
        size = u * (g.abs() + (u * g.abs()).sum(1, keepdim=True))
        d = u * (g - (u * g).sum(1, keepdim=True))
        if scoring == "sigmoid":
            d, size = d * (1 - own), size * (1 - own)
    else:
        d = g * own * (1 - own)
        size = d.abs()
    zero = torch.zeros_like(p)
    return (zero.scatter_add(1, at, torch.where(none, 0.0, d)),
            zero.scatter_add(1, at, torch.where(none, 0.0, size)))


def check_gradient(dw, x, e, scoring, renormalize, scale, **kw):
    d = st.route_backward(dw, x, e, scoring=scoring, renormalize=renormalize, scale=scale, **kw)
    torch.cuda.synchronize()
    assert d.dtype == x.dtype and d.shape == x.shape
    want, size = plain_gradient(dw, x, e, scoring, renormalize, scale)
    inner = 4.0 * U * size  # rounded to 32 bits, added up, rounded
    if scoring == "softmax" and not renormalize:
        inner = inner + (x.shape[1] / 64 + 6 + spread(x)) * U * size
    eps = torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -126
    bound = eps * (want.abs() + inner) + inner + tiny
    assert bool(((d.double() - want).abs() <= bound).all())
    return d


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (5, 8, 2), (37, 60, 6), (100, 128, 8),
                                              (3, 1000, 64), (0, 8, 2), (9, 65, 64)])
def test_gradient(tokens, experts, k, renormalize, scoring, dtype):
    g = gen(tokens + experts)
    x = logits_of(g, tokens, experts, dtype, ruled=0.1 if experts > 8 else 0.0)
    _, e = st.route(x, k, scoring=scoring)
    dw = torch.randn(tokens, k, generator=g, device=DEV)
    dw[e < 0] = math.nan  # of slots without an expert: anything
    check_gradient(dw, x, e, scoring, renormalize, 1.5)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("experts,k", [(2, 1), (64, 1), (64, 8), (200, 3), (1000, 64)])
def test_gradient_of_a_confident_router(experts, k, dtype):
    # One expert far above the others: its gradient p (g - <g, p>) is g p times what little is
    # left for the others.
    g = gen(experts + k)
    gap = torch.tensor([4.0, 8.0, 12.0, 16.0, 20.0, 24.0], device=DEV)[:, None]
    x = torch.rand(6, experts, generator=g, device=DEV) - gap
    at = torch.randint(0, experts, (6, 1), generator=g, device=DEV)
    x = x.scatter_(1, at, 0.0).to(dtype)
    _, e = st.route(x, k, renormalize=False)
    assert torch.equal(e[:, :1].long(), at)
    dw = torch.randn(6, k, generator=g, device=DEV)
    dw[:, 0] += 3.0
    d = st.route_backward(dw, x, e, renormalize=False, scale=1.5).double()
    # g - <g, p> as the sum of p_j (g - g_j), which leaves nothing to cancel but g - g_j.
    p = torch.softmax(x.double(), 1)
    full = torch.zeros_like(p).scatter_(1, e.long(), 1.5 * dw.double())
    want = p * (p[:, None, :] * (full[:, :, None] - full[:, None, :])).sum(2)
    # In 64 bits: the softmax's sum, the mean and the difference, each of the size of g.
    size = p * (full.abs() + (p * full.abs()).sum(1, keepdim=True))
    inner = (experts / 64 + 12) * 2.0 ** -53 * size + 2.0 ** -48 * want.abs()
    eps = torch.finfo(dtype).eps / 2 + U  # by way of 32 bits
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133
    assert bool(((d - want).abs() <= eps * want.abs() + 2 * inner + tiny).all())


def test_gradient_slots_that_are_odd():
    g = gen(6)
    x = logits_of(g, 20, 16, torch.float32)
    e = torch.randint(-3, 20, (20, 5), generator=g, device=DEV).int()  # outside, and the same twice
    dw = torch.randn(20, 5, generator=g, device=DEV)
    check_gradient(dw, x, e, "softmax", False, 1.0)
    check_gradient(dw, x, e, "sigmoid", False, 1.0)
    out = torch.full((20, 40), 7.0, device=DEV)
    d = check_gradient(dw, x, e, "softmax", False, 1.0, out=out[:, 3:19])
    assert d.data_ptr() == out[:, 3:19].data_ptr()
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 19:] == 7).all())
    x[3] = -math.inf
    assert bool((st.route_backward(dw, x, e, renormalize=False)[3] == 0).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences(renormalize, scoring):
    g = gen(11)
    x = logits_of(g, 6, 12, torch.float32)
    w, e = st.route(x, 4, scoring=scoring, renormalize=renormalize)
    dw = torch.randn(6, 4, generator=g, device=DEV)
    d = st.route_backward(dw, x, e, scoring=scoring, renormalize=renormalize)
    h = 1e-5
    for c in range(12):
        step = torch.zeros(12, device=DEV, dtype=torch.float64)
        step[c] = h
        hi, lo = ((plain_weights(x.double() + s * step, e, scoring, renormalize, 1.0) * dw).sum(1)
                  for s in (1, -1))
        # Central differences: h^2 times a third derivative of at most 6 |dw| in sum, and rounding.
        bound = 6 * h * h * dw.abs().sum(1).double() + 1e-15 / h * dw.abs().sum(1) + 4 * U * dw.abs().sum(1)
        assert bool((((hi - lo) / (2 * h) - d[:, c].double()).abs() <= bound).all())


def test_graph():
    g = gen(2)
    x = logits_of(g, 64, 64, torch.bfloat16)
    bias = 0.1 * torch.randn(64, generator=g, device=DEV)
    dw = torch.randn(64, 8, generator=g, device=DEV)
    run = lambda: (*st.route(x, 8, bias=bias, groups=8, kept_groups=3), )  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w, e = run()
        d = st.route_backward(dw, x, e)
    for i in range(3):
        x.copy_(logits_of(g, 64, 64, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        w2, e2 = run()
        assert torch.equal(w, w2) and torch.equal(e, e2)
        assert torch.equal(d, st.route_backward(dw, x, e2))


def test_refusals():
    x = torch.zeros(4, 12, device=DEV)
    for kw in (dict(k=0), dict(k=13), dict(k=2, groups=5), dict(k=2, groups=0), dict(k=2, groups=4, kept_groups=5),
               dict(k=4, groups=4, kept_groups=1), dict(k=2, groups=4, kept_groups=0),
               dict(k=2, group_best=3), dict(k=2, scoring="tanh"), dict(k=2, bias=torch.zeros(11, device=DEV)),
               dict(k=2, bias=torch.zeros(12))):
        with pytest.raises(ValueError):
            st.route(x, **kw)
    with pytest.raises(ValueError):
        st.route(torch.zeros(4, 1025, device=DEV), 2)
    with pytest.raises(ValueError):
        st.route(torch.zeros(4, 100, device=DEV), 65)
    for kw in (dict(k=2.5), dict(k=2, bias=torch.zeros(12, device=DEV, dtype=torch.float64))):
        with pytest.raises(TypeError):
            st.route(x, **kw)
    with pytest.raises(TypeError):
        st.route(x.double(), 2)
    with pytest.raises(st.SegTopKError):
        st.route(x, 2, scale=math.inf)
    e, dw = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    for bad in (dict(e=e[:3]), dict(dw=dw[:, :1]), dict(e=e[:, :0], dw=dw[:, :0])):
        with pytest.raises(ValueError):
            st.route_backward(bad.get("dw", dw), x, bad.get("e", e))
    with pytest.raises(TypeError):
        st.route_backward(dw, x, e.long())
    with pytest.raises(TypeError):
        st.route_backward(dw.half(), x, e)
    with pytest.raises(TypeError):
        st.route_backward(dw, x, e, out=torch.empty(4, 12, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError):
        st.route_backward(dw, x, e, out=torch.empty(4, 11, device=DEV))
