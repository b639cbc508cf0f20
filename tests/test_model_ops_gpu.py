"""The operators around the selection against plain implementations in 64 bits.

Tolerances are counted, not tried.  A value rounded once to type t is off by
half a step at most: eps(t) / 2 of it (and half the smallest subnormal of f16).
A sum of n products in 32 bits is off by at most (n + 1) * 2^-24 of the sum of
their magnitudes.  Integers and copies are equal.
"""
import math

import numpy as np
import pytest
import torch

import segmented_top_selection_amd as st

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24  # half a step of 32 bits
TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16",
       torch.int32: "i32", torch.int64: "i64"}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def half_step(t, exact):
    return torch.finfo(t).eps / 2 * exact.abs() + (2.0 ** -25 if t == torch.float16 else 2.0 ** -149)


def close(got, exact, inner=0.0):
    """got is exact, off by `inner` before it was rounded to its type."""
    e = exact.double()
    bound = half_step(got.dtype, e.abs() + inner) + inner
    err = (got.double() - e).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= bound).all()), f"off by {float((err / bound).max()):.3g} of the bound"


# --------------------------------------------------------------------------
# sort_ids
# --------------------------------------------------------------------------
def plain_sort(ids, segments):
    key = ids.reshape(-1).cpu().numpy().astype(np.int64)
    key = np.where((key >= 0) & (key < segments), key, segments)
    order = np.argsort(key, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(order.size)
    offsets = np.searchsorted(key[order], np.arange(segments + 1))
    return order, position, offsets


def check_sort(ids, segments, **kw):
    order, position, offsets = st.sort_ids(ids, segments, **kw)
    torch.cuda.synchronize()
    eo, ep, ef = plain_sort(ids, segments)
    assert order.dtype == position.dtype == torch.int32 and offsets.dtype == torch.int64
    assert position.shape == ids.shape
    assert np.array_equal(order.cpu().numpy(), eo)
    assert np.array_equal(position.reshape(-1).cpu().numpy(), ep)
    assert np.array_equal(offsets.cpu().numpy(), ef)
    return order, position, offsets


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=IDS.get)
@pytest.mark.parametrize("segments", [1, 2, 37, 64, 128, 511, 512, 4099, 131072, 300001])
@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 1000, 1025, 8191, 8192, 8193, 33333])
def test_sort_ids(n, segments, dtype):
    g = gen(n * 7 + segments)
    ids = torch.randint(-2, segments + 2, (n,), generator=g, device=DEV).to(dtype)
    check_sort(ids, segments)


@pytest.mark.parametrize("what", ["same", "last", "dropped", "descending", "skewed"])
@pytest.mark.parametrize("n,segments", [(3000, 128), (8000, 5000), (300000, 128), (70001, 100000)])
def test_sort_ids_orders(what, n, segments):
    i = torch.arange(n, device=DEV)
    ids = {"same": i * 0 + 3, "last": i * 0 + segments - 1, "dropped": i * 0 - 1,
           "descending": (n - 1 - i) * segments // n,
           "skewed": torch.where(i % 17 == 0, i % segments, 5)}[what]
    check_sort(ids, segments)


def test_sort_ids_large_and_far_ids():
    g = gen(3)
    check_sort(torch.randint(0, 256, (1 << 20, 3), generator=g, device=DEV), 256)  # blocks in turn
    check_sort(torch.randint(0, 70000, (3 * (1 << 20) + 77,), generator=g, device=DEV), 70000)
    # 64-bit ids whose low 32 bits look like segments are outside.
    ids = torch.tensor([2 ** 32 + 1, 1, -2 ** 32 + 1, 2 ** 62, 0, 1, -2 ** 63], device=DEV)
    check_sort(ids, 4)
    check_sort(torch.randint(0, 1 << 28, (50000,), generator=g, device=DEV), 1 << 28)
    check_sort(torch.randint(0, 9, (50, 7), generator=g, device=DEV).t(), 9)


def test_sorted_offsets_serve_as_segments_of_the_selection():
    g = gen(4)
    ids = torch.randint(0, 12, (5000,), generator=g, device=DEV)
    order, _, offsets = st.sort_ids(ids, 12)
    scores = randn(g, 5000)
    top, _ = st.batched_topk(scores[order.long()].contiguous(), offsets, 5)
    for e in range(12):
        mine = scores[ids == e]
        assert torch.equal(top[e, :min(5, mine.numel())], mine.sort(descending=True).values[:5])


# --------------------------------------------------------------------------
# dispatch, combine and their gradients
# --------------------------------------------------------------------------
def slots(g, tokens, k, experts, dropped):
    ids = torch.stack([torch.randperm(experts, generator=g, device=DEV)[:k] for _ in range(tokens)]) \
        if tokens else torch.zeros(0, k, dtype=torch.int64, device=DEV)
    if dropped:
        ids = torch.where(torch.rand(tokens, k, generator=g, device=DEV) < dropped, -1, ids)
    _, position, offsets = st.sort_ids(ids, experts)
    return ids, position, offsets


SHAPES = [(1, 1, 1), (1, 2, 8), (3, 1, 7), (5, 8, 64), (2, 9, 100), (33, 3, 1001), (17, 6, 1410),
          (64, 2, 2048), (7, 17, 4104), (300, 4, 33)]


def move_all(g, tokens, k, width, dtype, wdtype, dropped, pad=0):
    """Every move over one set of slots, checked; rows `pad` elements apart."""
    def matrix(rows):
        return randn(g, rows, width + pad, dtype=dtype)[:, pad:]
    experts = max(k, 9)
    ids, position, offsets = slots(g, tokens, k, experts, dropped)
    n, kept = tokens * k, ids.reshape(-1) >= 0
    p = position.reshape(-1).long()
    x, y, dout = matrix(tokens), matrix(n), matrix(tokens)
    w = torch.rand(tokens, k, generator=g, device=DEV).to(wdtype) if wdtype else None
    wx = w.double() if wdtype else torch.ones(tokens, k, dtype=torch.float64, device=DEV)
    live = kept.view(tokens, k)
    # Rows of dropped slots may hold anything.
    y[p[~kept]] = float("nan")

    rows = st.dispatch(x, position, offsets)
    expect = torch.zeros(n, width, dtype=dtype, device=DEV)
    expect[p[kept]] = x.repeat_interleave(k, 0)[kept]
    assert torch.equal(rows, expect)

    yd = torch.where(live[:, :, None], y[p].view(tokens, k, width).double(), 0.0)
    exact = (yd * wx[:, :, None]).sum(1)
    out = st.combine(y, position, offsets, w)
    close(out, exact, (k + 1) * U * (yd * wx[:, :, None]).abs().sum(1))

    dx = st.dispatch_backward(y, position, offsets)
    close(dx, yd.sum(1), (k + 1) * U * yd.abs().sum(1))

    dy, dw = st.combine_backward(dout, y, position, offsets, w)
    dd = dout.double()[:, None, :]
    exact = torch.zeros(n, width, dtype=torch.float64, device=DEV)
    exact[p] = (dd * (wx * live)[:, :, None]).reshape(n, width)
    close(dy, exact, 2 * U * exact.abs())
    assert dw.dtype == (wdtype or torch.float32) and dw.shape == position.shape
    close(dw, (dd * yd).sum(2), (width + 1) * U * (dd * yd).abs().sum(2))
    again, none = st.combine_backward(dout, None, position, offsets, w)
    assert none is None and torch.equal(again, dy)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("tokens,k,width", SHAPES)
def test_rows_moved(tokens, k, width, dtype):
    g = gen(tokens * 100 + width)
    for wdtype, dropped in ((torch.float32, 0.0), (dtype, 0.3), (None, 0.3)):
        move_all(g, tokens, k, width, dtype, wdtype, dropped)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_rows_moved_between_slices_of_wider_rows(dtype, pad):
    move_all(gen(pad), 21, 4, 515, dtype, torch.float32, 0.2, pad)


@pytest.mark.parametrize("tokens,dropped", [(0, 0.0), (40, 1.1)])
def test_no_tokens_and_no_kept_slots(tokens, dropped):
    move_all(gen(5), tokens, 3, 70, torch.bfloat16, torch.float32, dropped)


def test_other_layouts_are_copied_and_outputs_taken():
    g = gen(6)
    ids, position, offsets = slots(g, 24, 2, 9, 0.1)
    x = randn(g, 64, 24).t()  # columns far apart
    rows = st.dispatch(x, position, offsets)
    assert torch.equal(rows, st.dispatch(x.contiguous(), position, offsets))
    one = randn(g, 1, 64).expand(24, 64)  # one row for all, as a broadcast's gradient
    assert torch.equal(st.dispatch(one, position, offsets), st.dispatch(one.contiguous(), position, offsets))
    wide = torch.full((48, 80), 7.0, device=DEV)
    out = wide[:, 8:72]
    assert st.dispatch(x, position, offsets, out=out) is out
    assert torch.equal(out, rows) and bool((wide[:, :8] == 7).all()) and bool((wide[:, 72:] == 7).all())
    w = torch.rand(2, 24, generator=g, device=DEV).t()
    assert torch.equal(st.combine(rows, position, offsets, w),
                       st.combine(rows, position, offsets, w.contiguous()))
    # One slot a token, without a second dimension; no offsets: all kept.
    p = torch.randperm(24, generator=g, device=DEV).int()
    assert torch.equal(st.combine(st.dispatch(x, p), p), x)


def test_positions_outside_the_rows_are_skipped():
    x = randn(gen(7), 3, 40)
    position = torch.tensor([[0, -5], [2 ** 31 - 1, 4], [6, 1]], dtype=torch.int32, device=DEV)
    out = torch.full((6, 40), 5.0, device=DEV)
    st.dispatch(x, position, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[4], x[1]) and torch.equal(out[1], x[2])
    assert bool((out[[2, 3, 5]] == 5).all())
    back = st.combine(out, position)
    assert torch.equal(back, x)
    drows, dw = st.combine_backward(x, out, position, out=torch.full((6, 40), 5.0, device=DEV))
    assert torch.equal(drows, out)
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and dw[2, 0] == 0
    # A count outside the rows is cut to them.
    far = torch.tensor([0, 100], device=DEV)
    assert torch.equal(st.combine(out, position, far), x)
    assert bool((st.combine(out, position, -far) == 0).all())


def test_gradients_of_the_moves_against_differences():
    # Loss L = <c, combine(y, w)> is linear in y and in w: a difference of it in
    # 64 bits is exact up to its own rounding, and the gradient at dout = c has
    # to equal it up to the 32-bit sums.
    g = gen(8)
    tokens, k, width = 9, 3, 20
    ids, position, offsets = slots(g, tokens, k, 5, 0.2)
    y, c = randn(g, tokens * k, width), randn(g, tokens, width)
    w = torch.rand(tokens, k, generator=g, device=DEV)
    dy, dw = st.combine_backward(c, y, position, offsets, w)
    live = (ids >= 0).double()

    def loss(y, w):
        return ((y[position.long()] * (w * live)[:, :, None]).sum(1) * c.double()).sum()
    for t in range(0, tokens, 2):
        for j in range(k):
            e = torch.zeros(tokens, k, dtype=torch.float64, device=DEV)
            e[t, j] = 0.5
            d = loss(y.double(), w.double() + e) - loss(y.double(), w.double() - e)
            assert abs(float(d) - float(dw[t, j])) <= (width + 2) * U * float(
                (c[t].double() * y[position[t, j]].double()).abs().sum()) + 1e-12
            h = torch.zeros(tokens * k, width, dtype=torch.float64, device=DEV)
            h[position[t, j], 7] = 0.5
            d = loss(y.double() + h, w.double()) - loss(y.double() - h, w.double())
            assert abs(float(d) - float(dy[position[t, j], 7])) <= 2 * U * abs(float(d)) + 1e-12


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("n,num_rows,width", [(1, 1, 1), (1, 5, 4096), (64, 1000, 257), (333, 50, 64),
                                              (1000, 7, 1001), (4, 9, 8200)])
def test_embedding(n, num_rows, width, dtype):
    g = gen(n + width)
    table = randn(g, num_rows, width, dtype=dtype)
    for idtype in (torch.int32, torch.int64):
        ids = torch.randint(-1, num_rows + 1, (n,), generator=g, device=DEV).to(idtype)
        there = (ids >= 0) & (ids < num_rows)
        exact = table[ids.long().clamp(0, num_rows - 1)].double() * there[:, None]
        out = st.embedding(table, ids)
        assert torch.equal(out.double(), exact)
        scale = float(np.float32(math.sqrt(width)))
        close(st.embedding(table, ids, scale=scale), exact * scale, U * (exact * scale).abs())


def test_embedding_shapes_and_slices():
    g = gen(10)
    table = randn(g, 30, 75, dtype=torch.bfloat16)[:, 3:70]
    ids = torch.randint(0, 30, (4, 6), generator=g, device=DEV)
    assert torch.equal(st.embedding(table, ids), table[ids])
    assert torch.equal(st.embedding(table, ids.t()), table[ids.t()])
    assert st.embedding(table, ids[:0]).shape == (0, 6, 67)
    assert bool((st.embedding(table[:0], ids) == 0).all())
    out = torch.empty(24, 100, dtype=torch.bfloat16, device=DEV)[:, :67]
    assert st.embedding(table, ids, out=out) is out and torch.equal(out, table[ids.view(-1)])


def exact_table(dout, ids, num_rows, padding=None):
    ids = ids.reshape(-1).long()
    ok = (ids >= 0) & (ids < num_rows)
    if padding is not None:
        ok &= ids != padding
    d = torch.zeros(num_rows, dout.shape[1], dtype=torch.float64, device=DEV)
    mag, cnt = d.clone(), torch.zeros(num_rows, dtype=torch.float64, device=DEV)
    d.index_put_((ids[ok],), dout[ok].double(), accumulate=True)
    mag.index_put_((ids[ok],), dout[ok].double().abs(), accumulate=True)
    cnt.index_put_((ids[ok],), torch.ones_like(ids[ok], dtype=torch.float64), accumulate=True)
    return d, (cnt[:, None] + 2) * U * mag, cnt > 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("n,num_rows,width", [
    (0, 5, 33), (1, 1, 1), (1, 700, 64), (31, 3, 65), (32, 3, 65), (33, 3, 65), (64, 1, 100),
    (65, 2, 4100), (500, 40, 257), (4096, 600, 40), (5000, 100000, 24), (3001, 1, 1001)])
def test_embedding_backward(n, num_rows, width, dtype):
    g = gen(n + width + num_rows)
    dout = randn(g, n, width, dtype=dtype)
    ids = torch.randint(-1, num_rows + 1, (n,), generator=g, device=DEV)
    scale = float(np.float32(math.sqrt(width)))
    exact, inner, _ = exact_table(dout, ids, num_rows)
    got = st.embedding_backward(dout, ids, num_rows, scale=scale)
    assert got.dtype == dtype
    close(got, exact * scale, inner * scale)
    assert torch.equal(got, st.embedding_backward(dout, ids.int(), num_rows, scale=scale))
    whole = st.embedding_backward(dout, ids, num_rows, dtype=torch.float32)
    close(whole, exact, inner)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("what", ["same", "borders", "skewed", "padding only"])
def test_embedding_backward_runs_over_chunks(what, dtype):
    n, num_rows, width = 1500, 90, 130
    g = gen(11)
    i = torch.arange(n, device=DEV)
    ids = {"same": i * 0 + 17, "borders": i // 48, "padding only": i * 0 + 2,
           "skewed": torch.where(i % 3 == 0, i % num_rows, 4)}[what]
    dout = randn(g, n, width, dtype=dtype)
    dout[ids == 2] = float("nan")  # the padding's gradient may hold anything
    exact, inner, touched = exact_table(dout, ids, num_rows, padding=2)
    close(st.embedding_backward(dout, ids, num_rows, padding_id=2), exact, inner)
    # Added to what is there; rows that do not occur keep their bits, NaN too.
    for odt in {dtype, torch.float32}:
        base = randn(g, num_rows, width, dtype=odt)
        base[~touched] = float("nan")
        out = base.clone()
        res = st.embedding_backward(dout, ids, num_rows, padding_id=2, out=out, accumulate=True)
        assert res is out
        bits = torch.int32 if odt == torch.float32 else torch.int16
        assert torch.equal(out[~touched].view(bits), base[~touched].view(bits))
        if bool(touched.any()):
            sum_ = (exact + base.double())[touched]
            close(out[touched], sum_, inner[touched] + U * (sum_.abs() + exact[touched].abs()))


def test_embedding_backward_layouts():
    g = gen(12)
    ids = torch.randint(0, 20, (6, 7), generator=g, device=DEV)
    dout = randn(g, 6, 7, 35)
    want = st.embedding_backward(dout, ids, 20)
    assert torch.equal(want, st.embedding_backward(dout.view(42, 35), ids.view(-1), 20))
    wide = torch.full((20, 50), 3.0, device=DEV)
    out = wide[:, 5:40]
    st.embedding_backward(dout, ids, 20, out=out)
    assert torch.equal(out, want) and bool((wide[:, :5] == 3).all()) and bool((wide[:, 40:] == 3).all())
    row = randn(g, 35)
    assert torch.equal(st.embedding_backward(row.expand(42, 35), ids, 20),
                       st.embedding_backward(row.repeat(42, 1), ids, 20))
    # Against differences: the lookup is linear in the table.
    c, scale = randn(g, 42, 35), 3.0
    got = st.embedding_backward(c, ids, 20, scale=scale)
    for v in range(20):
        e = torch.zeros(20, 35, dtype=torch.float64, device=DEV)
        e[v, v] = 1.0
        d = float((e[ids.view(-1)] * scale * c.double()).sum())
        mag = float(c[ids.view(-1) == v, v].double().abs().sum()) * scale
        assert abs(d - float(got[v, v])) <= 44 * U * mag


# --------------------------------------------------------------------------
# policy loss
# --------------------------------------------------------------------------
def exact_policy(q, kl, low, high, temperature, grad_scale=1.0):
    """(loss, logp, dlogits) in 64 bits on the CPU, and bounds on the error of
    32-bit evaluation: of the loss, of each logp, of each row's slope."""
    z = q["logits"].double().cpu() / temperature
    tokens = q["tokens"].cpu().long()
    off = q["offsets"].cpu().tolist()
    T, V = z.shape
    S = len(off) - 1
    old, ref, adv = (q[n].double().cpu() for n in ("old", "ref", "adv"))
    live = (tokens >= 0) & (tokens < V) & (z.max(1).values > -math.inf)
    inside = torch.zeros(T, dtype=torch.bool)
    weight = torch.zeros(T, dtype=torch.float64)
    named = (tokens >= 0) & (tokens < V)
    for b, e in zip(off[:-1], off[1:]):
        inside[b:e] = True
        weight[b:e] = 1.0 / (S * max(1, int(named[b:e].sum())))
    live &= inside
    weight = weight * live
    logp, dz = torch.zeros(T, dtype=torch.float64), torch.zeros_like(z)
    loss, loss_err = 0.0, 0.0
    lp_err, dz_err = torch.zeros(T, dtype=torch.float64), torch.zeros_like(z)
    for t in torch.nonzero(live)[:, 0].tolist():
        m = z[t].max()
        p = torch.exp(z[t] - m)
        lse = m + torch.log(p.sum())
        p = torch.exp(z[t] - lse)
        lp = float(z[t, tokens[t]] - lse)
        r, A = math.exp(lp - old[t]), float(adv[t])
        c = min(max(r, 1 - low), 1 + high)
        free = r * A <= c * A
        term = -min(r * A, c * A)
        slope = -r * A if free else 0.0
        # In 32 bits, base 2: a scaled logit is off by 2 roundings and lse by as
        # much, by the sum of V terms of 2 roundings each (V / 1024 + 32 additions
        # deep), and by its logarithm's; then 4 more for the product with ln 2.
        far = max(abs(v) for v in (float(m), lp, float(z[t, tokens[t]])) if math.isfinite(v))
        e = U * (8 * far + V / 1024 + 64)
        er = e + 8 * U + U * abs(lp - old[t])  # relative, of r
        slope_err = abs(A) * r * er
        term_err = abs(A) * max(r, c) * er
        if kl:
            d = float(ref[t]) - lp
            term += kl * (math.exp(d) - d - 1)
            slope += kl * (1 - math.exp(d))
            ek = e + 8 * U + U * abs(d)
            term_err += kl * (math.exp(d) * ek + abs(d) * ek + 4 * U)
            slope_err += kl * (math.exp(d) * ek + U)
        hot = torch.zeros(V, dtype=torch.float64)
        hot[tokens[t]] = 1
        k = float(weight[t]) / temperature * grad_scale
        dz[t] = slope * k * (hot - p)
        # A probability is off by its exponent's error; then four products.
        finite = torch.where(torch.isfinite(z[t]), z[t].abs(), 0.0)
        ep = p * (U * 6 * finite + e + 8 * U)
        dz_err[t] = abs(k) * (slope_err * (hot - p).abs() + abs(slope) * (ep + 6 * U * (hot + p)))
        logp[t], lp_err[t] = lp, e
        loss += float(weight[t]) * term
        loss_err += float(weight[t]) * (term_err + 4 * U * abs(term))
    return loss, logp, dz, loss_err, lp_err, dz_err


def policy_inputs(g, T, V, S, dtype, masked=0.3, idtype=torch.int64, scale=3.0):
    logits = (torch.randn(T, V, generator=g, device=DEV) * scale).to(dtype)
    tokens = torch.randint(0, V, (T,), generator=g, device=DEV)
    now = torch.log_softmax(logits.float(), 1).gather(1, tokens[:, None])[:, 0] if T else torch.zeros(0, device=DEV)
    q = dict(logits=logits,
             # Ratios well inside, well below and well above the borders.
             old=now + torch.tensor([0.0, 0.5, -0.5, 0.1, -0.1], device=DEV).repeat(T // 5 + 1)[:T],
             ref=now + 0.3 * torch.randn(T, generator=g, device=DEV),
             adv=torch.randn(T, generator=g, device=DEV))
    off = torch.randint(0, T + 1, (max(0, S - 1),), generator=g, device=DEV).sort().values
    q["offsets"] = torch.cat([torch.tensor([0], device=DEV), off, torch.tensor([T], device=DEV)])[:S + 1]
    out = torch.rand(T, generator=g, device=DEV) < masked
    tokens = torch.where(out, torch.where(torch.arange(T, device=DEV) % 2 == 0, -1, V), tokens)
    q["tokens"] = tokens.to(idtype)
    return q


def run_policy(q, kl, temperature=1.0, fn=st.policy_loss_grad, **kw):
    return fn(q["logits"], q["tokens"], q["old"], q["adv"], q["offsets"],
              ref_logp=q["ref"] if kl else None, kl_coef=kl, temperature=temperature, **kw)


def check_policy(q, kl=0.0, temperature=1.0, grad_scale=1.0, low=0.2, high=0.2):
    exact, logp, dz, loss_err, lp_err, dz_err = exact_policy(q, kl, low, high, temperature, grad_scale)
    kw = dict(clip_low=low, clip_high=high)
    loss, lp, d = run_policy(q, kl, temperature, grad_scale=grad_scale, **kw)
    loss2, lp2 = run_policy(q, kl, temperature, fn=st.policy_loss, **kw)
    torch.cuda.synchronize()
    assert loss.shape == () and loss.dtype == lp.dtype == torch.float32
    assert torch.equal(loss, loss2) and torch.equal(lp, lp2)
    assert abs(float(loss) - exact) <= loss_err + 2 * U * abs(exact) + 1e-30
    fine = torch.isfinite(logp)
    assert torch.equal(lp.cpu().double()[~fine], logp[~fine])
    assert bool(((lp.cpu().double() - logp).abs() <= lp_err)[fine].all())
    close(d.cpu(), dz, dz_err)
    return loss, lp, d


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("T,V,S", [(1, 1, 1), (2, 7, 1), (5, 8, 2), (6, 1000, 3), (9, 4099, 2),
                                   (11, 32003, 4), (3, 131072, 1), (2, 200001, 2), (70, 50, 12)])
def test_policy_loss(T, V, S, dtype):
    g = gen(T + V)
    for kl, temperature, idtype in ((0.0, 1.0, torch.int64), (0.05, 0.7, torch.int32)):
        check_policy(policy_inputs(g, T, V, S, dtype, idtype=idtype), kl, temperature)


def test_policy_loss_options_and_layouts():
    g = gen(20)
    q = policy_inputs(g, 20, 515, 3, torch.bfloat16)
    check_policy(q, 0.1, 1.0, grad_scale=64.0, low=0.0, high=0.6)
    check_policy(q, 0.1, 1.5, grad_scale=-1.0, low=1.0, high=0.0)
    wide = torch.randn(20, 600, generator=g, device=DEV).bfloat16()
    want = check_policy(dict(q, logits=wide[:, 7:522].contiguous()), 0.1)
    part = dict(q, logits=wide[:, 7:522])
    for a, b in zip(want, check_policy(part, 0.1)):
        assert torch.equal(a, b)
    far = dict(q, logits=part["logits"].t().contiguous().t())
    for a, b in zip(want, run_policy(far, 0.1)):
        assert torch.equal(a, b)
    buf = wide.clone()
    view = buf[:, 7:522]
    loss, lp, d = run_policy(dict(q, logits=view), 0.1, dlogits=view)
    assert d is view and torch.equal(d, want[2]) and torch.equal(loss, want[0])
    assert torch.equal(buf[:, :7], wide[:, :7]) and torch.equal(buf[:, 522:], wide[:, 522:])


def test_policy_loss_in_place_every_type():
    for dtype in TYPES:
        for V in (33, 5000, 40000, 70001, 140000, 270001):
            q = policy_inputs(gen(V), 4, V, 1, dtype)
            want = run_policy(q, 0.1)
            got = run_policy(q, 0.1, dlogits=q["logits"])
            assert got[2] is q["logits"]
            for a, b in zip(want, got):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_policy_rows_left_out_and_ruled_out_tokens(dtype):
    g = gen(21)
    for V in (40, 9001):
        q = policy_inputs(g, 12, V, 3, dtype, masked=0.0)
        low = torch.finfo(dtype).min
        q["tokens"][[0, 3]] = -1
        q["tokens"][5] = 2 ** 40
        for n in ("old", "ref", "adv"):
            q[n][[0, 3, 5]] = float("nan")
        q["logits"][0] = float("nan")       # left out: whatever it holds
        q["logits"][3] = float("inf")
        q["logits"][4] = -float("inf")      # nothing to draw from
        q["logits"][6, V // 2:] = -float("inf")
        q["tokens"][6] = 1
        q["logits"][7, 2:] = low            # the type's lowest value as a mask
        q["tokens"][7] = 0
        q["logits"][8] = -float("inf")      # one token left: certain, no gradient
        q["logits"][8, 3] = 2.0
        q["tokens"][8] = 3
        q["logits"][9, :] = low             # all equal, however low
        q["offsets"] = torch.tensor([1, 1, 6, 11], device=DEV)  # an empty answer, rows outside
        q["old"][[6, 7, 8, 9]] = torch.tensor([-2.0, -1.0, 0.05, -math.log(V) + 0.05], device=DEV)
        q["ref"][[6, 7, 8, 9]] = torch.tensor([-2.2, -0.5, 0.1, -math.log(V)], device=DEV)
        clean = {n: torch.nan_to_num(v, nan=0.0) if n in ("old", "ref", "adv") else v for n, v in q.items()}
        exact, logp, dz, loss_err, lp_err, dz_err = exact_policy(clean, 0.05, 0.2, 0.2, 1.0)
        loss, lp, d = run_policy(q, 0.05)
        assert abs(float(loss) - exact) <= loss_err + 2 * U * abs(exact)
        assert bool(((lp.cpu().double() - logp).abs() <= lp_err).all())
        close(d.cpu(), dz, dz_err)
        for t in (0, 3, 4, 5, 11):
            assert bool((d[t] == 0).all()) and lp[t] == 0
        # A sampled token that is ruled out has probability zero.
        q["tokens"][6] = V - 1
        lp = run_policy(q, 0.0)[1]
        assert float(lp[6]) == -math.inf


def test_policy_loss_without_rows_or_answers():
    q = policy_inputs(gen(22), 0, 10, 2, torch.float32)
    loss, lp, d = run_policy(q, 0.0)
    assert float(loss) == 0 and lp.shape == (0,) and d.shape == (0, 10)
    q = policy_inputs(gen(22), 6, 10, 1, torch.float32)
    q["offsets"] = q["offsets"][:1]
    loss, lp, d = run_policy(q, 0.1)
    assert float(loss) == 0 and bool((lp == 0).all()) and bool((d == 0).all())
    q = policy_inputs(gen(22), 6, 10, 2, torch.float32)
    q["tokens"][:] = -1
    loss, lp, d = run_policy(q, 0.1)
    assert float(loss) == 0 and bool((lp == 0).all()) and bool((d == 0).all())


def test_policy_gradient_against_differences():
    # Central differences of the 64-bit loss: off by h^2 / 6 of the third
    # derivative, which with h = 1e-4 is below 1e-7 of the loss's scale here.
    g = gen(23)
    q = policy_inputs(g, 6, 30, 2, torch.float32, masked=0.2, scale=1.0)
    d = run_policy(q, 0.3, 0.9)[2].cpu().double()
    *_, dz_err = exact_policy(q, 0.3, 0.2, 0.2, 0.9)
    for t in range(6):
        for c in {0, 17, int(q["tokens"][t].clamp(0, 29))}:
            pair = []
            for h in (1e-4, -1e-4):
                z = q["logits"].double().clone()
                z[t, c] += h
                pair.append(exact_policy(dict(q, logits=z), 0.3, 0.2, 0.2, 0.9)[0])
            diff = (pair[0] - pair[1]) / 2e-4
            assert abs(diff - float(d[t, c])) <= float(dz_err[t, c]) + U * abs(diff) + 1e-7


# --------------------------------------------------------------------------
# Streams, graphs, repeated calls, far offsets, refusals
# --------------------------------------------------------------------------
def everything(s, stream=None):
    """One call of each operator; the outputs."""
    kw = dict(stream=stream)
    order, position, offsets = st.sort_ids(s["ids"], 9, **kw)
    rows = st.dispatch(s["x"], position, offsets, **kw)
    out = st.combine(rows, position, offsets, s["w"], **kw)
    dy, dw = st.combine_backward(out, rows, position, offsets, s["w"], **kw)
    dx = st.dispatch_backward(dy, position, offsets, **kw)
    e = st.embedding(s["table"], s["tokens"], scale=2.0, **kw)
    dt = st.embedding_backward(e, s["tokens"], 300, scale=2.0, padding_id=1, **kw)
    loss, lp, dl = st.policy_loss_grad(s["logits"], s["tokens"], s["old"], s["adv"], s["answers"],
                                       ref_logp=s["old"], kl_coef=0.1, **kw)
    return [order, position, offsets, rows, out, dy, dw, dx, e, dt, loss, lp, dl]


def some_state(seed):
    g = gen(seed)
    T = 200
    return dict(ids=torch.randint(-1, 9, (T, 2), generator=g, device=DEV), x=randn(g, T, 96).bfloat16(),
                w=torch.rand(T, 2, generator=g, device=DEV), table=randn(g, 300, 77).half(),
                tokens=torch.randint(0, 300, (T,), generator=g, device=DEV),
                logits=randn(g, T, 300), old=-torch.rand(T, generator=g, device=DEV) * 6,
                adv=randn(g, T), answers=torch.tensor([0, 50, 120, T], device=DEV))


def same_bits(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dim() else x, y.view(torch.uint8) if y.dim() else y)
               for x, y in zip(a, b))


def test_same_bits_every_time_and_on_another_stream():
    s = some_state(30)
    want = everything(s)
    torch.cuda.synchronize()
    for _ in range(3):
        assert same_bits(want, everything(s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(s, stream=side)
    side.synchronize()
    assert same_bits(want, got)
    with torch.cuda.stream(side):
        got = everything(s)
    side.synchronize()
    assert same_bits(want, got)


def test_captured_into_a_graph():
    s = some_state(31)
    everything(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything(s)
    for seed in (32, 33, 31, 34):
        new = some_state(seed)
        for name, v in new.items():
            s[name].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(everything(new), outs)
        torch.cuda.synchronize()


def test_sums_do_not_depend_on_what_else_is_in_the_batch():
    g = gen(35)
    ids, position, offsets = slots(g, 40, 3, 9, 0.0)
    y, w = randn(g, 120, 200).bfloat16(), torch.rand(40, 3, generator=g, device=DEV)
    whole = st.combine(y, position, offsets, w)
    for t in (0, 13, 39):
        one = st.combine(y[position[t].long()].contiguous(), torch.arange(3, device=DEV).int()[None], None, w[t:t + 1])
        assert torch.equal(one[0], whole[t])


@pytest.mark.slow
def test_offsets_past_32_bits():
    g = gen(36)
    width, tokens, k = 32768, 8800, 8  # 2.3 G elements of packed rows
    x = randn(g, 8, width).bfloat16().repeat(tokens // 8, 1)
    position = torch.randperm(tokens * k, generator=g, device=DEV).int().view(tokens, k)
    rows = st.dispatch(x, position)
    last = (position == tokens * k - 1).nonzero()[0]
    assert torch.equal(rows[-1], x[last[0]])
    w = torch.full((tokens, k), 0.125, device=DEV)
    assert torch.equal(st.combine(rows, position, None, w), x)
    drows, dw = st.combine_backward(x, rows, position, None, w)
    assert torch.equal(drows[-1].float(), x[last[0]].float() / 8)
    close(dw[-1], (x[-1].double() ** 2).sum().expand(k), (width + 1) * U * float((x[-1].double() ** 2).sum()))
    del drows
    ids = torch.tensor([tokens * k - 1, 0, tokens * k - 2, 65536], device=DEV)
    assert torch.equal(st.embedding(rows, ids), rows[ids])
    d = st.embedding_backward(x[:4], ids, tokens * k, out=rows)
    assert torch.equal(d[-1], x[0]) and torch.equal(d[65536], x[3]) and not bool(d[-3].any())
    del rows, d
    T, V = 16400, 131072
    logits = torch.empty(T, V, dtype=torch.bfloat16, device=DEV)
    logits.view(torch.int16).zero_()
    logits[-1] = randn(g, V).bfloat16()
    tokens = torch.full((T,), -1, device=DEV)
    tokens[-1] = V - 1
    q = dict(logits=logits, tokens=tokens, old=torch.full((T,), -12.0, device=DEV),
             adv=torch.full((T,), -1.0, device=DEV), offsets=torch.tensor([0, T], device=DEV))
    small = dict(q, logits=logits[-1:].clone(), tokens=tokens[-1:], old=q["old"][-1:],
                 adv=q["adv"][-1:], offsets=torch.tensor([0, 1], device=DEV))
    want = run_policy(small, 0.0)
    got = run_policy(q, 0.0, dlogits=logits)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1][-1:], want[1])
    assert torch.equal(got[2][-1:], want[2]) and not bool(got[2][0].any())


def test_refusals_of_the_binding():
    x, f = torch.zeros(4, 8, device=DEV), torch.zeros(4, device=DEV)
    pos = torch.arange(8, device=DEV).int().view(4, 2)
    rows = torch.zeros(8, 8, device=DEV)
    off, ids = torch.tensor([0, 8], device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    bad = [
        (TypeError, lambda: st.sort_ids(f, 3)), (ValueError, lambda: st.sort_ids(ids, -1)),
        (TypeError, lambda: st.sort_ids(ids.short(), 3)),
        (TypeError, lambda: st.dispatch(x.double(), pos, off)),
        (TypeError, lambda: st.dispatch(x, pos.long(), off)),
        (TypeError, lambda: st.dispatch(x, pos, off.int())),
        (ValueError, lambda: st.dispatch(x, pos[:3], off)),
        (ValueError, lambda: st.dispatch(x, pos.cpu(), off)),
        (ValueError, lambda: st.dispatch(x, pos, off.cpu())),
        (ValueError, lambda: st.dispatch(x[:, :0], pos, off)),
        (ValueError, lambda: st.dispatch(x, pos[:, :0], off)),
        (ValueError, lambda: st.dispatch(x, pos, off, out=rows[:7])),
        (TypeError, lambda: st.dispatch(x, pos, off, out=rows.half())),
        (ValueError, lambda: st.dispatch(x, pos, off, out=rows.t())),
        (ValueError, lambda: st.dispatch(x, pos, off, out=rows[:1].expand(8, 8))),
        (ValueError, lambda: st.combine(x, pos, off)),
        (ValueError, lambda: st.combine(rows, pos, off, w.t())),
        (TypeError, lambda: st.combine(rows, pos, off, w.half())),
        (ValueError, lambda: st.combine(rows, pos, off, w.cpu())),
        (ValueError, lambda: st.combine_backward(rows, rows, pos, off)),
        (ValueError, lambda: st.combine_backward(x, x, pos, off)),
        (TypeError, lambda: st.combine_backward(x, rows.half(), pos, off)),
        (TypeError, lambda: st.embedding(x, f)), (TypeError, lambda: st.embedding(ids[:, None], ids)),
        (ValueError, lambda: st.embedding(x, ids, out=rows)),
        (ValueError, lambda: st.embedding_backward(x, ids[:3], 5)),
        (ValueError, lambda: st.embedding_backward(x, ids, 5, accumulate=True)),
        (TypeError, lambda: st.embedding_backward(x, ids, 5, dtype=torch.float16)),
        (ValueError, lambda: st.embedding_backward(x, ids, 5, out=rows)),
        (ValueError, lambda: st.embedding_backward(x, ids, -5)),
        (ValueError, lambda: st.policy_loss(x, ids[:3], f, f, off)),
        (ValueError, lambda: st.policy_loss(x, ids, f[:3], f, off)),
        (TypeError, lambda: st.policy_loss(x, ids, f.double(), f, off)),
        (TypeError, lambda: st.policy_loss(x, f, f, f, off)),
        (ValueError, lambda: st.policy_loss(x, ids, f, f, off, kl_coef=0.1)),
        (st.SegTopKError, lambda: st.policy_loss(x, ids, f, f, off, temperature=0.0)),
        (st.SegTopKError, lambda: st.policy_loss(x, ids, f, f, off, clip_low=-1.0)),
        (TypeError, lambda: st.policy_loss_grad(x, ids, f, f, off, dlogits=x.half())),
        (ValueError, lambda: st.policy_loss_grad(x.t(), ids.repeat(2), f.repeat(2), f.repeat(2), off,
                                                 dlogits=x)),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
    y = x.t()
    with pytest.raises(ValueError):
        st.policy_loss_grad(y, ids.repeat(2), f.repeat(2), f.repeat(2), off, dlogits=y)
