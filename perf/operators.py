"""The operators around the two top-k selections of a language model, as they are measured.

A router's top-k picks each token's experts; a sampler's top-k picks the next
token from the vocabulary's logits.  Around them stand

  route        tokens sorted by expert, gathered into expert order, and brought
               back with the gate weights applied; and the gradients
  embed        the lookup of token rows in an embedding table, scaled, and the
               table's gradient by sorted tokens
  policy       the clipped policy loss with a KL term over the logits of sampled
               tokens, alone or with its gradient

``own`` False computes the plain form (elementary torch operations, 32 or 64
bits, rounded once at the end); True makes the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # One token of a decode step through a small mixture: the least work
        # there is, all latency.
        dict(name="route one token", kind="route", backward=False, T=1, k=2, E=8, H=2048,
             dtype="f16", wdtype="f32", index="i32", dropped=0.0),
        # A decode step of a serving batch, each token with 8 experts of 64.
        dict(name="route decode", kind="route", backward=False, T=64, k=8, E=64, H=4096,
             dtype="bf16", wdtype="f32", index="i32", dropped=0.0),
        # Odd sizes in 32 bits; one slot in ten dropped by its expert's capacity.
        dict(name="route ragged", kind="route", backward=False, T=1003, k=3, E=37, H=1001,
             dtype="f32", wdtype="f32", index="i64", dropped=0.1),
        # A prefill or training batch.
        dict(name="route prefill", kind="route", backward=False, T=8192, k=8, E=128, H=4096,
             dtype="bf16", wdtype="f32", index="i64", dropped=0.0),
        # The gradients of that training batch: rows, weights and tokens.
        dict(name="route backward", kind="route", backward=True, T=8192, k=8, E=128, H=4096,
             dtype="bf16", wdtype="f32", index="i64", dropped=0.0),
        # A small fine-tuning micro-batch with dropped slots, weights in 16 bits.
        dict(name="route backward ragged", kind="route", backward=True, T=777, k=6, E=60, H=1410,
             dtype="f16", wdtype="f16", index="i32", dropped=0.05),
        # The lookup of a decode step.
        dict(name="embed decode", kind="embed", backward=False, N=64, V=131072, H=4096,
             dtype="bf16", index="i64", pad=0.0),
        # The lookup of a training batch, with padding.
        dict(name="embed batch", kind="embed", backward=False, N=32768, V=131072, H=4096,
             dtype="bf16", index="i64", pad=0.1),
        # The table's gradient for that batch: tokens as skewed as text.
        dict(name="embed gradient", kind="embed", backward=True, N=32768, V=131072, H=4096,
             dtype="bf16", index="i64", pad=0.1),
        # A small table in 32 bits, odd width, few rows of the table left out.
        dict(name="embed gradient ragged", kind="embed", backward=True, N=5003, V=4099, H=1001,
             dtype="f32", index="i32", pad=0.05),
        # Scoring of a few short answers, no gradient.
        dict(name="policy score", kind="policy", backward=False, T=96, V=32003, S=3,
             dtype="f16", kl=0.0, masked=0.2, temperature=1.0),
        # A training step on sampled answers over the library's 128 Ki-entry
        # bf16 logits rows.
        dict(name="policy step", kind="policy", backward=True, T=4096, V=131072, S=16,
             dtype="bf16", kl=0.04, masked=0.25, temperature=0.8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route", "embed", "embed", "policy"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "route":
        E = _log_int(rng, 4, 256)
        T = _log_int(rng, 1, 8192 if dtype != "f32" else 4096)
        return dict(kind=kind, backward=rng.random() < 0.5, T=T, k=rng.randint(1, min(8, E)), E=E,
                    H=_log_int(rng, 64, 4096), dtype=dtype,
                    wdtype=rng.choice(["f32", dtype]), index=rng.choice(["i32", "i64"]),
                    dropped=rng.choice([0.0, 0.0, 0.05, 0.3]))
    if kind == "embed":
        N = _log_int(rng, 1, 32768)
        V = _log_int(rng, 1000, 131072 if dtype != "f32" else 65536)
        return dict(kind=kind, backward=rng.random() < 0.5, N=N, V=V, H=_log_int(rng, 64, 4096),
                    dtype=dtype, index=rng.choice(["i32", "i64"]), pad=rng.choice([0.0, 0.1, 0.5]))
    T = _log_int(rng, 8, 4096)
    V = _log_int(rng, 1000, 131072 if dtype != "f32" else 65536)
    return dict(kind=kind, backward=rng.random() < 0.7, T=T, V=V,
                S=rng.randint(1, max(1, min(32, T // 4))), dtype=dtype,
                kl=rng.choice([0.0, 0.04, 0.1]), masked=rng.choice([0.0, 0.25, 0.5]),
                temperature=rng.choice([1.0, 0.8, 1.3]))


def work(c):
    b = BYTES[c["dtype"]]
    if c["kind"] == "route":
        T, k, E, H = c["T"], c["k"], c["E"], c["H"]
        N, wb = T * k, BYTES[c["wdtype"]]
        if not c["backward"]:
            # ids in; order, position, offsets out; x in, rows out; expert
            # rows and weights in, tokens out
            ib = 8 if c["index"] == "i64" else 4
            return {"bytes": N * ib + N * 8 + 8 * (E + 1) + (2 * T + 2 * N) * H * b + N * wb,
                    "flops": 2 * N * H}
        # dout, y, drows in; dy, dx out; weights in, their gradient out
        return {"bytes": (T + N + N + N + T) * H * b + N * 4 + 2 * N * wb, "flops": 4 * N * H}
    if c["kind"] == "embed":
        N, V, H = c["N"], c["V"], c["H"]
        ib = 8 if c["index"] == "i64" else 4
        # The gradient is written whole; of the table only the rows of distinct
        # tokens are read: the i-th most frequent of them is among the N with
        # probability 1 - (1 - p_i)^N.
        i = torch.arange(V, dtype=torch.float64)
        p = (1 - c["pad"]) * torch.log1p(1 / (i + 1)) / math.log(V + 1.0)
        rows = V if c["backward"] else float((1 - (1 - p) ** N).sum())
        return {"bytes": N * ib + (N + rows) * H * b, "flops": N * H}
    T, V = c["T"], c["V"]
    return {"bytes": T * V * b * (2 if c["backward"] else 1) + T * 24, "flops": 5 * T * V}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _index(case, t):
    return t.to(torch.int64 if case["index"] == "i64" else torch.int32)


def _randn(g, shape, dtype, scale=1.0):
    # In pieces, so that the 32-bit numbers of a large array are never whole.
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, generator=g, device=DEV) * scale).to(dtype)
    return out


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["kind"] == "route":
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        # Some experts are liked better than others.
        scores = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
        top, ids = torch.topk(scores, k, dim=1)
        if case["dropped"]:
            ids = torch.where(torch.rand(T, k, generator=g, device=DEV) < case["dropped"], -1, ids)
        s["ids"] = _index(case, ids)
        s["weights"] = torch.softmax(top, 1).to(DTYPES[case["wdtype"]])
        s["y"] = _randn(g, (T * k, H), dt)
        if case["backward"]:
            # What the forward pass left: where each slot went.
            _, s["position"], s["offsets"] = _plain_sort(s["ids"], E)
            s["dout"] = _randn(g, (T, H), dt, 0.1)
            s["drows"] = _randn(g, (T * k, H), dt, 0.1)
        else:
            s["x"] = _randn(g, (T, H), dt)
    elif case["kind"] == "embed":
        N, V, H = case["N"], case["V"], case["H"]
        # The i-th most frequent token with a share of about 1 / i, at a
        # shuffled place in the table.
        u = torch.rand(N, generator=g, device=DEV, dtype=torch.float64)
        rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp(0, V - 1)
        ids = (rank * 7919 + 13) % V
        if case["pad"]:
            ids = torch.where(torch.rand(N, generator=g, device=DEV) < case["pad"], 0, ids)
        s["ids"] = _index(case, ids)
        s["scale"] = math.sqrt(H)
        if case["backward"]:
            s["dout"] = _randn(g, (N, H), dt, 0.1)
        else:
            s["table"] = _randn(g, (V, H), dt, 0.02)
    else:
        T, V, S = case["T"], case["V"], case["S"]
        s["logits"] = _randn(g, (T, V), dt, 3.0)
        # The sampled tokens and the log-probability of each now; what it was
        # when it was sampled, and under the reference, is a little off.
        tokens = torch.empty(T, dtype=torch.int64, device=DEV)
        now = torch.empty(T, device=DEV)
        step = max(1, (1 << 26) // V)
        for i in range(0, T, step):
            z = s["logits"][i:i + step].float() / case["temperature"]
            race = z - torch.empty_like(z).exponential_(generator=g).log()
            tokens[i:i + step] = race.argmax(1)
            now[i:i + step] = z.gather(1, tokens[i:i + step, None])[:, 0] - torch.logsumexp(z, 1)
        s["old"] = now + 0.15 * torch.randn(T, generator=g, device=DEV)
        s["ref"] = now + 0.3 * torch.randn(T, generator=g, device=DEV)
        cut = torch.randperm(T - 1, generator=g, device=DEV)[:S - 1].sort().values + 1
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cut,
                                  torch.full((1,), T, dtype=torch.int64, device=DEV)])
        # One advantage for each answer; prompt tokens are left out.
        adv = torch.randn(S, generator=g, device=DEV)
        s["adv"] = adv.repeat_interleave(s["offsets"].diff()).contiguous()
        if case["masked"]:
            tokens = torch.where(torch.rand(T, generator=g, device=DEV) < case["masked"], -1, tokens)
        s["tokens"] = tokens
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_sort(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    ordered, order = torch.sort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.searchsorted(ordered, torch.arange(E + 1, device=order.device))
    return order.int(), position.int().view(ids.shape), offsets


def _plain_route(s):
    case, x, y = s["case"], s["x"], s["y"]
    T, k = s["ids"].shape
    order, position, offsets = _plain_sort(s["ids"], case["E"])
    kept = torch.arange(T * k, device=x.device) < offsets[-1]
    rows = x[(order // k).long()].float() * kept[:, None]
    slot = position.long()
    w = s["weights"].float() * (slot < offsets[-1])
    out = (y.float()[slot] * w[:, :, None]).sum(1)
    return order, position, offsets, rows.to(x.dtype), out.to(y.dtype)


def _plain_route_backward(s):
    y, dout, drows, w = s["y"].float(), s["dout"].float(), s["drows"].float(), s["weights"].float()
    slot = s["position"].long()
    kept = (slot < s["offsets"][-1])[:, :, None]
    dy = torch.zeros_like(y)
    dy[slot.reshape(-1)] = (dout[:, None, :] * w[:, :, None] * kept).reshape(y.shape)
    dw = (dout[:, None, :] * y[slot] * kept).sum(2)
    dx = (drows[slot] * kept).sum(1)
    return dy.to(s["y"].dtype), dw.to(s["weights"].dtype), dx.to(s["drows"].dtype)


def _plain_policy(s):
    case, z = s["case"], s["logits"].float() / s["case"]["temperature"]
    T, V = z.shape
    tokens, off = s["tokens"], s["offsets"]
    S = off.numel() - 1
    live = (tokens >= 0) & (tokens < V)
    at = torch.where(live, tokens, 0)
    m = z.max(1).values
    e = torch.exp(z - m[:, None])
    total = e.sum(1)
    logp = z.gather(1, at[:, None])[:, 0] - m - torch.log(total)
    seg = torch.searchsorted(off, torch.arange(T, device=z.device), right=True) - 1
    n = torch.zeros(S, device=z.device).index_add_(0, seg, live.float())
    weight = live / (S * n[seg]).clamp(min=1)
    ratio, adv = torch.exp(logp - s["old"]), s["adv"]
    bounded = ratio.clamp(0.8, 1.2)
    free = ratio * adv <= bounded * adv
    term = -torch.where(free, ratio * adv, bounded * adv)
    slope = -torch.where(free, ratio * adv, 0.0)
    if case["kl"]:
        apart = s["ref"] - logp
        term = term + case["kl"] * (torch.exp(apart) - apart - 1)
        slope = slope + case["kl"] * (1 - torch.exp(apart))
    loss = (term.double() * weight.double()).sum().float()
    logp = torch.where(live, logp, 0.0)
    if not case["backward"]:
        return loss, logp
    slope = slope * weight / case["temperature"]
    d = -(e / total[:, None]) * slope[:, None]
    d.scatter_add_(1, at[:, None], slope[:, None])
    return loss, logp, d.to(s["logits"].dtype)


def _plain(s):
    case = s["case"]
    if case["kind"] == "route":
        return _plain_route_backward(s) if case["backward"] else _plain_route(s)
    if case["kind"] == "policy":
        return _plain_policy(s)
    ids = s["ids"].long()
    if not case["backward"]:
        return (s["table"][ids].float() * s["scale"]).to(s["table"].dtype)
    # Token 0 is the padding: it has a row, and that row no gradient.
    g = s["dout"].float() * (ids != 0)[:, None]
    d = torch.zeros(case["V"], case["H"], device=DEV).index_add_(0, ids, g)
    return (d * s["scale"]).to(s["dout"].dtype)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if not own:
        return _plain(s)
    import segmented_top_selection_amd as st
    case = s["case"]
    if case["kind"] == "route":
        if case["backward"]:
            dy, dw = st.combine_backward(s["dout"], s["y"], s["position"], s["offsets"], s["weights"])
            return dy, dw, st.dispatch_backward(s["drows"], s["position"], s["offsets"])
        order, position, offsets = st.sort_ids(s["ids"], case["E"])
        rows = st.dispatch(s["x"], position, offsets)
        return order, position, offsets, rows, st.combine(s["y"], position, offsets, s["weights"])
    if case["kind"] == "embed":
        if case["backward"]:
            return st.embedding_backward(s["dout"], s["ids"], case["V"], scale=s["scale"], padding_id=0)
        return st.embedding(s["table"], s["ids"], scale=s["scale"])
    loss = st.policy_loss_grad if case["backward"] else st.policy_loss
    return loss(s["logits"], s["tokens"], s["old"], s["adv"], s["offsets"], ref_logp=s["ref"],
                kl_coef=case["kl"], clip_low=0.2, clip_high=0.2, temperature=case["temperature"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(case, s):
    E, k, T = case["E"], case["k"], case["T"]
    if case["backward"]:
        position, count = s["position"].long(), int(s["offsets"][-1])
    else:
        # Slots listed expert by expert, the dropped ones last.
        flat = s["ids"].reshape(-1).cpu().tolist()
        lists = [[] for _ in range(E + 1)]
        for i, e in enumerate(flat):
            lists[e if 0 <= e < E else E].append(i)
        offsets = [0]
        for one in lists[:-1]:
            offsets.append(offsets[-1] + len(one))
        order = torch.tensor([i for one in lists for i in one], device=DEV)
        count = offsets[-1]
        position = torch.argsort(order).view(T, k)
    y = s["y"].double()
    if case["backward"]:
        dout, drows = s["dout"].double(), s["drows"].double()
        dy, dx = torch.zeros_like(y), torch.zeros_like(dout)
        dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            p = position[:, j]
            live = p < count
            dy[p[live]] = dout[live] * s["weights"][live, j].double()[:, None]
            dw[live, j] = torch.linalg.vecdot(dout[live], y[p[live]])
            dx[live] += drows[p[live]]
        return dy, dw, dx
    rows, out = torch.zeros_like(y), torch.zeros(T, case["H"], dtype=torch.float64, device=DEV)
    for j in range(k):
        p = position[:, j]
        live = p < count
        rows[p[live]] = s["x"][live].double()
        out[live] += y[p[live]] * s["weights"][live, j].double()[:, None]
    return (order.int(), position.int(), torch.tensor(offsets, device=DEV), rows, out)


def _exact_policy(case, s):
    T, V = s["logits"].shape
    tokens, off = s["tokens"], s["offsets"].tolist()
    S = len(off) - 1
    logp = torch.zeros(T, dtype=torch.float64, device=DEV)
    live = tokens >= 0
    at = tokens.clamp(min=0)
    step = max(1, (1 << 27) // V)
    for i in range(0, T, step):
        full = torch.log_softmax(s["logits"][i:i + step].double() / case["temperature"], 1)
        logp[i:i + step] = torch.take_along_dim(full, at[i:i + step, None], 1)[:, 0]
    leaf = logp.clone().requires_grad_()
    loss = torch.zeros((), dtype=torch.float64, device=DEV)
    for b, e in zip(off[:-1], off[1:]):
        here = live[b:e].nonzero()[:, 0] + b
        if not here.numel():
            continue
        lp, A = leaf[here], s["adv"][here].double()
        r = (lp - s["old"][here].double()).exp()
        one = -torch.minimum(r * A, r.clamp(0.8, 1.2) * A)
        if case["kl"]:
            apart = s["ref"][here].double() - lp
            one = one + case["kl"] * (torch.expm1(apart) - apart)
        loss = loss + one.mean() / S
    logp = torch.where(live, logp, 0.0)
    if not case["backward"]:
        return loss.detach(), logp
    loss.backward()
    d = torch.empty(T, V, dtype=torch.float64, device=DEV)
    for i in range(0, T, step):
        p = torch.softmax(s["logits"][i:i + step].double() / case["temperature"], 1)
        hot = torch.zeros_like(p).scatter_(1, at[i:i + step, None], 1.0)
        d[i:i + step] = (hot - p) * (leaf.grad[i:i + step] / case["temperature"])[:, None]
    return loss.detach(), logp, d


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "route":
        return _exact_route(case, s)
    if case["kind"] == "policy":
        return _exact_policy(case, s)
    ids = s["ids"].long()
    if not case["backward"]:
        return torch.index_select(s["table"], 0, ids).double() * math.sqrt(case["H"])
    kept = ids != 0
    d = torch.zeros(case["V"], case["H"], dtype=torch.float64, device=DEV)
    d.index_put_((ids[kept],), s["dout"][kept].double(), accumulate=True)
    return d * math.sqrt(case["H"])
