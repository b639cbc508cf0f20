"""Operators next to the two selections of a language model, as they are measured.

  route      a router's whole selection: scores, bias, groups, top-k, gate
             weights; and the gradient of its logits
  experts    the experts' products in 8 bits with a scale for each block of 128:
             tokens quantized into expert order and multiplied by their expert's
             weights; and the gradient of the weights
  verify     drafted tokens verified against the target's probabilities from
             given random numbers, and the token that follows them

``own`` False computes the plain form (elementary torch operations, 32 or 64
bits, rounded once at the end); True makes the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0   # the largest value of 8 bits
FLOOR = 2.0 ** -96  # a block's largest magnitude counts as this at least


def listed():
    return [
        # One token of a decode step: all latency.
        dict(name="route one token", kind="route", backward=False, T=1, E=64, k=8, dtype="f32",
             scoring="softmax", bias=False, groups=1, kept=1, best=2, renormalize=True, scale=1.0,
             ruled=0.0),
        # A training batch through a large router: sigmoid scores, a bias for
        # balance, the four best of eight groups.
        dict(name="route batch", kind="route", backward=False, T=32768, E=256, k=8, dtype="f32",
             scoring="sigmoid", bias=True, groups=8, kept=4, best=2, renormalize=True, scale=2.5,
             ruled=0.0),
        # The gradient of a prefill or training batch.
        dict(name="route backward", kind="route", backward=True, T=8192, E=128, k=8, dtype="bf16",
             scoring="softmax", bias=False, groups=1, kept=1, best=2, renormalize=True, scale=1.0,
             ruled=0.0),
        # A small micro-batch, odd sizes, some experts ruled out, weights as they are.
        dict(name="route backward ragged", kind="route", backward=True, T=777, E=60, k=6,
             dtype="f16", scoring="sigmoid", bias=True, groups=1, kept=1, best=2,
             renormalize=False, scale=1.5, ruled=0.1),
        # One token of a decode step through two experts.
        dict(name="experts one token", kind="experts", backward=False, T=1, k=2, E=8, K=2048,
             N=4096, dtype="f16", out="f16", dropped=0.0),
        # A decode step of a serving batch, each token with 8 experts of 64: the
        # weights of all of them are read for a few rows each.
        dict(name="experts decode", kind="experts", backward=False, T=64, k=8, E=64, K=4096, N=2048,
             dtype="bf16", out="bf16", dropped=0.0),
        # Odd sizes; one slot in ten dropped by its expert's capacity.
        dict(name="experts ragged", kind="experts", backward=False, T=1003, k=3, E=37, K=1001,
             N=777, dtype="f32", out="f32", dropped=0.1),
        # A prefill or training batch: compute.
        dict(name="experts prefill", kind="experts", backward=False, T=8192, k=8, E=128, K=4096,
             N=2048, dtype="bf16", out="bf16", dropped=0.0),
        # The gradient of that batch's weights.
        dict(name="weights gradient", kind="experts", backward=True, T=8192, k=8, E=128, K=4096,
             N=2048, dtype="bf16", out="bf16", dropped=0.0),
        # The same in a small micro-batch of odd sizes, with dropped slots.
        dict(name="weights gradient ragged", kind="experts", backward=True, T=777, k=6, E=60,
             K=1410, N=333, dtype="f16", out="f32", dropped=0.05),
        # One request, four drafted tokens.
        dict(name="verify one request", kind="verify", R=1, most=4, V=32003, dtype="f16",
             drafted=True, temperature=1.0),
        # A serving batch with up to seven drafted tokens each over the library's
        # 128 Ki-entry rows.
        dict(name="verify batch", kind="verify", R=64, most=7, V=131072, dtype="bf16", drafted=True,
             temperature=0.8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route", "experts", "experts", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log_int(rng, 4 if groups > 1 else 8, 512 // groups)
        kept = rng.randint(1, groups)
        k, backward = rng.randint(1, min(8, E // groups * kept)), rng.random() < 0.4
        # One weight that is renormalized is the scale, whatever the logits.
        return dict(kind=kind, backward=backward, T=_log_int(rng, 1, 32768), E=E, k=k, dtype=dtype,
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, kept=kept, best=rng.choice([1, 2]),
                    renormalize=rng.random() < 0.7 and k > 1, scale=rng.choice([1.0, 2.5]),
                    ruled=rng.choice([0.0, 0.0, 0.1] if backward else [0.0, 0.0, 0.1, 0.5]))
    if kind == "experts":
        E = _log_int(rng, 1, 128)
        k = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 65536 // k if dtype != "f32" else 16384 // k)
        K, N = _log_int(rng, 64, 4096), _log_int(rng, 64, 2048)
        return dict(kind=kind, backward=rng.random() < 0.4, T=T, k=k, E=E, K=K, N=N, dtype=dtype,
                    out=rng.choice([dtype, dtype, "f32"]), dropped=rng.choice([0.0, 0.0, 0.05, 0.3]))
    return dict(kind=kind, R=_log_int(rng, 1, 64), most=rng.randint(0, 7),
                V=_log_int(rng, 1000, 131072 if dtype != "f32" else 65536), dtype=dtype,
                drafted=rng.random() < 0.6, temperature=rng.choice([0.0, 0.8, 1.0, 1.3]))


def work(c):
    b = BYTES[c["dtype"]]
    if c["kind"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        if not c["backward"]:
            return {"bytes": T * E * b + T * k * 8, "flops": 4 * T * E}
        # logits, the chosen and their gradients in; the gradient out.  Only where
        # the softmax is over all experts are logits other than the chosen ones read.
        read = E if c["scoring"] == "softmax" and not c["renormalize"] else k
        return {"bytes": T * (read + E) * b + T * k * 8, "flops": 2 * T * (read + E)}
    if c["kind"] == "experts":
        T, k, E, K, N = c["T"], c["k"], c["E"], c["K"], c["N"]
        rows = T * k * (1 - c["dropped"])
        if c["backward"]:
            return {"bytes": rows * (K + N) * b + E * N * K * BYTES[c["out"]],
                    "flops": 2 * rows * K * N}
        # An expert is read if a slot chose it.
        used = E * (1 - (1 - (1 - c["dropped"]) * k / E) ** T)
        blocks = -(-N // 128) * -(-K // 128)
        return {"bytes": T * K * b + used * (N * K + 4 * blocks) + T * k * N * BYTES[c["out"]] + T * k * 4,
                "flops": 2 * rows * K * N}
    drafts = sum(c["most"] - r % (c["most"] + 1) for r in range(c["R"]))
    rows = drafts + c["R"] + (drafts if c["drafted"] else 0)
    return {"bytes": rows * c["V"] * b + (drafts + c["R"]) * 24, "flops": 4 * rows * c["V"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    # In pieces, so that the 32-bit numbers of a large array are never whole.
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, generator=g, device=DEV) * scale).to(dtype)
    return out


def _weights(g, E, N, K):
    """Experts' weights as a checkpoint holds them: 8 bits, and a scale for each block of 128 x 128."""
    nb, kb = -(-N // 128), -(-K // 128)
    # Rows begin at a multiple of 128 bytes.
    q = torch.zeros(E, N, kb * 128, dtype=F8, device=DEV)[:, :, :K]
    scales = torch.empty(E, nb, kb, device=DEV)
    for e in range(E):
        w = torch.zeros(nb * 128, kb * 128, device=DEV)
        w[:N, :K] = torch.randn(N, K, generator=g, device=DEV) * K ** -0.5
        most = w.view(nb, 128, kb, 128).abs().amax((1, 3)).clamp(min=FLOOR)
        scales[e] = _ratio(most, F8_MAX)
        w = w.view(nb, 128, kb, 128) * _ratio(F8_MAX, most)[:, None, :, None]
        q[e] = w.view(nb * 128, kb * 128)[:N, :K].to(F8)
    return q, scales


def _prepare_verify(case, s, g, dt):
    R, V, most = case["R"], case["V"], case["most"]
    # All lengths from `most` down to none, in turn.
    count = most - torch.arange(R, device=DEV) % (most + 1)
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), count.cumsum(0)])
    D = int(s["offsets"][-1])
    s["target"] = _randn(g, (D + R, V), dt, 3.0)
    # The rows of the drafted tokens: the target's, without each request's last.
    row = torch.arange(D, device=DEV)
    row = row + torch.searchsorted(s["offsets"], row, right=True) - 1
    # A draft model that is near the target's.
    near = (s["target"][row].float() + 0.8 * torch.randn(D, V, generator=g, device=DEV)).to(dt)
    z = near.float() / max(case["temperature"], 0.1)
    s["tokens"] = (z - torch.empty_like(z).exponential_(generator=g).log()).argmax(1) if D else row
    s["draft"] = near if case["drafted"] else None
    s["accept"] = torch.rand(D, generator=g, device=DEV)
    s["sample"] = torch.rand(R, generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["kind"] == "verify":
        _prepare_verify(case, s, g, dt)
        return s
    if case["kind"] == "route":
        T, E = case["T"], case["E"]
        x = 1.5 * torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
        if case["ruled"]:
            x = torch.where(torch.rand(T, E, generator=g, device=DEV) < case["ruled"], -math.inf, x)
        s["logits"] = x.to(dt)
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        if case["backward"]:
            s["experts"] = _plain_route(s)[1]
            s["dweights"] = torch.randn(T, case["k"], generator=g, device=DEV)
        return s
    T, k, E, K, N = case["T"], case["k"], case["E"], case["K"], case["N"]
    # Some experts are liked better than others.
    liked = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    ids = torch.topk(liked, k, dim=1).indices
    if case["dropped"]:
        ids = torch.where(torch.rand(T, k, generator=g, device=DEV) < case["dropped"], -1, ids)
    # What the sort of the ids gives: where each slot goes, and each expert's rows.
    key = torch.where(ids >= 0, ids, E).view(-1)
    ordered, order = torch.sort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(T * k, device=DEV)
    s["position"] = position.int().view(T, k)
    s["offsets"] = torch.searchsorted(ordered, torch.arange(E + 1, device=DEV))
    if case["backward"]:
        s["x"] = _randn(g, (T * k, K), dt)
        s["dout"] = _randn(g, (T * k, N), dt, 0.01)
    else:
        s["x"] = _randn(g, (T, K), dt)
        s["w"], s["wscales"] = _weights(g, E, N, K)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_route(s):
    case, x = s["case"], s["logits"].double()
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    out = x == -math.inf
    if case["scoring"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = 1 / (1 + torch.exp(-x))
    pick = p if s["bias"] is None else p + s["bias"].double()
    pick = torch.where(out, -math.inf, pick)
    if G > 1:
        each = pick.view(T, G, E // G)
        top = torch.topk(each, min(case["best"], E // G), 2).values
        group = torch.where(top == -math.inf, 0.0, top).sum(2)
        group = torch.where(top[:, :, 0] == -math.inf, -math.inf, group)
        order = torch.sort(group, dim=1, descending=True, stable=True).indices
        rank = torch.argsort(order, 1)
        pick = torch.where((rank < case["kept"])[:, :, None], each, -math.inf).view(T, E)
    top, experts = torch.sort(pick, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    none = top == -math.inf
    w = torch.where(none, 0.0, p.gather(1, experts))
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return (w * case["scale"]).float(), torch.where(none, -1, experts).int()


def _plain_route_backward(s):
    case, x = s["case"], s["logits"].float()
    none = s["experts"] < 0
    at = torch.where(none, 0, s["experts"]).long()
    g = torch.where(none, 0.0, s["dweights"] * case["scale"])
    if case["scoring"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e30))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        p = 1 / (1 + torch.exp(-x))
    chosen = torch.where(none, 0.0, p.gather(1, at))
    if case["renormalize"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-30)
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    g = torch.where(none, 0.0, g)
    dp = torch.zeros_like(p).scatter_add_(1, at, g)
    if case["scoring"] == "softmax":
        d = p * (dp - (dp * p).sum(1, keepdim=True))
    else:
        d = dp * p * (1 - p)
    return d.to(s["logits"].dtype)


def _ratio(a, b):
    """a / b rounded once to 32 bits (torch multiplies by a number's reciprocal)."""
    a, b = (torch.as_tensor(v, dtype=torch.float64, device=DEV) for v in (a, b))
    return (a / b).float()


def _blocks(x, dim):
    """x in 8 bits with a scale for each 128 along `dim` (a multiple of 128): the values that stand for it."""
    b = x.unflatten(dim, (-1, 128))
    most = b.abs().amax(dim + 1, keepdim=True).clamp(min=FLOOR)
    return ((b * _ratio(F8_MAX, most)).to(F8).float() * _ratio(most, F8_MAX)).flatten(dim, dim + 1)


def _pad(x, n):
    return torch.nn.functional.pad(x, (0, n - x.shape[-1]))


def _places(s, multiple):
    """Where each row lies among rows padded to the same number for each expert, the last place for dropped ones."""
    off, n = s["offsets"], s["position"].numel()
    most = max(1, int(off.diff().max()))
    most = -(-most // multiple) * multiple
    row = torch.arange(n, device=DEV)
    e = torch.searchsorted(off, row, right=True) - 1
    kept = row < off[-1]
    e = torch.where(kept, e, 0)
    return torch.where(kept, e * most + row - off[e], s["case"]["E"] * most), most, kept


def _plain_experts(s):
    case = s["case"]
    E, k, K, N = case["E"], case["k"], case["K"], case["N"]
    kb, nb = -(-K // 128), -(-N // 128)
    place, most, kept = _places(s, 1)
    x = _blocks(_pad(s["x"].float(), kb * 128), 1)[:, :K]
    order = torch.empty_like(place)
    order[s["position"].view(-1).long()] = torch.arange(place.numel(), device=DEV)
    rows = torch.zeros(E * most + 1, K, device=DEV)
    rows[place] = x[order // k]
    scales = s["wscales"].repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :N, :K]
    w = (s["w"].float() * scales).transpose(1, 2).contiguous()
    out = torch.bmm(rows[:-1].view(E, most, K), w).view(E * most, N)
    out = torch.where(kept[:, None], out[place.clamp(max=E * most - 1)], 0.0)
    return out.to(DTYPES[case["out"]])


def _plain_weights_gradient(s):
    case = s["case"]
    E, K, N = case["E"], case["K"], case["N"]
    place, most, _ = _places(s, 128)
    x = torch.zeros(E * most + 1, K, device=DEV)
    x[place] = s["x"].float()
    d = torch.zeros(E * most + 1, N, device=DEV)
    d[place] = s["dout"].float()
    x = _blocks(x[:-1].view(E, most, K), 1)
    d = _blocks(d[:-1].view(E, most, N), 1).transpose(1, 2).contiguous()
    return torch.bmm(d, x).to(DTYPES[case["out"]])


def _plain_verify(s):
    case, off = s["case"], s["offsets"]
    R, V, D = case["R"], case["V"], s["tokens"].numel()
    t = case["temperature"]
    draft = torch.arange(D, device=DEV)
    request = torch.searchsorted(off, draft, right=True) - 1
    x = s["target"].double()
    if t > 0:
        p = torch.exp((x - x.amax(1, keepdim=True)) / t)
        p = p / p.sum(1, keepdim=True)
    else:
        best = x == x.amax(1, keepdim=True)
        p = (best & (best.cumsum(1) == 1)).double()
    hot = torch.nn.functional.one_hot(s["tokens"], V) if D else torch.zeros(0, V, device=DEV)
    if s["draft"] is not None and t > 0:
        y = s["draft"].double()
        q = torch.exp((y - y.amax(1, keepdim=True)) / t)
        q = q / q.sum(1, keepdim=True)
    else:
        q = hot.double()
    at = s["tokens"][:, None]
    took = s["accept"].double() * q.gather(1, at)[:, 0] < p[draft + request].gather(1, at)[:, 0]
    # The first that is turned down of each request, or the end of its drafts.
    stop = off[1:].scatter_reduce(0, request, torch.where(took, D, draft), "amin")
    ended = stop == off[1:]
    row = stop + torch.arange(R, device=DEV)
    q = torch.cat([q, torch.zeros(1, V, dtype=torch.float64, device=DEV)])
    rest = (p[row] - q[torch.where(ended, D, stop)]).clamp(min=0)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p[row])
    c = rest.cumsum(1)
    last = (c <= s["sample"].double()[:, None] * c[:, -1:]).sum(1).clamp(max=V - 1)
    tokens = torch.full((D + R,), -1, dtype=torch.int64, device=DEV)
    tokens[draft + request] = torch.where(draft < stop[request], s["tokens"], -1)
    tokens[row] = last
    return tokens, (stop - off[:-1] + 1).int()


def _plain(s):
    case = s["case"]
    if case["kind"] == "route":
        return _plain_route_backward(s) if case["backward"] else _plain_route(s)
    if case["kind"] == "experts":
        return _plain_weights_gradient(s) if case["backward"] else _plain_experts(s)
    return _plain_verify(s)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if not own:
        return _plain(s)
    import segmented_top_selection_amd as st
    case = s["case"]
    if case["kind"] == "route":
        how = dict(scoring=case["scoring"], renormalize=case["renormalize"], scale=case["scale"])
        if case["backward"]:
            return st.route_backward(s["dweights"], s["logits"], s["experts"], **how)
        return st.route(s["logits"], case["k"], bias=s["bias"], groups=case["groups"],
                        kept_groups=case["kept"], group_best=case["best"], **how)
    if case["kind"] == "experts":
        dtype = DTYPES[case["out"]]
        if case["backward"]:
            return st.expert_matmul_dweights(s["dout"], s["x"], s["offsets"], dtype=dtype)
        rows, scales = st.dispatch_quantized(s["x"], s["position"], s["offsets"])
        return st.expert_matmul(rows, scales, s["w"], s["wscales"], s["offsets"], dtype=dtype)
    return st.verify_drafts(s["target"], s["tokens"], s["offsets"], s["accept"], s["sample"],
                            draft_logits=s["draft"], temperature=case["temperature"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(case, s):
    x, E, G, k = s["logits"].double(), case["E"], case["groups"], case["k"]
    column = torch.arange(E, device=DEV)
    p = torch.softmax(x, 1).nan_to_num(0.0) if case["scoring"] == "softmax" else torch.sigmoid(x)
    if case["backward"]:
        # By automatic differentiation of the weights.
        x = torch.where(x == -math.inf, -1e4, x).requires_grad_()
        p = torch.softmax(x, 1) if case["scoring"] == "softmax" else torch.sigmoid(x)
        none = s["experts"] < 0
        w = torch.where(none, 0.0, torch.take_along_dim(p, s["experts"].long().clamp(min=0), 1))
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        (w * case["scale"] * s["dweights"].double()).sum().backward()
        return x.grad
    score = p + (0.0 if s["bias"] is None else s["bias"].double())
    free = x > -math.inf
    if G > 1:
        # A group is kept if fewer than `kept` are before it.
        g = torch.where(free, score, -math.inf).view(-1, G, E // G).sort(2, descending=True).values
        value = g[:, :, 0] if case["best"] == 1 or E == G else g[:, :, 0] + g[:, :, 1].clamp(min=-1e9) * (g[:, :, 1] > -math.inf)
        a, b = value[:, :, None], value[:, None, :]
        i = torch.arange(G, device=DEV)
        before = ((b > a) | ((b == a) & (i[None, :] < i[:, None]))).sum(2)
        free = free & (before < case["kept"]).repeat_interleave(E // G, 1)
    picked = []
    for _ in range(k):
        best = torch.where(free, score, -math.inf).amax(1, keepdim=True)
        at = torch.where(free & (score == best), column, E).amin(1, keepdim=True)
        picked.append(torch.where(at < E, torch.take_along_dim(p, at.clamp(max=E - 1), 1), 0.0))
        free = free & (column != at)
    w = torch.cat(picked, 1)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return w * case["scale"], None


def _eight_bits(x):
    """x (n, up to 128 numbers): the values that stand for them."""
    most = torch.linalg.vector_norm(x, math.inf, dim=1, keepdim=True).clamp(min=FLOOR)
    down, up = F8_MAX / most.double(), most.double() / F8_MAX
    return (x * down.float()).to(F8).double() * up.float().double()


def _exact_experts(case, s):
    off, K, N = s["offsets"].tolist(), case["K"], case["N"]
    if case["backward"]:
        out = torch.zeros(case["E"], N, K, dtype=torch.float64, device=DEV)
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            for i in range(a, b, 128):
                d, x = (_eight_bits(t[i:min(i + 128, b)].float().t()) for t in (s["dout"], s["x"]))
                out[e].addmm_(d, x.t())
        return out
    x = torch.cat([_eight_bits(s["x"][:, i:i + 128].float()) for i in range(0, K, 128)], 1)
    token = torch.argsort(s["position"].view(-1)) // case["k"]
    out = torch.zeros(token.numel(), N, dtype=torch.float64, device=DEV)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if a < b:
            w = s["w"][e].double()
            for i in range(0, N, 128):
                w[i:i + 128] *= s["wscales"][e, i // 128].double().repeat_interleave(128)[:K]
            out[a:b] = x[token[a:b]] @ w.t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "route":
        return _exact_route(case, s)
    if case["kind"] == "experts":
        return _exact_experts(case, s)
    return None  # whole numbers
