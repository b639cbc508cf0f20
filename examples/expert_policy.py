"""A small mixture-of-experts model trained by sampling, on the library's operators.

The model reads one token and scores the next:

    h   = scale * table[token]
    e   = the top 2 of 8 experts by h W_router, weighted by the softmax of their scores
    out = (h + sum_e weight_e relu(h A_e) B_e) W_out

Both selections are ``batched_topk``: over each token's expert scores, and over
each row of logits, from whose best entries the next token is drawn.  Between
them stand ``embedding``, ``sort_ids``, ``dispatch`` and ``combine``; the answers
are scored by ``policy_loss`` and trained on by ``policy_loss_grad``, and the
gradient goes back through ``combine_backward``, ``dispatch_backward`` and
``embedding_backward``.  An answer's reward is its share of even tokens.

    python examples/expert_policy.py --steps 120

prints the mean reward as it rises from a half to above nine tenths.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import segmented_top_selection_amd as st  # noqa: E402

VOCAB, WIDTH, HIDDEN, EXPERTS, PER_TOKEN = 512, 96, 128, 8, 2
SCALE = math.sqrt(WIDTH)
KL, CLIP_LOW, CLIP_HIGH = 0.02, 0.2, 0.28
NORM = 0.3  # of the gradient, at most


def init(seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def matrix(*shape):
        return torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[-2])
    return {"table": torch.randn(VOCAB, WIDTH, generator=g, device=device) / SCALE,
            "router": matrix(WIDTH, EXPERTS), "up": matrix(EXPERTS, WIDTH, HIDDEN),
            "down": matrix(EXPERTS, HIDDEN, WIDTH), "out": matrix(WIDTH, VOCAB)}


def rows_of(n, width, device):
    """Offsets of n segments of equal width: the rows of a matrix."""
    return torch.arange(n + 1, device=device) * width


def forward(p, tokens):
    """The logits of the token after each of `tokens`, and what the gradient needs."""
    dev, n = tokens.device, tokens.numel()
    h = st.embedding(p["table"], tokens, scale=SCALE)
    scores = h @ p["router"]
    expert = torch.arange(EXPERTS, dtype=torch.int32, device=dev).repeat(n)
    best, chosen = st.batched_topk(scores.view(-1), rows_of(n, EXPERTS, dev), PER_TOKEN, values=expert,
                                   max_segment_size=EXPERTS)
    weights = torch.softmax(best, 1)
    _, position, offsets = st.sort_ids(chosen, EXPERTS)
    rows = st.dispatch(h, position, offsets)
    bounds = offsets.tolist()
    y, mid = torch.empty_like(rows), torch.empty(rows.shape[0], HIDDEN, device=dev)
    for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        mid[a:b] = torch.relu(rows[a:b] @ p["up"][e])
        torch.mm(mid[a:b], p["down"][e], out=y[a:b])
    mixed = h + st.combine(y, position, offsets, weights)
    return mixed @ p["out"], dict(tokens=tokens, h=h, chosen=chosen, weights=weights, position=position,
                                  offsets=offsets, bounds=bounds, rows=rows, mid=mid, y=y, mixed=mixed)


def backward(p, s, dlogits):
    """The gradients of the parameters."""
    d = {"out": s["mixed"].t() @ dlogits, "up": torch.zeros_like(p["up"]),
         "down": torch.zeros_like(p["down"])}
    dmixed = dlogits @ p["out"].t()
    dy, dweights = st.combine_backward(dmixed, s["y"], s["position"], s["offsets"], s["weights"])
    drows = torch.empty_like(dy)
    for e, (a, b) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        d["down"][e] = s["mid"][a:b].t() @ dy[a:b]
        dmid = (dy[a:b] @ p["down"][e].t()) * (s["mid"][a:b] > 0)
        d["up"][e] = s["rows"][a:b].t() @ dmid
        drows[a:b] = dmid @ p["up"][e].t()
    w = s["weights"]
    dbest = w * (dweights - (w * dweights).sum(1, keepdim=True))
    dscores = torch.zeros(w.shape[0], EXPERTS, device=w.device).scatter_(1, s["chosen"].long(), dbest)
    d["router"] = s["h"].t() @ dscores
    dh = dmixed + st.dispatch_backward(drows, s["position"], s["offsets"]) + dscores @ p["router"].t()
    d["table"] = st.embedding_backward(dh, s["tokens"], VOCAB, scale=SCALE)
    return d


def draw(logits, generator, best=VOCAB // 2):
    """The next token of each row, drawn from its `best` highest logits."""
    n, dev = logits.shape[0], logits.device
    ids = torch.arange(VOCAB, dtype=torch.int32, device=dev).repeat(n)
    top, token = st.batched_topk(logits.view(-1), rows_of(n, VOCAB, dev), best, values=ids,
                                 max_segment_size=VOCAB)
    noise = torch.empty_like(top).exponential_(generator=generator).log()
    return token.gather(1, (top - noise).argmax(1, keepdim=True))[:, 0]


def answers(p, count, length, generator):
    """`count` answers of `length` tokens: (the tokens read, the tokens drawn), answer by answer."""
    token = torch.randint(0, VOCAB, (count,), generator=generator, device=generator.device).int()
    read, drawn = [], []
    for _ in range(length):
        read.append(token)
        token = draw(forward(p, token)[0], generator)
        drawn.append(token)
    return torch.stack(read, 1).view(-1), torch.stack(drawn, 1).view(-1)


def train(steps, count=64, length=16, epochs=2, rate=1.0, seed=0, device="cuda"):
    """Trains a new model; yields (mean reward, loss) of each step."""
    g = torch.Generator(device=device)
    g.manual_seed(seed + 1)
    p = init(seed, device)
    frozen = {n: v.clone() for n, v in p.items()}
    offsets = rows_of(count, length, g.device)
    zero = torch.zeros(count * length, device=device)
    for _ in range(steps):
        read, drawn = answers(p, count, length, g)
        reward = (drawn % 2 == 0).float().view(count, length).mean(1)
        advantage = (reward - reward.mean()) / (reward.std() + 1e-6)
        advantage = advantage.repeat_interleave(length)
        _, old = st.policy_loss(forward(p, read)[0], drawn, zero, zero, offsets)
        _, ref = st.policy_loss(forward(frozen, read)[0], drawn, zero, zero, offsets)
        for _ in range(epochs):
            logits, saved = forward(p, read)
            loss, _, dlogits = st.policy_loss_grad(
                logits, drawn, old, advantage, offsets, ref_logp=ref, kl_coef=KL,
                clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dlogits=logits)
            grads = backward(p, saved, dlogits)
            norm = torch.stack([d.norm() for d in grads.values()]).norm()
            step = rate * (NORM / norm).clamp(max=1.0)
            for name, d in grads.items():
                p[name].sub_(d * step)
        yield float(reward.mean()), float(loss)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=120)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    for i, (reward, loss) in enumerate(train(args.steps, seed=args.seed)):
        print(f"step {i:3d}  reward {reward:.3f}  loss {loss:+.4f}", flush=True)


if __name__ == "__main__":
    main()
