"""The example that runs the operators together: its gradients against automatic
differentiation in 64 bits, and its training."""
import importlib.util
import os

import pytest
import torch

import segmented_top_selection_amd as st

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "expert_policy.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("expert_policy", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain_loss(ex, p, tokens, drawn, chosen, old, ref, adv, answers):
    h = p["table"][tokens] * ex.SCALE
    best = (h @ p["router"]).gather(1, chosen)
    w = torch.softmax(best, 1)
    mixed = h.clone()
    for j in range(ex.PER_TOKEN):
        for e in range(ex.EXPERTS):
            here = (chosen[:, j] == e).nonzero()[:, 0]
            y = torch.relu(h[here] @ p["up"][e]) @ p["down"][e]
            mixed = mixed.index_add(0, here, w[here, j:j + 1] * y)
    lp = torch.log_softmax(mixed @ p["out"], 1).gather(1, drawn[:, None])[:, 0]
    r = (lp - old).exp()
    term = -torch.minimum(r * adv, r.clamp(1 - ex.CLIP_LOW, 1 + ex.CLIP_HIGH) * adv)
    term = term + ex.KL * ((ref - lp).exp() - (ref - lp) - 1)
    return term.view(answers, -1).mean(1).mean(), lp


def test_gradients_of_the_whole_model(ex):
    # In 32 bits every sum along the way is off by at most its length times 2^-24
    # of its magnitudes; the lengths on the longest path (width, hidden, vocabulary,
    # tokens, and the same back) add up to about 2000, which is 1.2e-4, and the sums
    # cancel to no less than a tenth of their magnitudes: 1.2e-3 of the norm.
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    p = ex.init(3)
    answers, length = 12, 10
    read, drawn = ex.answers(p, answers, length, g)
    offsets = ex.rows_of(answers, length, "cuda")
    logits, s = ex.forward(p, read)
    now = torch.log_softmax(logits, 1).gather(1, drawn[:, None].long())[:, 0]
    old = now + 0.3 * torch.randn(now.shape, generator=g, device="cuda")
    ref = now + 0.3 * torch.randn(now.shape, generator=g, device="cuda")
    adv = torch.randn(now.shape, generator=g, device="cuda")
    loss, lp, dlogits = st.policy_loss_grad(logits, drawn, old, adv, offsets, ref_logp=ref, kl_coef=ex.KL,
                                            clip_low=ex.CLIP_LOW, clip_high=ex.CLIP_HIGH)
    got = ex.backward(p, s, dlogits)
    q = {n: v.double().cpu().requires_grad_() for n, v in p.items()}
    exact, elp = plain_loss(ex, q, read.long().cpu(), drawn.long().cpu(), s["chosen"].long().cpu(),
                            *(v.double().cpu() for v in (old, ref, adv)), answers)
    exact.backward()
    assert abs(float(loss) - float(exact.detach())) <= 1e-4
    assert float((lp.cpu().double() - elp.detach()).abs().max()) <= 1e-4
    for name, v in q.items():
        far = float((got[name].double().cpu() - v.grad).norm() / v.grad.norm())
        assert far <= 1.2e-3, f"{name}: {far:.2g}"


def test_training_raises_the_reward(ex):
    rewards = [r for r, _ in ex.train(40)]
    again = [r for r, _ in ex.train(3)]
    assert all(torch.isfinite(torch.tensor(rewards)))
    assert sum(rewards[-5:]) / 5 > sum(rewards[:5]) / 5 + 0.08
    assert again == rewards[:3]
