"""Rows of the policy loss that hold NaN, infinities, or a sampled token that is
ruled out."""
import math

import pytest
import torch

import segmented_top_selection_amd as st
from test_model_ops_gpu import DEV, IDS, TYPES, gen, policy_inputs, run_policy, same_bits

pytestmark = pytest.mark.gpu

# Rows of one or two pieces, of several groups of pieces, and of more than a
# workgroup holds; all with elements past the last whole piece.
VOCABS = [43, 9001, 140001]


def poisoned(q, what, row):
    """q with one live row's value replaced."""
    q = {n: v.clone() for n, v in q.items()}
    V, token = q["logits"].shape[1], int(q["tokens"][row])
    where, value = {"nan logit": ((token + V // 2) % V, math.nan), "nan at the token": (token, math.nan),
                    "nan at the end": (V - 1, math.nan), "nan everywhere": (slice(None), math.nan),
                    "inf logit": ((token + V // 2) % V, math.inf), "inf at the token": (token, math.inf),
                    "inf at the end": (V - 1, math.inf)}.get(what, (None, math.nan))
    if where is None:
        q[what][row] = value
    else:
        q["logits"][row, where] = value
    return q


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_nan_of_a_live_row_reaches_loss_and_gradient(kl, V, dtype):
    q = policy_inputs(gen(V), 6, V, 2, dtype, masked=0.0)
    _, lp, d = run_policy(q, kl)
    kinds = ["nan logit", "nan at the token", "nan at the end", "nan everywhere", "inf logit",
             "inf at the token", "inf at the end", "old", "adv"] + (["ref"] if kl else [])
    for i, what in enumerate(kinds):
        row = i % 6
        others = torch.arange(6, device=DEV) != row
        for advantage in (1.0, -1.0):
            q["adv"][row] = advantage
            bad = poisoned(q, what, row)
            got = run_policy(bad, kl)
            assert math.isnan(float(got[0])), what
            assert bool(got[2][row].isnan().all()), what
            assert math.isnan(float(got[1][row])) == (what not in ("old", "adv", "ref")), what
            assert torch.equal(got[1][others], lp[others]) and torch.equal(got[2][others], d[others]), what
            alone = run_policy(bad, kl, fn=st.policy_loss)
            assert math.isnan(float(alone[0])) and same_bits(alone[1:], got[1:2])
            into = run_policy(bad, kl, dlogits=bad["logits"])
            assert bool(into[2][row].isnan().all()) and torch.equal(into[2][others], d[others]), what
        q["adv"][row] = policy_inputs(gen(V), 6, V, 2, dtype, masked=0.0)["adv"][row]


@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_no_advantage_and_a_ratio_past_the_range(kl):
    # exp(logp - old_logp) overflows 64 bits; times no advantage it is still nothing.
    q = policy_inputs(gen(7), 4, 50, 1, torch.float32, masked=0.0)
    q["old"][1], q["adv"][1] = -1000.0, 0.0
    loss, _, d = run_policy(q, kl)
    q["old"][1] = 0.0
    want = run_policy(q, kl)
    assert math.isfinite(float(loss)) and torch.equal(loss, want[0]) and torch.equal(d, want[2])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("advantage", [1.0, -1.0, 0.0])
def test_a_sampled_token_that_is_ruled_out(advantage, V, dtype):
    # Its probability is zero and so is its ratio: the clipped term is finite.  The KL
    # term grows past every bound as a logit falls, and with it the slope in logp, by
    # which the row's gradient, slope (1[c = token] - p_c), is multiplied.
    q = policy_inputs(gen(V + 1), 6, V, 2, dtype, masked=0.0, scale=1.0)
    q["adv"][2] = advantage
    _, lp, d = run_policy(q, 0.05)
    others = torch.arange(6, device=DEV) != 2
    out = torch.arange(V, device=DEV) % 3 == 1
    for token in (1, V // 3 * 3 - 2):
        q["logits"][2, out] = -math.inf
        q["tokens"][2] = token
        bad = {n: v.clone() for n, v in q.items()}
        for scale in (1.0, -2.0):
            got = run_policy(bad, 0.05, grad_scale=scale)
            assert float(got[0]) == math.inf and float(got[1][2]) == -math.inf
            want = torch.where(out, 0.0, math.inf)
            want[token] = -math.inf
            assert torch.equal(got[2][2].float(), want * scale if scale > 0 else -want)
            assert torch.equal(got[1][others], lp[others])
            if scale == 1.0:
                assert torch.equal(got[2][others], d[others])
        alone = run_policy(bad, 0.05, fn=st.policy_loss)
        assert float(alone[0]) == math.inf and torch.equal(alone[1], got[1])
        into = run_policy(bad, 0.05, grad_scale=-2.0, dlogits=bad["logits"])
        assert torch.equal(into[2], got[2])
        # Without the KL term all is finite; where the unclipped side counts, it is zero.
        loss, _, free = run_policy(q, 0.0)
        assert math.isfinite(float(loss)) and not bool(free[2].any())


@pytest.mark.parametrize("token", [3, 42])
def test_a_reference_without_the_sampled_token(token):
    # ref_logp of -inf: the KL term is infinite, its slope is not.
    q = policy_inputs(gen(9), 4, 43, 1, torch.float32, masked=0.0)
    q["tokens"][1], q["adv"][1] = token, 0.0
    q["ref"][1] = -math.inf
    loss, _, d = run_policy(q, 0.05)
    assert float(loss) == math.inf
    p = torch.softmax(q["logits"][1].double(), 0)
    hot = torch.zeros_like(p)
    hot[token] = 1.0
    want = 0.05 / 4 * (hot - p)
    # Two roundings of the slope, its product, the exponent's six, the exponential's.
    assert bool(((d[1].double() - want).abs() <= 40 * 2.0 ** -24 * (0.05 / 4) * (hot + p)).all())
