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
