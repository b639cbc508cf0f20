"""The forms of the row moves, the lookup and the policy loss that large inputs
choose: several rows to a thread, a wave or a workgroup to a token, outputs stored
past the caches."""
import math

import numpy as np
import pytest
import torch

import segmented_top_selection_amd as st
from test_model_ops_gpu import (DEV, IDS, TYPES, U, close, gen, move_all, policy_inputs, randn,
                                run_policy)

pytestmark = pytest.mark.gpu

PIECES = 4 * 256 * 2048  # of 16 bytes: from here on four rows to a thread
STREAMED = 128 << 20     # bytes of an output: from here on past the caches


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("units", [7, 256, 257])  # pieces and single elements of a row
@pytest.mark.parametrize("size", ["below", "four rows", "streamed"])
def test_embedding_of_many_rows(size, units, dtype):
    width = 16 // dtype.itemsize * (units - 1) + 1
    n = {"below": PIECES // units - 1, "four rows": -(-PIECES // units) + 2,
         "streamed": -(-STREAMED // (width * dtype.itemsize)) + 1}[size]
    g = gen(units)
    table = randn(g, 501, width, dtype=dtype)
    ids = torch.randint(-1, 502, (n,), generator=g, device=DEV)
    there = ((ids >= 0) & (ids < 501))[:, None]
    rows = table[ids.clamp(0, 500)]
    out = torch.full((n + 1, width), 5.0, dtype=dtype, device=DEV)
    assert torch.equal(st.embedding(table, ids, out=out[:n]), rows * there)
    assert bool((out[n] == 5.0).all())
    scale = float(np.float32(math.sqrt(width)))
    got = st.embedding(table, ids.int(), scale=scale)
    for b in range(0, n, 1 << 16):  # in pieces: 64 bits of all rows are large
        exact = (rows[b:b + (1 << 16)] * there[b:b + (1 << 16)]).double() * scale
        close(got[b:b + (1 << 16)], exact, U * exact.abs())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("tokens,k,width", [
    (5300, 6, 2305),                  # more than four slots, stored past the caches
    (2047, 3, 1410), (2048, 5, 1410)  # of rows between 128 and 256 pieces of 16 bits
])
def test_moves_of_many_tokens(tokens, k, width, dtype):
    move_all(gen(tokens), tokens, k, width, dtype, dtype, 0.1)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("kib", [2, 16, 32, 64])  # of a row: held by 256, 256, 512 and 1024 threads
def test_policy_gradient_stored_past_the_caches(kib, dtype):
    # One answer a row: each half of the rows by itself, at half the scale, has the same
    # gradient bit by bit, and is stored through the caches.
    V = kib * 1024 // dtype.itemsize - 1
    half = -(-STREAMED // (2 * V * dtype.itemsize)) + 1
    q = policy_inputs(gen(kib), 2 * half, V, 1, dtype, masked=0.2)
    q["offsets"] = torch.arange(2 * half + 1, device=DEV)
    loss, lp, d = run_policy(q, 0.05)
    total, size = 0.0, abs(float(loss))
    for rows in (slice(0, half), slice(half, 2 * half)):
        part = {n: v[rows] for n, v in q.items() if n != "offsets"}
        part["offsets"] = torch.arange(half + 1, device=DEV)
        one, lp1, d1 = run_policy(part, 0.05, grad_scale=0.5)
        assert torch.equal(lp[rows], lp1) and torch.equal(d[rows], d1)
        total += float(one) / 2
        size += abs(float(one)) / 2
    # Each of the three losses is rounded once to 32 bits.
    assert abs(float(loss) - total) <= U * size + 1e-12
    into = run_policy(q, 0.05, dlogits=q["logits"])
    assert torch.equal(into[2], d) and torch.equal(into[0], loss)
