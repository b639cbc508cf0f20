"""The operators around the selection at the sizes where their kernels change:
one launch or several, rows held in registers or read again, outputs stored past
the caches, many rows arriving at the loss.  Tolerances as in
test_model_ops_gpu."""
import math

import pytest
import torch

import segmented_top_selection_amd as st
from test_model_ops_gpu import (DEV, IDS, TYPES, U, check_policy, check_sort, close, everything,
                                exact_table, gen, move_all, policy_inputs, randn, run_policy, same_bits,
                                some_state)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("segments", [128, 511, 512, 30000])
@pytest.mark.parametrize("n", [15, 16, 17, 1024, 4096, 5119, 5120, 5121, 6145, 9001, 15360, 15361,
                               20480, 20481, 131073])
def test_sort_ids_where_its_launches_change(n, segments):
    ids = torch.randint(-1, segments + 1, (n,), generator=gen(n + segments), device=DEV)
    check_sort(ids, segments)


@pytest.mark.parametrize("n", [15360, 40000, 1100000])
@pytest.mark.parametrize("segments", [300, 70000])
def test_sort_ids_of_one_id(n, segments):
    for v in (0, segments - 1, segments):
        check_sort(torch.full((n,), v, dtype=torch.int32, device=DEV), segments)


def test_sort_ids_in_many_chunks():
    # Above 2^20 ids the chunks are whole blocks, and up to 256 of them.
    for n in ((1 << 20) + 1, (1 << 21) + 8193, 5000011):
        check_sort(torch.randint(0, 200, (n,), generator=gen(n), device=DEV), 200)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_large_outputs_of_odd_width(dtype):
    # 128 MiB and more of rows, which are stored past the caches.
    tokens = 5000 if dtype == torch.float32 else 10000
    move_all(gen(41), tokens, 3, 2305, dtype, torch.float32, 0.1)
    g = gen(42)
    table = randn(g, 300, 2305, dtype=dtype)
    ids = torch.randint(-1, 301, (3 * tokens,), generator=g, device=DEV)
    there = (ids >= 0) & (ids < 300)
    got = st.embedding(table, ids)
    assert torch.equal(got, table[ids.clamp(0, 299)] * there[:, None])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("n,num_rows,width", [
    (40000, 300, 24),      # chunks of 64 rows
    (33001, 5000, 2100),   # two workgroups side by side over a row
    (15361, 70000, 33),    # ids sorted in several launches, the table cleared beside them
    (9000, 40000, 1001),
    (100, 70001, 1025),    # a table of 128 MiB and more, an odd number of bytes past 16
    (5, 3, 3), (20000, 100, 1),
])
def test_embedding_backward_at_other_sizes(n, num_rows, width, dtype):
    g = gen(n + width)
    dout = randn(g, n, width, dtype=dtype)
    # As skewed as text, so that runs cross many chunks.
    ids = (num_rows ** torch.rand(n, generator=g, device=DEV, dtype=torch.float64)).long() - 1
    exact, inner, touched = exact_table(dout, ids, num_rows, padding=1)
    out = torch.full((num_rows, width), float("nan"), dtype=dtype, device=DEV)
    got = st.embedding_backward(dout, ids, num_rows, padding_id=1, out=out)
    assert got is out
    close(got, exact, inner)
    assert not bool(got[~touched].any())
    # A table at an address between multiples of 16 bytes, and rows apart from each other.
    flat = torch.full((num_rows * width + 1,), float("nan"), dtype=dtype, device=DEV)
    st.embedding_backward(dout, ids, num_rows, padding_id=1, out=flat[1:].view(num_rows, width))
    assert torch.equal(flat[1:].view(num_rows, width), got) and math.isnan(float(flat[0]))
    wide = torch.full((num_rows, width + 5), 3.0, dtype=dtype, device=DEV)
    st.embedding_backward(dout, ids, num_rows, padding_id=1, out=wide[:, 2:-3])
    assert torch.equal(wide[:, 2:-3], got)
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, -3:] == 3).all())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("kib", [16, 32, 64, 128])
def test_policy_rows_where_the_workgroup_changes(kib, dtype):
    whole = kib * 1024 // dtype.itemsize
    for V in (whole - 1, whole, whole + 1, whole + 9):
        q = policy_inputs(gen(V), 3, V, 1, dtype)
        want = check_policy(q, 0.1)
        for a, b in zip(want, run_policy(q, 0.1, dlogits=q["logits"])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,S", [(63, 5), (64, 1), (65, 64), (128, 2), (129, 7), (5003, 1), (5003, 4000), (129, 70000)])
def test_policy_loss_of_many_rows(T, S):
    # Terms of both signs that nearly cancel.  A row's log-probability is off by its
    # sum's error alone, relative: 20 additions deep, a product, its exponent's error
    # and the exponential's own (40 halves of a step); then 64 bits.
    q = policy_inputs(gen(T + S), T, 50, S, torch.float32, masked=0.2)
    q["adv"] -= q["adv"].mean()
    z = torch.log_softmax(q["logits"].double(), 1)
    live = (q["tokens"] >= 0) & (q["tokens"] < 50)
    lp = z.gather(1, q["tokens"].clamp(0, 49)[:, None])[:, 0]
    r, A = (lp - q["old"].double()).exp(), q["adv"].double()
    term = -torch.minimum(r * A, r.clamp(0.8, 1.2) * A)
    seg = torch.searchsorted(q["offsets"], torch.arange(T, device=DEV), right=True) - 1
    n = torch.zeros(S, dtype=torch.float64, device=DEV).index_add_(0, seg, live.double())
    weight = live / (S * n[seg]).clamp(min=1)
    exact, size = float((weight * term).sum()), float((weight * r.clamp(min=1) * A.abs()).sum())
    for _ in range(3):
        loss, got, d = run_policy(q, 0.0)
        assert abs(float(loss) - exact) <= 40 * U * size + U * abs(exact)
        assert bool(((got.double() - torch.where(live, lp, 0.0)).abs() <= 40 * U + U * lp.abs()).all())
        # The gradient of a row adds up to nothing.
        slope = (weight * r * A.abs())[:, None]
        assert bool((d.double().sum(1, keepdim=True).abs() <= 60 * U * slope + 1e-30).all())


def test_temperatures_far_from_one():
    q = policy_inputs(gen(50), 6, 300, 2, torch.float32, masked=0.0)
    for temperature in (1e-3, 30.0, 1e6):
        check_policy(q, 0.0, temperature)
    q["tokens"] = q["logits"].argmax(1)
    _, lp = st.policy_loss(q["logits"], q["tokens"], q["old"], q["adv"], q["offsets"], temperature=1e-30)
    assert bool((lp == 0).all())  # certain


def large_state(seed):
    s, g, T = some_state(seed), gen(seed + 1000), 9000
    s["ids"] = torch.randint(-1, 9, (T, 2), generator=g, device=DEV)
    s["x"], s["w"] = randn(g, T, 96).bfloat16(), torch.rand(T, 2, generator=g, device=DEV)
    s["tokens"] = torch.randint(0, 300, (T,), generator=g, device=DEV)
    s["logits"], s["old"] = randn(g, T, 300), -torch.rand(T, generator=g, device=DEV) * 6
    s["adv"] = randn(g, T)
    s["answers"] = torch.tensor([0, 50, 4000, T], device=DEV)
    return s


def test_a_graph_of_the_calls_in_several_launches():
    s = large_state(51)
    table = torch.empty(40000, 96, device=DEV)

    def calls(s):
        some = s["x"].float()
        far = s["tokens"].repeat(2) * 131 % 40000
        return everything(s) + [st.embedding_backward(some.repeat(2, 1), far, 40000, out=table).clone()]
    calls(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(s)
    for seed in (52, 53, 51):
        new = large_state(seed)
        for name, v in new.items():
            s[name].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        kept = [v.clone() for v in outs]
        assert same_bits(calls(new), kept)
        torch.cuda.synchronize()


def test_inputs_freed_before_their_stream_has_used_them():
    g = gen(60)
    side = torch.cuda.Stream()
    table = randn(g, 700, 129)
    want = table.clone()
    ids = torch.arange(700, device=DEV).flip(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20000000)
    got = st.embedding(table, ids, stream=side)
    del table, ids
    for _ in range(4):  # would be given the same memory
        torch.full((700, 129), -1.0, device=DEV)
        torch.zeros(700, dtype=torch.int64, device=DEV)
    side.synchronize()
    assert torch.equal(got, want.flip(0))
    with pytest.raises(ValueError):
        st.embedding(want.cpu(), torch.zeros(3, dtype=torch.int64), stream=side)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("n,num_rows,width", [
    (2, 1, 1), (7, 100, 513), (255, 3, 64), (256, 2, 65), (257, 900, 7), (1024, 30, 512),
    (1024, 5, 1024), (1024, 3, 1025), (1025, 40, 100), (128, 9, 8191), (1, 70000, 5), (600, 1, 40)])
def test_embedding_backward_of_few_tokens(n, num_rows, width, dtype):
    g = gen(n + width)
    for what in ("random", "same", "ends"):
        ids = torch.randint(-1, num_rows + 1, (n,), generator=g, device=DEV)
        if what == "same":
            ids[:] = num_rows - 1
        elif what == "ends":  # an id's first and last token far apart
            ids[[0, -1]] = num_rows // 2
        dout = randn(g, n, width, dtype=dtype)
        for padding in (None, 0):
            exact, inner, touched = exact_table(dout, ids, num_rows, padding)
            out = torch.full((num_rows, width + 3), 5.0, dtype=dtype, device=DEV)
            got = st.embedding_backward(dout, ids, num_rows, padding_id=padding, out=out[:, 1:-2])
            close(got, exact, inner)
            assert not bool(got[~touched].any())
            assert bool((out[:, :1] == 5).all()) and bool((out[:, -2:] == 5).all())
            assert torch.equal(got, st.embedding_backward(dout, ids.int(), num_rows, padding_id=padding))
            base = randn(g, num_rows, width)
            res = st.embedding_backward(dout, ids, num_rows, padding_id=padding, out=base.clone(),
                                        accumulate=True)
            assert torch.equal(res[~touched], base[~touched])
            total = exact + base.double()
            close(res, total, inner + U * (total.abs() + exact.abs()))
