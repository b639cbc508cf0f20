"""What the binding takes and refuses, and what it tells autograd."""
import numpy as np
import pytest
import torch

import segmented_top_selection_amd as st
from test_model_ops_gpu import DEV, gen, randn

pytestmark = pytest.mark.gpu

CALLS = ["dispatch", "combine", "dispatch_backward", "combine_backward", "embedding", "embedding_backward",
         "accumulate", "dlogits", "logits", "stream"]


@pytest.mark.parametrize("bad", [7.0, 7.9, "7", None, [7], torch.tensor(7.5)])
def test_sizes_that_are_no_integers_are_refused(bad):
    x, ids = torch.zeros(4, 8, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        st.sort_ids(ids, bad)
    with pytest.raises(TypeError):
        st.embedding_backward(x, ids, bad)
    if bad is not None:
        with pytest.raises(TypeError):
            st.embedding_backward(x, ids, 9, padding_id=bad)


@pytest.mark.parametrize("kind", [int, np.int32, np.int64, np.uint8, torch.tensor])
def test_sizes_of_every_integer_type(kind):
    ids = torch.tensor([1, 6, 0, 7], device=DEV)
    assert st.sort_ids(ids, kind(7))[2].tolist() == [0, 1, 2, 2, 2, 2, 2, 3]
    d = st.embedding_backward(torch.ones(4, 2, device=DEV), ids, kind(8), padding_id=kind(6))
    assert d[:, 0].tolist() == [1, 1, 0, 0, 0, 0, 0, 1]


def writes(buffer):
    """Each call that writes into a caller's tensor, by name."""
    g = gen(3)
    x, ids = randn(g, 6, 8), torch.tensor([0, 3, 1, 5, 3, 2], device=DEV)
    position = torch.randperm(6, generator=g, device=DEV).int()
    f, answers = randn(g, 6), torch.tensor([0, 6], device=DEV)
    return {
        "dispatch": lambda: st.dispatch(x, position, out=buffer),
        "combine": lambda: st.combine(x, position, out=buffer),
        "dispatch_backward": lambda: st.dispatch_backward(x, position, out=buffer),
        "combine_backward": lambda: st.combine_backward(x, x, position, out=buffer),
        "embedding": lambda: st.embedding(x, ids, out=buffer),
        "embedding_backward": lambda: st.embedding_backward(x, ids, 6, out=buffer),
        "accumulate": lambda: st.embedding_backward(x, ids, 6, out=buffer, accumulate=True),
        "dlogits": lambda: st.policy_loss_grad(x, ids, f, f, answers, dlogits=buffer),
        "logits": lambda: st.policy_loss_grad(buffer, ids, f, f, answers, dlogits=buffer),
        "stream": lambda: st.embedding(x, ids, out=buffer, stream=torch.cuda.current_stream()),
    }


@pytest.mark.parametrize("name", CALLS)
def test_autograd_is_told_of_what_is_overwritten(name):
    buffer = randn(gen(4), 6, 8)
    w = randn(gen(5), 6, 8).requires_grad_()
    loss = (w * buffer).sum()  # keeps buffer for w's gradient
    before = buffer._version
    writes(buffer)[name]()
    assert buffer._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inputs_and_tensors_outside_autograd_are_left_as_they_were():
    g = gen(6)
    x, ids = randn(g, 6, 8), torch.arange(6, device=DEV)
    st.embedding(x, ids)
    assert x._version == ids._version == 0
    with torch.inference_mode():
        out = torch.empty(6, 8, device=DEV)
        st.embedding(x, ids, out=out)
    st.embedding(x, ids, out=out)  # has no version to count
    assert torch.equal(out, x)


@pytest.mark.parametrize("count", [-1, 2 ** 31 - 1, 2 ** 40, 2 ** 63 - 1])
def test_counts_past_the_limits_are_refused_before_anything_is_allocated(count):
    x, ids = torch.zeros(4, 8, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    held = torch.cuda.max_memory_allocated()
    with pytest.raises(ValueError):
        st.sort_ids(ids, count)
    with pytest.raises(ValueError):
        st.embedding_backward(x, ids, count)
    assert torch.cuda.max_memory_allocated() == held
