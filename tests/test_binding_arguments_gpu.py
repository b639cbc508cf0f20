"""What the binding takes and refuses."""
import numpy as np
import pytest
import torch

import segmented_top_selection_amd as st
from test_model_ops_gpu import DEV

pytestmark = pytest.mark.gpu


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
