"""The gradient of an embedding table without any tokens, on tables past the size
that one launch takes."""
import pytest
import torch

import segmented_top_selection_amd as st
from segmented_top_selection_amd import model_ops as mo
from test_model_ops_gpu import DEV, IDS, TYPES

pytestmark = pytest.mark.gpu

ROWS, WIDTH = 65537, 4097  # 2^28 elements and more


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_no_tokens_and_a_large_table(dtype):
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    dout = torch.empty(0, WIDTH, dtype=dtype, device=DEV)
    out = torch.full((ROWS, WIDTH), 3.0, dtype=dtype, device=DEV)
    assert st.embedding_backward(dout, none, ROWS, out=out) is out
    assert not bool(out.any())
    out.fill_(3.0)
    st.embedding_backward(dout, none.int(), ROWS, out=out, accumulate=True)
    assert bool((out == 3.0).all())
    del out
    wide = torch.full((ROWS, WIDTH + 2), 3.0, dtype=dtype, device=DEV)  # rows apart from each other
    st.embedding_backward(dout, none, ROWS, out=wide[:, 1:-1])
    assert not bool(wide[:, 1:-1].any())
    assert bool((wide[:, 0] == 3.0).all()) and bool((wide[:, -1] == 3.0).all())


@pytest.mark.parametrize("rows,width", [(7, 33), (ROWS, WIDTH)])
def test_no_tokens_and_null_pointers(rows, width):
    table = torch.full((rows, width), 3.0, dtype=torch.bfloat16, device=DEV)
    call = mo.entry("segtopk_embedding_backward")
    stream = torch.cuda.current_stream().cuda_stream
    assert mo.entry("segtopk_embedding_backward_workspace")(0, rows, width) == 0
    for accumulate in (1, 0):
        view = mo._Rows(table.data_ptr(), width, 1)
        assert call(None, view, None, 8, 0, rows, width, 1.0, -1, accumulate, None, 0, stream) == 0
        torch.cuda.synchronize()
        assert bool((table == 3.0).all()) if accumulate else not bool(table.any())
