"""Norms around a block at the ends of their range: empty batches, sizes that are refused."""
import pytest
import torch

from activation_sparse_transformer_tma_b200 import build as tw_build
from activation_sparse_transformer_tma_b200 import twell


@pytest.fixture(scope="module")
def L():
    tw_build.build()
    return twell.lib()


@pytest.mark.parametrize("group", [0, 1, 7, 2 ** 31 - 1])
def test_workspace_of_an_empty_batch_and_of_refused_sizes_is_empty(L, group):
    size = L.norm_residual_backward_workspace_size
    assert size(0, 64, group) == 0
    for T, d in ((-1, 64), (10, 0), (10, -8), (10, 60), (10, 8200), (10, 2 ** 31 - 8)):
        assert size(T, d, group) == 0, (T, d)
    assert size(10, 64, -1) == 0
    for T, d in ((1, 8), (10, 64), (2 ** 31 - 1, 8192)):
        # a partial row of each of the two vectors' gradients at least
        assert size(T, d, group) >= 2 * 4 * d, (T, d)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 1, 5])
def test_backward_of_an_empty_batch_with_the_workspace_it_asks_for(group):
    d = 72
    e = torch.empty((0, d), device="cuda")
    q = torch.empty(0, device="cuda")
    w = torch.ones(d, device="cuda")
    dw = torch.full((2, d), 7.0, device="cuda")
    ws = twell.norm_residual_backward_workspace(0, d, group)
    gate = e if group else None
    twell.norm_residual_backward(e, e, e, e, w, gate, w, q, q, e, e, dw[0],
                                 e.clone() if group else None, dw[1], ws, gate_group=group)
    torch.cuda.synchronize()
    assert (dw == 0).all()
