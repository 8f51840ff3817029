"""Gated feed-forward block at sizes that one launch, or 32 bits, cannot hold."""
import pytest
import torch

import ring_all_reduce_scatter_amd as rar

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("hidden,dim", [(40, 72), (1 << 20, 1 << 14)])
def test_no_rows_and_many_weights(hidden, dim):
    """Without rows the weights' gradients become zeros: of the larger size 2^34
    elements each, four to a thread more threads than a launch has."""
    t = torch.bfloat16
    w = torch.ones(1, dim, dtype=t, device=DEV).expand(hidden, dim)
    x, none = torch.empty(0, dim, dtype=t, device=DEV), torch.empty(0, hidden, dtype=t, device=DEV)
    dw = [torch.full((hidden, dim), 3.0, dtype=t, device=DEV) for _ in range(2)]
    rar.gated_ff_backward(none, x, w, w, none, none.clone(), None, *dw, None, accumulate=True)
    assert all(bool((d[i] == 3.0).all()) for d in dw for i in (0, hidden // 2, hidden - 1))
    rar.gated_ff_backward(none, x, w, w, none, none.clone(), None, *dw, None)
    for d in dw:
        for part in d.view(torch.int16).split(1 << 16):
            assert not bool(part.any())
