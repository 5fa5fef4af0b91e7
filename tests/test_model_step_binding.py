"""The model steps' binding refuses tensors of another number of dimensions as it
refuses other shapes (no GPU)."""
import pytest
import torch

from context_merge_gb300 import cpdr


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("k,state", [((), (5, 2, 64, 64)), ((3, 2, 64), ()), ((3, 2, 64), (5,)), ((128,), (5, 2, 64, 64))])
def test_delta_step_dimensions(cpdr_lib, k, state):
    ctx = cpdr.Context(1, 64, 2, 64, 1, dtype="bf16", host_only=True)
    q = bf(3, 2, 64)
    with pytest.raises(ValueError, match="k must be"):
        ctx.delta_step(q, bf(*k), q, bf(3, 2), torch.zeros(3, 2), torch.zeros(state), q.clone())
