"""Beam selection and state reordering on the GPU: calls at the border of what
the documentation allows."""
import pytest
import torch

import gated_delta_rule_25_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("last", ["parents", "overlap", "twice"])
def test_refused_reorder_of_many_states_moves_none(last):
    """More tensors than one call of the library takes, the last of them to be
    refused: the others are as they were, and the call can be made again."""
    buf = torch.randn(6, 40, device=DEV)
    p = torch.tensor([[1, 0, 0], [2, 2, 1]], dtype=torch.int32, device=DEV)
    states = [torch.randn(6, 33, device=DEV) for _ in range(8)] + [buf.view(-1)[:60].view(6, 10)]
    before = [x.clone() for x in states]
    bad = {"parents": p.view(6, 1), "overlap": buf.view(-1)[30:90].view(6, 10), "twice": states[0]}[last]
    with pytest.raises(ValueError):
        kda.beam_reorder([*states, bad], p)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(states, before))
    kda.beam_reorder(states, p)
    torch.cuda.synchronize()
    at = torch.tensor([1, 0, 0, 5, 5, 4], device=DEV)
    assert all(torch.equal(x, y[at]) for x, y in zip(states, before))
