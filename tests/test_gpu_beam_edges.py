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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [1e6, 1e18, 3e38, float("inf")])
@pytest.mark.parametrize("n", [1, 2, 3])
def test_select_of_large_equal_logits(dtype, top, n):
    """n tokens at a large logit and nothing near it: each has 1 / n of the
    beam's probability (+inf counts as the largest finite number).  Scores are
    rounded once, and the sum of exponentials is off by at most 2^-20."""
    x = torch.zeros(1, 2, 300, dtype=dtype, device=DEV)
    at = [7, 100, 299][:n]
    x[0, :, at] = top
    s = torch.tensor([[-0.5, -1.5]], device=DEV)
    scores, tokens, parents, _ = kda.beam_select(x, s)
    torch.cuda.synchronize()
    log_n = torch.tensor(float(n), dtype=torch.float64).log()
    want = [(-0.5, 0, 7), (-1.5, 1, 7)] if n == 1 else [(-0.5, 0, 7), (-0.5, 0, 100)]
    for i, (score, beam, token) in enumerate(want):
        w = float(score - log_n)
        assert abs(float(scores[0, i]) - w) <= 2.0 ** -24 * abs(w) + 2.0 ** -20
        assert (int(parents[0, i]), int(tokens[0, i])) == (beam, token)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("beams", [1, 2])
def test_select_orders_logits_whose_scores_are_equal(dtype, beams):
    """Logits of 2^-60 and less beside one of 5: their scores are the same
    number in 64 bits, but within a beam the larger logit comes first."""
    K, V = 6, 40
    x = torch.exp2(torch.arange(V, dtype=torch.float64) - 100).to(dtype)
    x[3] = 5
    x = x.expand(1, K, V).contiguous().to(DEV)
    s = torch.full((1, K), -float("inf"), device=DEV)
    s[0, 1:1 + beams] = -2.0
    _, tokens, parents, _ = kda.beam_select(x, s)
    torch.cuda.synchronize()
    tokens, parents = tokens[0].tolist(), parents[0].tolist()
    n = K - beams
    assert tokens == [3] * beams + [V - 1 - i for i in range(n)]
    assert parents == [1 + i for i in range(beams)] + [1] * n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [2, 5, 16])
@pytest.mark.parametrize("V,gap", [(700, 1), (700, 64), (40000, 1), (40000, 8), (40000, 2048 * 8)])
def test_select_whose_best_share_parts_or_do_not(dtype, K, V, gap):
    """A row's best tokens next to one another (in one thread's part of the
    row), and `gap` tokens apart; the best of all in the last beam."""
    g = torch.Generator().manual_seed(V + K + gap)
    x = torch.randn(1, K, V, generator=g).clamp(max=3).to(dtype)
    at = (13 + gap * torch.arange(K + 2)) % V
    x[0, :, at] = (8 + 0.25 * torch.randperm(K + 2, generator=g)).to(dtype)
    s = torch.full((1, K), -60.0)
    s[0, K - 1] = -1.0
    _, tokens, parents, _ = kda.beam_select(x.to(DEV), s.to(DEV))
    torch.cuda.synchronize()
    want = x[0, K - 1].double().sort(descending=True, stable=True).indices[:K]
    assert tokens[0].tolist() == want.tolist() and parents[0].tolist() == [K - 1] * K
