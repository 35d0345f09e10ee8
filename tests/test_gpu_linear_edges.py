"""Per-head-decay linear attention on the GPU: calls at the border of what the
documentation allows, against the 64-bit definition of tests/linear_testlib.py."""
import pytest
import torch

import linear_testlib as lt
import gated_delta_rule_25_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = 1


@pytest.mark.parametrize("per_head", [0, 1])
@pytest.mark.parametrize("seg", [-1, 64])
def test_no_tokens_and_no_tensors_of_them(per_head, seg):
    """total_tokens 0 with NULL for everything that holds tokens: the states
    pass through, and the gradient of a constant decay is zero."""
    lib, n, h = kda._load(), 2, 3
    d = lt.make([0, 0], h, h, "bf16", "token", True, 21, DEV)
    fin, ds, dg = torch.empty_like(d["initial_state"]), torch.empty_like(d["initial_state"]), torch.ones(h, device=DEV)
    P, stream = kda._ptr, kda._stream(fin.device)
    need = int(lib.kda_linear_chunk_bwd_workspace_bytes(n, 0, h, h, per_head, 1, 1, 128, 128, BF16, seg))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    rc = lib.kda_linear_chunk_fwd(None, None, None, None, P(d["initial_state"]), P(d["cu_seqlens"]), n, 0, h, h,
                                  per_head, 128, 128, BF16, seg, None, P(fin), P(ws), need, stream)
    torch.cuda.synchronize()
    assert rc == kda.KDA_OK and torch.equal(fin, d["initial_state"])
    rc = lib.kda_linear_chunk_bwd(None, None, None, None, P(d["initial_state"]), P(d["cu_seqlens"]), None,
                                  P(d["d_final_state"]), n, 0, h, h, per_head, 128, 128, BF16, seg, None, None, None,
                                  P(dg), P(ds), P(ws), need, stream)
    torch.cuda.synchronize()
    assert rc == kda.KDA_OK and torch.equal(ds, d["d_final_state"])
    assert not per_head or torch.equal(dg, torch.zeros_like(dg))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("per_head", [False, True])
def test_decode_drops_a_state_that_holds_anything(dtype, what, per_head):
    """A decay of -inf: the new state is k v^T alone."""
    n, h = 3, 4
    d = lt.make([n], h, h, dtype, "token", False, 22, DEV)
    la = d["log_decay"][0].contiguous() if per_head else d["log_decay"]
    la[..., 1] = -float("inf")
    good = torch.randn(n, h, 128, 128, generator=torch.Generator().manual_seed(2)).to(DEV)
    bad = good.clone()
    bad[:, 1] = what
    good[:, 1] = 0
    o, want = (kda.linear_decode_step(S, d["q"], d["k"], d["v"], la) for S in (bad, good))
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(bad, good) and bool(torch.isfinite(bad).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 1, 40, 64, 129])
@pytest.mark.parametrize("seg", [-1, 64, 128])
def test_chunks_drop_a_state_that_holds_anything(dtype, what, at, seg):
    """Token `at` of each sequence has a decay of -inf: from there on nothing
    depends on the initial state, nor before it on the final state's gradient."""
    lengths, h = [200, 150], 2
    d = lt.make(lengths, h, h, dtype, "token", True, 23, DEV)
    behind = torch.zeros(sum(lengths), dtype=torch.bool, device=DEV)
    for b, L in ((0, 200), (200, 150)):
        d["log_decay"][b + at] = -float("inf")
        behind[b + at:b + L] = True
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    states = torch.full_like(d["initial_state"], what), torch.zeros_like(d["initial_state"])
    (o, fin), (wo, wfin) = (kda.linear_chunk_fwd(*args, s, d["cu_seqlens"], segment_tokens=seg) for s in states)
    torch.cuda.synchronize()
    assert torch.equal(o[behind], wo[behind]) and torch.equal(fin, wfin)
    got, want = (kda.linear_chunk_bwd(*args, d["d_o"], s, d["cu_seqlens"], d["d_final_state"], segment_tokens=seg)
                 for s in states)
    torch.cuda.synchronize()
    assert torch.equal(got[0][behind], want[0][behind])                  # dq reads the state
    assert all(torch.equal(got[i], want[i]) for i in (1, 2, 4))          # dk, dv and the state's do not
    got, want = (kda.linear_chunk_bwd(*args, d["d_o"], d["initial_state"], d["cu_seqlens"], s, segment_tokens=seg,
                                      need_d_log_decay=False) for s in states)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[4], want[4])
    assert all(torch.equal(got[i][~behind], want[i][~behind]) for i in (1, 2))
