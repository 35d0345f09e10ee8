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
