"""In-place continuation of the gated delta rule where sequences are cut into
segments, whose workgroups run in any order: the final state in the initial one's
place gives the bits of a call with states of their own, by arithmetic (the same
products and sums), whatever else runs on the card."""
import math

import pytest
import torch

import gated_delta_rule_25_amd as kda
from delta_testlib import check_forward, cu_of, forward, make

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]


def both(args, s0, cu, seg):
    """(o, final_state) with a state of its own, and in place."""
    o, fin = kda.delta_chunk_fwd(*args, s0, cu, segment_tokens=seg)
    st = s0.clone()
    o2, fin2 = kda.delta_chunk_fwd(*args, st, cu, final_state=st, segment_tokens=seg)
    assert fin2 is st
    return o, fin, o2, fin2


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("lengths,h,hq,seg", [
    ([1024], 2, 2, 0),                               # cut by the library's own choice
    ([8192], 8, 8, 0),
    ([65], 1, 1, 64),                                # last segments of one token
    ([129, 1, 0, 65, 193, 64, 0], 3, 1, 64),         # and of one, none and whole ones beside them
    ([129, 1, 0, 65, 193, 64, 0], 66, 22, 64),       # the first segments walked ahead
])
def test_in_place_is_what_a_state_of_its_own_gives(lengths, h, hq, seg, dtype):
    q, k, v, la, b, s0 = make(sum(lengths), h, hq, dtype, 71, N=len(lengths), decay=0.05)
    cu = cu_of(lengths) if len(lengths) > 1 else None
    o, fin, o2, fin2 = both((q, k, v, la, b), s0, cu, seg)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)
    if sum(lengths) <= 1024 and h <= 3:
        check_forward(o2, fin2, forward(q, k, v, la, b, s0, lengths))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_in_place_beside_other_work(dtype):
    """Two calls at once and matrix products on a third stream hold the units, so that first segments begin late."""
    ins = [make(4096 + 1, 8, 8, dtype, 72 + i, decay=0.05) for i in range(2)]
    want = [kda.delta_chunk_fwd(*x[:5], x[5], segment_tokens=512) for x in ins]
    streams = [torch.cuda.Stream() for _ in range(3)]
    m = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for _ in range(3):
        states = [x[5].clone() for x in ins]
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[2]):
            for _ in range(4):
                torch.mm(m, m)
        got = []
        for x, st, s in zip(ins, states, streams):
            with torch.cuda.stream(s):
                got.append(kda.delta_chunk_fwd(*x[:5], st, final_state=st, segment_tokens=512))
        torch.cuda.synchronize()
        for (o, fin), (o2, fin2) in zip(want, got):
            assert torch.equal(o, o2) and torch.equal(fin, fin2)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("h", [2, 66])
def test_a_dropped_state_in_place(h, dtype):
    lengths = [200, 64, 65, 0]
    q, k, v, la, b, s0 = make(sum(lengths), h, h, dtype, 75, N=4, decay=0.05)
    la[[0, 200, 264]] = -math.inf
    bad = s0.clone()
    bad[:3] = math.nan
    bad[0, :, :64] = math.inf
    cu = cu_of(lengths)
    o, fin = kda.delta_chunk_fwd(q, k, v, la, b, torch.cat([torch.zeros_like(s0[:3]), s0[3:]]), cu, segment_tokens=64)
    o2, fin2 = kda.delta_chunk_fwd(q, k, v, la, b, bad, cu, final_state=bad, segment_tokens=64)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)


def test_in_place_in_a_graph():
    """Each replay goes on from the state that the last one left."""
    q, k, v, la, b, s0 = make(1024, 2, 2, torch.bfloat16, 76, decay=0.05)
    st, out = s0.clone(), torch.empty_like(v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kda.delta_chunk_fwd(q, k, v, la, b, st, out=out, final_state=st)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.delta_chunk_fwd(q, k, v, la, b, st, out=out, final_state=st)
    st.copy_(s0)
    want = s0
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        o, want = kda.delta_chunk_fwd(q, k, v, la, b, want)
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(st, want)
