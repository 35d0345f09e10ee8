"""Per-head-decay linear attention on the GPU against its 64-bit definition
(tests/linear_testlib.py, where the bounds are derived)."""
import pytest
import torch

import linear_testlib as lt

pytestmark = pytest.mark.gpu

# lengths, heads, query/key heads
SHAPES = [
    ([1], 1, 1),
    ([31], 2, 1),
    ([64], 2, 2),
    ([65], 3, 3),
    ([129, 0, 1, 63], 4, 2),
    ([0, 0, 200], 2, 2),
    ([300], 4, 1),
]


def kda():
    import gated_delta_rule_25_amd as m
    return m


def check_forward(d, lengths, dtype, **kw):
    o, fin = kda().linear_chunk_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], d["cu_seqlens"], **kw)
    torch.cuda.synchronize()
    want, wfin = lt.forward(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], lengths)
    mq, mk, mv, ms = lt.magnitudes(d["q"], d["k"], d["v"], d["initial_state"])
    mag, mfin = lt.forward(mq, mk, mv, d["log_decay"], ms, lengths)
    T = max(lengths)
    e = lt.excess(o, want, lt.bf16_bound(mag) if dtype == "bf16" else lt.f32_bound(mag, T))
    f = lt.excess(fin, wfin, lt.f32_bound(mfin, T))
    assert o.dtype == d["v"].dtype and fin.dtype == torch.float32
    assert e <= 1 and f <= 1, (e, f)


def check_backward(d, lengths, dtype, need_dg=True, anchor=1024, **kw):
    with_state = d["initial_state"] is not None
    dq, dk, dv, dg, ds = kda().linear_chunk_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["initial_state"],
                                                d["cu_seqlens"], d["d_final_state"], need_d_log_decay=need_dg, **kw)
    torch.cuda.synchronize()
    want = lt.backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["initial_state"], lengths,
                       d["d_final_state"])
    mq, mk, mv, mo, ms, mf = lt.magnitudes(d["q"], d["k"], d["v"], d["d_o"], d["initial_state"], d["d_final_state"])
    mag = lt.backward(mq, mk, mv, d["log_decay"], mo, ms, lengths, mf)
    T = max(lengths)
    lossy = lt.bf16_bound if dtype == "bf16" else (lambda m: lt.f32_bound(m, T))
    r = {n: lt.excess(x, want[n], lossy(mag[n])) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))}
    r["ds0"] = lt.excess(ds, want["ds0"], lt.f32_bound(mag["ds0"], T))
    if need_dg:
        bound = lt.f32_bound(mag["dg"] + lt.suffix_within(mag["rc"], lengths, anchor), T)
        if d["log_decay"].dim() == 1:
            r["dg"] = lt.excess(dg, want["dg"].sum(0), bound.sum(0))
        else:
            r["dg"] = lt.excess(dg, want["dg"], bound)
    else:
        assert dg is None
    assert with_state or d["d_final_state"] is None
    assert max(r.values()) <= 1, r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head", "none", "strong", "reset"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%s-h%d/%d" % ("+".join(map(str, s[0])), s[1], s[2]))
def test_forward(dtype, decay, shape):
    lengths, h, hq = shape
    state = decay != "strong"
    check_forward(lt.make(lengths, h, hq, dtype, decay, state, 11, "cuda"), lengths, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", [-1, 64, 128, 192])
def test_forward_segmented(dtype, seg):
    lengths = [500, 0, 64, 1, 130]
    check_forward(lt.make(lengths, 2, 2, dtype, "token", True, 12, "cuda"), lengths, dtype, segment_tokens=seg)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head", "none", "strong", "reset"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%s-h%d/%d" % ("+".join(map(str, s[0])), s[1], s[2]))
def test_backward(dtype, decay, shape):
    lengths, h, hq = shape
    state = decay != "strong"
    check_backward(lt.make(lengths, h, hq, dtype, decay, state, 13, "cuda"), lengths, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("seg", [-1, 64, 128, 192])
def test_backward_segmented(dtype, decay, seg):
    lengths = [500, 0, 64, 1, 130]
    check_backward(lt.make(lengths, 2, 1, dtype, decay, True, 14, "cuda"), lengths, dtype, segment_tokens=seg)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_without_decay_gradient(dtype):
    lengths = [200, 70]
    check_backward(lt.make(lengths, 2, 2, dtype, "token", True, 15, "cuda"), lengths, dtype, need_dg=False)
    check_backward(lt.make(lengths, 2, 2, dtype, "token", True, 15, "cuda"), lengths, dtype, need_dg=False,
                   segment_tokens=64)


def test_long_backward_restarts_the_decay_gradient():
    # three stretches of 1024 tokens in one walk
    lengths = [2100]
    check_backward(lt.make(lengths, 1, 1, "bf16", "token", True, 16, "cuda"), lengths, "bf16", segment_tokens=-1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head", "none", "strong", "reset"])
@pytest.mark.parametrize("n,h,hq", [(1, 1, 1), (3, 4, 2), (70, 8, 8)])
def test_decode(dtype, decay, n, h, hq):
    if decay == "head":
        d = lt.make([n], h, hq, dtype, "head", False, 17, "cuda")
    else:
        d = lt.make([n], h, hq, dtype, decay, False, 17, "cuda")
    S0 = torch.randn(n, h, 128, 128, generator=torch.Generator().manual_seed(3)).cuda()
    S = S0.clone()
    o = kda().linear_decode_step(S, d["q"], d["k"], d["v"], d["log_decay"])
    torch.cuda.synchronize()
    per_head = d["log_decay"].dim() == 1
    for i in range(n):
        la = d["log_decay"] if per_head else d["log_decay"][i:i + 1]
        one = [d[x][i:i + 1] for x in ("q", "k", "v")]
        want, wfin = lt.forward(*one, la, S0[i:i + 1])
        m = lt.magnitudes(*one, S0[i:i + 1])
        mag, mfin = lt.forward(m[0], m[1], m[2], la, m[3])
        # one rounding of the output; the sum of 128 products and the exponential in fp32
        e = lt.excess(o[i:i + 1], want, (2.0 ** -8 * want.abs() + lt.f32_bound(mag, 128)) if dtype == "bf16"
                      else lt.f32_bound(mag, 128))
        f = lt.excess(S[i:i + 1], wfin, lt.f32_bound(mfin, 1))
        assert e <= 1 and f <= 1, (i, e, f)


def test_same_bits_every_time():
    lengths = [700, 0, 129]
    d = lt.make(lengths, 4, 2, "bf16", "head", True, 18, "cuda")
    for seg in (-1, 128):
        a = kda().linear_chunk_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], d["cu_seqlens"],
                                   segment_tokens=seg)
        b = kda().linear_chunk_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], d["cu_seqlens"],
                                   segment_tokens=seg)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        args = (d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["initial_state"], d["cu_seqlens"],
                d["d_final_state"])
        a, b = (kda().linear_chunk_bwd(*args, segment_tokens=seg) for _ in range(2))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("seg", [-1, 64])
def test_in_place_state_and_rows_behind_the_last_sequence(seg):
    lengths = [300, 5]
    d = lt.make(lengths, 3, 3, "bf16", "token", True, 19, "cuda")
    o, fin = kda().linear_chunk_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], d["cu_seqlens"],
                                    segment_tokens=seg)
    S = d["initial_state"].clone()
    # 40 rows of padding behind the last sequence: not read, and their outputs left as they were
    pad = {n: torch.cat([d[n], torch.full((40,) + d[n].shape[1:], float("nan"), dtype=d[n].dtype, device="cuda")])
           for n in ("q", "k", "v", "log_decay")}
    out = torch.full_like(pad["v"], 7.0)
    o2, S2 = kda().linear_chunk_fwd(pad["q"], pad["k"], pad["v"], pad["log_decay"], S, d["cu_seqlens"], out=out,
                                    final_state=S, segment_tokens=seg)
    torch.cuda.synchronize()
    assert S2 is S and torch.equal(S, fin)
    assert torch.equal(out[:305], o) and bool((out[305:] == 7.0).all())
