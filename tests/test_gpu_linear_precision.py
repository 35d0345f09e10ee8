"""fp32 results of per-head-decay linear attention are computed to fp32 accuracy,
also from bf16 inputs: norms of their errors against the 64-bit definition.

Bounds, derived before the first run.  u = 2^-24 is half a step of fp32, the
most that one rounding moves a value relatively.  Roundings are independent of
one another, so they add as squares, and each is taken at its largest:
  state      a token's term e^{..} k v^T: the hardware's 2^x (2 u), its product
             with v (u); the terms of a chunk are added into the accumulators in
             6 steps (bf16: 2 of 32 tokens in three terms each; fp32 16 per 64
             tokens), and the chunk's own factor is 2 more; per segment 4 for its
             factor, product and sum in the scan.  With n steps in all:
             sqrt(5 + n) u |S|.
  outputs    of fp32 I/O: the state's (or its transpose's), 32 steps of the sum
             over 128 channels, and for the pairs 32 for the products, 3 for
             their factor, 8 for the sum over the chunk, 2 for the row's factor:
             sqrt(5 + n + 77) u |o|.
  decays     r_t = q_t . dq_t and c_t = k_t . dk_t: with e = sqrt(5 + n + 77) u,
             the 128 channels of dq_t are off by e |dq_t| / sqrt(128) each, which
             makes e |q_t| |dq_t| / sqrt(128), and what they share (the row's
             factor) makes e |r_t|; c_t likewise.  They are summed from the
             stretch's end, as squares.  The boundary's <S, dS>: of the 128 x 128
             elements e |S| |dS| / 128, twice, and what a token's elements share
             (its factor) e times the r and c of all the sequence's tokens, as
             squares.  The sums themselves are in fp64; one rounding of the result.
A state kept or a factor formed to 16 bits is off by 2^-17 and more, 10 to 100
times these.
"""
import pytest
import torch

import linear_testlib as lt
import gated_delta_rule_25_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24

# lengths, heads, segment_tokens (0: as the library chooses, which cuts the last)
CASES = [([65], 2, -1), ([64], 2, 0), ([300], 2, -1), ([129, 0, 1, 63], 2, 0), ([500, 0, 64, 1, 130], 2, 64),
         ([500, 0, 64, 1, 130], 2, 192), ([2100], 1, -1), ([2100], 1, 0)]


def segment_of(lengths, h, seg, backward):
    """Tokens per segment, or None: the rule of segment_tokens = 0."""
    if seg > 0:
        return seg
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    T, n = sum(lengths), len(lengths)
    if seg < 0 or (5 if backward else 3) * n * h >= cus:
        return None
    s = max((-(-T * h // cus) + 255) // 256 * 256, 512)
    return s if n * s < T else None


def anchor_of(seg, per_head):
    a = 256 if per_head else 1024
    while seg and seg % a:
        a -= 64
    return a


def steps(T, dtype, seg):
    per_chunk = 8 if dtype == "bf16" else 18
    return per_chunk * -(-T // 64) + (4 * -(-T // seg) if seg else 0)


def per_sequence(x, lengths):
    b = 0
    for n in lengths:
        yield x[b:b + n]
        b += n


def check(r):
    print({k: "%.3g" % v for k, v in r.items()}, flush=True)
    assert max(r.values()) <= 1, r


def ratio(got, want, bound):
    """Norm of the error over its bound, per head the worst; got [.., H, ..] as want."""
    d = (got.detach().cpu().double() - want).norm()
    return 0.0 if float(d) == 0 else float(d / bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head", "none", "reset"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-h%d-seg%d" % ("+".join(map(str, c[0])), c[1], c[2]))
def test_forward_states(dtype, decay, case):
    lengths, h, seg = case
    d = lt.make(lengths, h, h, dtype, decay, True, 31, DEV)
    o, fin = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], d["cu_seqlens"],
                                  segment_tokens=seg)
    want, wfin = lt.forward(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], lengths)
    cut = segment_of(lengths, h, seg, False)
    r = {}
    for i, T in enumerate(lengths):
        n = steps(T, dtype, cut)
        for j in range(h):
            r["S%d.%d" % (i, j)] = ratio(fin[i, j], wfin[i, j], (5 + n) ** 0.5 * U * wfin[i, j].norm())
    if dtype == "f32":
        n = steps(max(lengths), dtype, cut)
        r["o"] = ratio(o, want, (5 + n + 77) ** 0.5 * U * want.norm())
    check(r)


def boundary_products(d, lengths, anchor):
    """(|S| |dS| / 128)^2 at the end of each token's stretch, [T, H]."""
    q, k, v, do = (d[n].cpu().double() for n in ("q", "k", "v", "d_o"))
    T, H = v.shape[0], v.shape[1]
    a = d["log_decay"].cpu().double().expand(T, H).exp()
    out = torch.zeros(T, H, dtype=torch.float64)
    b = 0
    for n, L in enumerate(lengths):
        ends = set(range(anchor, L, anchor)) | {L}
        S, s_at = d["initial_state"][n].cpu().double(), {}
        for t in range(L):
            S = S * a[b + t][:, None, None] + k[b + t][:, :, None] * v[b + t][:, None, :]
            if t + 1 in ends:
                s_at[t + 1] = S.flatten(1).norm(dim=-1)
        M = d["d_final_state"][n].cpu().double()
        for t in range(L, 0, -1):
            if t in ends:
                out[b + (t - 1) // anchor * anchor:b + t] = (s_at[t] * M.flatten(1).norm(dim=-1) / 128).square()
            M = (M + q[b + t - 1][:, :, None] * do[b + t - 1][:, None, :]) * a[b + t - 1][:, None, None]
        b += L
    return out


def gradient_ratios(d, got, lengths, dtype, cut):
    """Errors of linear_chunk_bwd's results over their bounds; d as lt.make gives it."""
    dq, dk, dv, dg, ds = got
    h, per_head = d["v"].shape[1], d["log_decay"].dim() == 1
    w = lt.backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["initial_state"], lengths, d["d_final_state"])
    anchor = anchor_of(cut, per_head)
    r = {}
    for i, T in enumerate(lengths):
        n = steps(T, dtype, cut)
        for j in range(h):
            r["dS%d.%d" % (i, j)] = ratio(ds[i, j], w["ds0"][i, j], (5 + n) ** 0.5 * U * w["ds0"][i, j].norm())
    n = steps(max(lengths), dtype, cut)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        if dtype == "f32":
            r[name] = ratio(x, w[name], (5 + n + 77) ** 0.5 * U * w[name].norm())
        else:  # three roundings to bf16: the result, the pair matrix, the state as an operand
            r[name] = ratio(x, w[name], 3 ** 0.5 * 2.0 ** -8 * w[name].norm())
    q, k = d["q"].cpu().double(), d["k"].cpu().double()
    own = (q * w["dq"]).sum(-1).square() + (k * w["dk"]).sum(-1).square()
    rc = own + ((q.norm(dim=-1) * w["dq"].norm(dim=-1)).square() + (k.norm(dim=-1) * w["dk"].norm(dim=-1)).square()) / 128
    at = 2 * boundary_products(d, lengths, anchor)
    b = 0
    for x in per_sequence(own, lengths):
        at[b:b + len(x)] += x.sum(0)
        b += len(x)
    bound = (5 + n + 77) * (lt.suffix_within(rc, lengths, anchor) + at) * U * U + (U * w["dg"]).square()
    if per_head:
        # the tokens' sums: those of a stretch share what is behind them, so they add up as they are
        total = 0.0
        for x in per_sequence(bound.sqrt(), lengths):
            for s in range(0, len(x), anchor):
                total = total + x[s:s + anchor].sum(0).square()
        want = w["dg"].sum(0)
        r["dg"] = ratio(dg, want, (total + (U * want).square()).sum().sqrt())
    else:
        r["dg"] = ratio(dg, w["dg"], bound.sum().sqrt())
    return r


def backward(d, seg):
    return kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["initial_state"], d["cu_seqlens"],
                                d["d_final_state"], segment_tokens=seg)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head", "none", "reset"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-h%d-seg%d" % ("+".join(map(str, c[0])), c[1], c[2]))
def test_backward_states_and_decays(dtype, decay, case):
    lengths, h, seg = case
    d = lt.make(lengths, h, h, dtype, decay, True, 32, DEV)
    check(gradient_ratios(d, backward(d, seg), lengths, dtype, segment_of(lengths, h, seg, True)))


# One sequence whose last dv walks take half heads, several ordered by length in
# whole and in half heads, whole heads in a walk each: as the library chooses.
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("lengths,h,heads", [([1100], 90, [0, 75, 76, 89]), ([3, 700, 1500, 0, 64], 70, [0, 69]),
                                             ([900, 5, 1030], 40, [0, 39]), ([1050, 1050], 128, [0, 127])])
def test_schedules_of_many_heads_over_several_stretches(lengths, h, heads, decay):
    """The heads are independent: some of them against the definition."""
    d = lt.make(lengths, h, h, "bf16", decay, True, 34, DEV)
    assert segment_of(lengths, h, 0, True) is None
    o, fin = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], d["cu_seqlens"])
    got = backward(d, 0)
    torch.cuda.synchronize()
    dim = {"log_decay": -1}
    one = {n: None if x is None else x if n == "cu_seqlens" else
           x.cpu().index_select(dim.get(n, 1), torch.tensor(heads)) for n, x in d.items()}
    part = [x[..., heads] if i == 3 else x[:, heads] for i, x in enumerate(got)]
    r = gradient_ratios(one, part, lengths, "bf16", None)
    want, wfin = lt.forward(one["q"], one["k"], one["v"], one["log_decay"], one["initial_state"], lengths)
    r["o"] = ratio(o[:, heads], want, 3 ** 0.5 * 2.0 ** -8 * want.norm())
    r["S"] = max(ratio(fin[i, h], wfin[i, j], (5 + steps(T, "bf16", None)) ** 0.5 * U * wfin[i, j].norm())
                 for i, T in enumerate(lengths) for j, h in enumerate(heads))
    check(r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,h,seg", [([200], 2, -1), ([300, 5, 70], 70, 0), ([500, 130], 2, 64), ([2100], 1, 0)])
def test_bits_do_not_depend_on_which_states_are_wanted(dtype, lengths, h, seg):
    """The outputs with and without the final state, and the gradients with
    and without the initial state's."""
    d = lt.make(lengths, h, h, dtype, "token", True, 33, DEV)
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    o, _ = kda.linear_chunk_fwd(*args, d["initial_state"], d["cu_seqlens"], segment_tokens=seg)
    o2, none = kda.linear_chunk_fwd(*args, d["initial_state"], d["cu_seqlens"], segment_tokens=seg,
                                    output_final_state=False)
    assert none is None and torch.equal(o, o2)
    a = kda.linear_chunk_bwd(*args, d["d_o"], d["initial_state"], d["cu_seqlens"], d["d_final_state"],
                             segment_tokens=seg)
    b = kda.linear_chunk_bwd(*args, d["d_o"], d["initial_state"], d["cu_seqlens"], d["d_final_state"],
                             segment_tokens=seg, need_d_initial_state=False)
    assert b[4] is None and all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))
