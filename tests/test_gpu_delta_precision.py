"""Accuracy of the gated delta rule where it is hardest: keys that are nearly the same
through a chunk, values far larger than the others of their chunk, and a state that the
chunk's decays all but remove.

Bounds.  Operands of a chunk are scaled by columns, by the largest m of what enters the
chunk and of its beta v, later tokens included; what is off by their smallest step is at
most 2^-19 m |q| of an output (delta_testlib), whatever the output's own size, and
2^-18 m |q| with the products' and sums' parts, which are 2^-19 of values below m.  The
state that the chunk leaves is off by as much, so the next chunk's outputs are by twice
that; later on it decays as the state does.

Keys that are the same: with beta near 1 every u_j replaces what the ones before left,
u_j = v_j - v_{j-1}, of sqrt(2) |v| where what remains is v.  bf16 dq and dk take u (and
y) rounded to fp16: 2^-11 of it at most, 2^-11.8 in the root mean square, and half of a
chunk's 64 on average: sqrt(32) sqrt(2) 2^-11.8 = 2^-8.8 of the result in norm, besides
their own rounding, 2^-9.2 in the root mean square: sqrt(2^-17.6 + 2^-18.4) < 3e-3.
"""
import math

import pytest
import torch

import gated_delta_rule_25_amd as kda
from delta_testlib import D, backward, check_backward, check_forward, forward, make, relative

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]


def grads_of(T, H, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, D, generator=g).to(dtype).cuda(), (0.3 * torch.randn(1, H, D, D, generator=g)).cuda()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("weight", [0.95, 0.999, 1.0])
@pytest.mark.parametrize("decay", [0.002, 0.02])
def test_keys_with_a_common_direction(weight, decay, dtype):
    T, H = 512, 2
    q, k, v, la, b, s0 = make(T, H, H, dtype, 61, beta=0.9)
    g = torch.Generator().manual_seed(62)
    common = torch.randn(1, H, D, generator=g)
    common = common / common.norm(dim=-1, keepdim=True)
    k = weight * common + math.sqrt(1 - weight * weight) * k.cpu().float()
    k = (0.999 * k / k.norm(dim=-1, keepdim=True)).to(dtype).cuda()
    la.fill_(-decay)
    d_o, d_fin = grads_of(T, H, dtype, 63)
    o, fin = kda.delta_chunk_fwd(q, k, v, la, b, s0)
    check_forward(o, fin, forward(q, k, v, la, b, s0))
    got = kda.delta_chunk_bwd(q, k, v, la, b, d_o, s0, None, d_fin)
    ref = backward(q, k, v, la, b, d_o, s0, None, d_fin)
    check_backward(got, ref, dtype)
    if dtype == torch.bfloat16:
        for name, x in zip(("dq", "dk"), got):
            assert relative(x, ref[name]) <= 3e-3, name


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("scale", [10, 20])
@pytest.mark.parametrize("at", [63, 40, 64])
def test_a_value_far_above_its_chunks_others(at, scale, dtype):
    T = 150
    q, k, v, la, b, s0 = make(T, 1, 1, dtype, 64, decay=0.05)
    s0.mul_(0.1)
    v[at] *= 2.0 ** scale
    ref = forward(q, k, v, la, b, s0)
    o, fin = kda.delta_chunk_fwd(q, k, v, la, b, s0)
    check_forward(o, fin, ref)
    # the rows before it, against the largest of their columns
    m = (b[at, 0] * v[at, 0].float()).abs().cpu().double()
    lim = q[:at, 0].float().norm(dim=-1).cpu().double()[:, None] * 2.0 ** -18 * m.clamp(min=16.0)
    err = (o[:at, 0].cpu().double() - ref[0][:at, 0]).abs()
    if dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * ref[0][:at, 0].abs()
    assert bool((err <= lim).all())
    # chunks before that one's do not know of it
    if at == 64:
        w = v.clone()
        w[64:] = 0
        assert torch.equal(kda.delta_chunk_fwd(q, k, w, la, b, s0)[0][:64], o[:64])
    d_o, d_fin = grads_of(T, 1, dtype, 65)
    d_o[at] *= 2.0 ** (scale / 2)
    got = kda.delta_chunk_bwd(q, k, v, la, b, d_o, s0, None, d_fin)
    check_backward(got, backward(q, k, v, la, b, d_o, s0, None, d_fin), dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("log_decay", [-14.0, -60.0, -math.inf])
def test_a_state_that_a_decay_within_the_chunk_removes(log_decay, dtype):
    T, at = 100, 20
    q, k, v, la, b, s0 = make(T, 1, 1, dtype, 66, decay=0.01)
    s0.mul_(2.0 ** 10)
    la[at] = log_decay
    ref = forward(q, k, v, la, b, s0)
    o, fin = kda.delta_chunk_fwd(q, k, v, la, b, s0)
    check_forward(o, fin, ref)
    m = s0[0, 0].abs().amax(0).cpu().double()
    lim = q[at:, 0].float().norm(dim=-1).cpu().double()[:, None] * 2.0 ** -18 * m
    err = (o[at:, 0].cpu().double() - ref[0][at:, 0]).abs()
    if dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * ref[0][at:, 0].abs()
    assert bool((err <= lim).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("scale", [10, 14])
def test_what_a_removed_state_leaves_to_later_chunks(scale, dtype):
    T, at = 200, 20
    q, k, v, la, b, s0 = make(T, 1, 1, dtype, 67, decay=0.01)
    s0.mul_(2.0 ** scale)
    la[at] = -math.inf
    o, fin = kda.delta_chunk_fwd(q, k, v, la, b, s0)
    ref, ref_fin, _ = forward(q, k, v, la, b, s0)
    m = s0[0, 0].abs().amax(0).cpu().double()
    lim = q[:, 0].float().norm(dim=-1).cpu().double()[:, None] * 2.0 ** -17 * m
    err = (o[:, 0].cpu().double() - ref[:, 0]).abs()
    if dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * ref[:, 0].abs()
    assert bool((err[at:] <= lim[at:]).all())
    # (a column of the state: through a query of unit length)
    assert bool(((fin.cpu().double() - ref_fin)[0, 0].norm(dim=0) <= 2.0 ** -17 * m).all())
    # a sequence of its own from there on is off by nothing of it
    cu = torch.tensor([0, at, T], dtype=torch.int32, device="cuda")
    two = torch.cat([s0, torch.zeros_like(s0)])
    o2, fin2 = kda.delta_chunk_fwd(q, k, v, la, b, two, cu)
    check_forward(o2, fin2, forward(q, k, v, la, b, two, [at, T - at]))
