"""Gradients of token log probabilities where the logits are large beside the log of
their sum: rows filled with the type's lowest value (as a finite mask leaves them),
infinities, and logits far from zero.

Bounds.  log p = (x - m) - log_s: x - m is exact or rounded once, 2^-24 of it, log_s
is off by the sum's terms (2^-22 each, added in fp64, and eight at a time in fp32:
2^-21) and its rounding, 2^-24 of at most 12; the exponential's argument by 2^-24 of
|d| (below 32 wherever p counts: e^-32 is 2^-46).  p: 2^-21 + 2 (32 + 12) 2^-24 <
2^-18 of itself; where |log_sum| is below the size from which rows are read twice, half
a step of it, 2^-15 in fp32 and 2^-13 in bf16, and what the forward call's sum is off
by, slack(n), besides.  Gradients with the entropy's: p's error times
|log p| + entropy + 1, and the entropy's own, slack(n) (2 + entropy).  Results: their
own rounding, half a step.  A p below fp32's smallest normal number may be zero, times
a gradient of a few and |log p| of 90: TINY.
"""
import math

import pytest
import torch

import gated_delta_rule_25_amd as kda
from test_gpu_logprob import definition, grad_definition, near, slack

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]
TINY = 2.0 ** -112


def rows_of(kind, dtype, n, rows=5):
    g = torch.Generator().manual_seed(n)
    x = 2.5 * torch.randn(rows, n, generator=g)
    if kind == "lowest":
        x = torch.full_like(x, torch.finfo(dtype).min)
    elif kind == "lowest but one":
        x = torch.full_like(x, torch.finfo(dtype).min)
        x[:, n // 2] = 1.5
    elif kind == "largest":
        x[:, ::3] = torch.finfo(dtype).max
    elif kind == "infinities":
        x[:, ::7] = math.inf
        x[:, 1::7] = -math.inf
        x[:, 2::7] = math.nan
    elif kind == "same":
        x = torch.full_like(x, -3.0e9)
    elif kind == "mixed":
        # rows on both sides of the sizes from which rows are read twice, and one masked throughout
        x += torch.tensor([0.0, 100.0, 150.0, -5000.0, 0.0])[:rows, None]
        x[4] = -math.inf
    else:
        x += kind
    t = torch.randint(0, n, (rows,), generator=g, dtype=torch.int32)
    t[rows - 2] = -1
    return x.to(dtype).cuda(), t.cuda()


KINDS = ["lowest", "lowest but one", "largest", "infinities", "same", "mixed", 127.0, 990.0, 1012.5, 1030.0, -3000.0, 4090.0, -4200.0, 1e5, -1e8]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [1, 9, 1000, 40003])
@pytest.mark.parametrize("kind", KINDS)
def test_gradient_of_far_rows(kind, n, dtype):
    x, t = rows_of(kind, dtype, n)
    r = kda.token_logprobs_fwd(x, t)
    w = definition(x, t)
    gen = torch.Generator().manual_seed(3)
    g, h = torch.randn(5, generator=gen).cuda(), torch.randn(5, generator=gen).cuda()
    size = 1024 if dtype == torch.float32 else 4096
    z = w["log_sum"].abs()
    p_rel = 2.0 ** -18 + slack(n) + torch.where(z < size * 1.001, z * 2.0 ** -24, torch.zeros_like(z))[..., None]
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    for hh in (None, h):
        got = kda.token_logprobs_bwd(x, t, r.log_sum, g, r.entropy if hh is not None else None, hh)
        want, _ = grad_definition(w, t, g, hh)
        p, ent = w["p"], w["entropy"][..., None]
        bound = g.double().abs()[..., None] * p * p_rel + TINY
        if hh is not None:
            logp = torch.where(p > 0, w["logp"].clamp(min=-1e4), torch.zeros_like(p)).abs()
            bound = bound + hh.double().abs()[..., None] * p * (p_rel * (logp + ent + 1) + slack(n) * (2 + ent))
        near(got, want, bound + half * want.abs(), "d_logits")
        inplace = x.clone()
        kda.token_logprobs_bwd(inplace, t, r.log_sum, g, r.entropy if hh is not None else None, hh, out=inplace)
        assert torch.equal(inplace, got)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_log_sum_of_more_than_the_row(dtype):
    """A log_sum that is not the row's alone (the caller's, over parts of a vocabulary) is taken as it is."""
    x, t = rows_of(8192.0, dtype, 1000)
    whole = torch.cat([x, x + 1], -1)
    z = kda.token_logprobs_fwd(whole).log_sum
    one = torch.ones(5, device="cuda")
    got = kda.token_logprobs_bwd(x, t, z, one)
    ok = (t >= 0).double()
    hot = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    hot.scatter_(-1, t.long().clamp(min=0)[:, None], ok[:, None])
    p = (x.double() - z.double()[:, None]).exp() * ok[:, None]
    want = hot - p
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    # (z is given: p's own 2^-18, and the difference of numbers of 8192 is exact)
    near(got, want, 2.0 ** -18 * p + half * want.abs() + TINY, "d_logits")


def test_far_rows_among_others_on_strides_and_repeated():
    wide = torch.zeros(700, 5011, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    wide.normal_(generator=g)
    wide[::3] -= 1.0e6
    wide[1::5] = torch.finfo(torch.float32).min
    x = wide[:, 3:5003]
    t = torch.randint(0, 5000, (700,), generator=g, dtype=torch.int32, device="cuda")
    r = kda.token_logprobs_fwd(x, t)
    one = torch.ones(700, device="cuda")
    want, _ = grad_definition(definition(x, t), t, one)
    bound = (2.0 ** -18 + slack(5000) + 2.0 ** -20) * definition(x, t)["p"] + 2.0 ** -24 * want.abs() + TINY
    # (a row's sum runs in an order that its alignment gives: the same bits on the same tensor only)
    for y in (x, x.contiguous()):
        got = kda.token_logprobs_bwd(y, t, r.log_sum, one)
        near(got, want, bound, "d_logits")
        for _ in range(3):
            assert torch.equal(got, kda.token_logprobs_bwd(y, t, r.log_sum, one))
    leaf = x.contiguous().requires_grad_()
    lp, _ = kda.token_logprobs(leaf, t)
    lp.sum().backward()
    near(leaf.grad, want, bound, "autograd")
