"""The definition of per-head-decay linear attention in 64 bits, token by token
on the CPU, and the error bounds its tests use.

Bounds.  With the absolute values of all inputs in place of the inputs, every
sum of the recurrence has only positive terms; call those results the
magnitudes A.  A rounding of relative size u somewhere in a product or sum
moves a result by at most u times its magnitude, so
  bf16 results   (3 * 2^-8) A: the result's own rounding, the pair matrix's
                 (or the state's) as an operand, and room for everything in
                 fp32 (a thousand steps of 2^-24 are 2^-14);
  fp32 results   (T + 256) 2^-24 A: one step per token of a sum of T terms, and
                 the rounding of products, exponentials and chunk factors;
  d_log_decay    D_t, summed from r_t - c_t back from the segment's end over at
                 most 1024 tokens: the fp32 bound on D's magnitude plus that of
                 the r and c that were summed.
"""
from __future__ import annotations

import torch

D = 128


def bf16_bound(mag):
    return 3.0 * 2.0 ** -8 * mag


def f32_bound(mag, tokens):
    return (tokens + 256) * 2.0 ** -24 * mag


def _heads(x, h):
    return x.repeat_interleave(h // x.shape[1], 1)


def forward(q, k, v, log_decay, initial_state=None, lengths=None):
    """(o, final_state) in float64; q, k [T, Hq, 128], v [T, H, 128]."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    T, H = v.shape[0], v.shape[1]
    q, k = _heads(q, H), _heads(k, H)
    a = log_decay.detach().cpu().double().expand(T, H).exp()
    lengths = [T] if lengths is None else lengths
    o = torch.zeros(T, H, D, dtype=torch.float64)
    fin = torch.zeros(len(lengths), H, D, D, dtype=torch.float64)
    t = 0
    for n, L in enumerate(lengths):
        S = torch.zeros(H, D, D, dtype=torch.float64)
        if initial_state is not None:
            S = initial_state[n].detach().cpu().double().clone()
        for t in range(t, t + L):
            S = S * a[t][:, None, None] + k[t][:, :, None] * v[t][:, None, :]
            o[t] = torch.matmul(q[t][:, None, :], S)[:, 0]
        t = t + 1 if L else t
        fin[n] = S
    return o, fin


def backward(q, k, v, log_decay, d_o, initial_state=None, lengths=None, d_final_state=None):
    """The gradients in float64, and r and c per token (what d_log_decay is summed from):
    dict(dq, dk, dv, dg [T, H], ds0, rc [T, H])."""
    q, k, v, d_o = (x.detach().cpu().double() for x in (q, k, v, d_o))
    T, Hq, H = v.shape[0], q.shape[1], v.shape[1]
    qh, kh = _heads(q, H), _heads(k, H)
    a = log_decay.detach().cpu().double().expand(T, H).exp()
    lengths = [T] if lengths is None else lengths
    dq, dk, dv = (torch.zeros(T, H, D, dtype=torch.float64) for _ in range(3))
    dg, rc = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    ds0 = torch.zeros(len(lengths), H, D, D, dtype=torch.float64)
    b = 0
    for n, L in enumerate(lengths):
        S = torch.zeros(H, D, D, dtype=torch.float64)
        if initial_state is not None:
            S = initial_state[n].detach().cpu().double().clone()
        before = []
        for t in range(b, b + L):
            before.append(S * a[t][:, None, None])
            rc[t] = (qh[t] * torch.matmul(before[-1], d_o[t][:, :, None])[:, :, 0]).sum(-1)
            S = before[-1] + kh[t][:, :, None] * v[t][:, None, :]
            dq[t] = torch.matmul(S, d_o[t][:, :, None])[:, :, 0]
        M = torch.zeros(H, D, D, dtype=torch.float64)
        if d_final_state is not None:
            M = d_final_state[n].detach().cpu().double().clone()
        for t in range(b + L - 1, b - 1, -1):
            # (without the token's own term, which is far larger than the rest under a strong decay)
            rc[t] += (kh[t] * torch.matmul(M, v[t][:, :, None])[:, :, 0]).sum(-1)
            M = M + qh[t][:, :, None] * d_o[t][:, None, :]
            dk[t] = torch.matmul(M, v[t][:, :, None])[:, :, 0]
            dv[t] = torch.matmul(kh[t][:, None, :], M)[:, 0]
            dg[t] = (before[t - b] * M).sum((-1, -2))
            M = M * a[t][:, None, None]
        ds0[n] = M
        b += L
    share = lambda x: x.view(T, Hq, H // Hq, D).sum(2)  # noqa: E731
    return dict(dq=share(dq), dk=share(dk), dv=dv, dg=dg, ds0=ds0, rc=rc)


def suffix_within(rc, lengths, anchor):
    """Per token, the sum of rc from it to the end of its stretch of `anchor` tokens."""
    out = torch.zeros_like(rc)
    b = 0
    for L in lengths:
        for s in range(0, L, anchor):
            e = min(L, s + anchor)
            out[b + s:b + e] = rc[b + s:b + e].flip(0).cumsum(0).flip(0)
        b += L
    return out


def magnitudes(*tensors):
    return [None if x is None else x.detach().cpu().double().abs() for x in tensors]


def make(lengths, heads, qk_heads, dtype, decay, state, seed, device):
    """Seeded inputs: unit q and k, N(0, 1) v and gradients; decays by kind."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(shape, generator=g)

    def unit(x):
        return x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()

    if decay == "head":
        la = -torch.exp2(-8.0 * (torch.arange(heads) + 1) / heads)
    elif decay == "none":
        la = torch.zeros(T, heads)
    elif decay == "strong":
        la = -40.0 * torch.rand((T, heads), generator=g)
    else:
        la = -0.3 * torch.nn.functional.softplus(normal(T, heads))
        if decay == "reset":  # some tokens drop the state altogether
            la[torch.rand((T, heads), generator=g) < 0.05] = -float("inf")
            if T:
                la[T // 2] = -float("inf")
    d = dict(q=unit(normal(T, qk_heads, D)).to(t), k=unit(normal(T, qk_heads, D)).to(t),
             v=normal(T, heads, D).to(t), log_decay=la.float(), d_o=normal(T, heads, D).to(t),
             initial_state=0.3 * normal(N, heads, D, D) if state else None,
             d_final_state=0.3 * normal(N, heads, D, D) if state else None)
    cu = [0]
    for L in lengths:
        cu.append(cu[-1] + L)
    d["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32) if N > 1 else None
    return {n: x.to(device) if x is not None else None for n, x in d.items()}


def excess(got, want, bound):
    """Largest ratio of an error to its bound (0 where both are exact); inf for anything not finite."""
    got = got.detach().cpu().double()
    if not torch.isfinite(got).all():
        return float("inf")
    d = (got - want).abs()
    r = torch.where(d == 0, torch.zeros_like(d), d / bound.clamp(min=1e-300))
    return float(r.max()) if r.numel() else 0.0
