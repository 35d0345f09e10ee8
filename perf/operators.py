"""The operators around a linear-attention layer with one decay per head, and around beam search over
recurrent states: the cases they are measured on, their plain form in elementary torch operations, and
their definition in 64 bits.

`run` computes the plain form; with the module's `own` set to True it makes the calls a user makes of
the package's operators instead.

Operators (d = 128; a state S is [128, 128], rows = key channels, columns = value channels):

  forward   S_t = a_t S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,  a_t = exp(log_decay_t) <= 1, one scalar a head
  backward  the gradients of sum <d_o, o> + <d_final_state, S_T>
  decode    one token of the forward for many sequences, the state advanced in place
  select    the K best continuations of K beams over a vocabulary, ties to the lowest index
  reorder   the beams' recurrent states follow the selected parents, in place
"""
import math
import random

import torch

own = False

D = 128
CHUNK = 128  # tokens the plain form treats as one block


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the prompt of one layer at the library's headline shape, continued from a carried state
        dict(name="prefill H96 T8192", op="forward", dtype="bf16", heads=96, qk_heads=96, decay="token",
             seqs=1, longest=8192, lengths_seed=0, state=True),
        # one long context on few heads (a tensor-parallel shard): too few chains to fill the GPU in order
        dict(name="prefill H8 T131072", op="forward", dtype="bf16", heads=8, qk_heads=8, decay="token",
             seqs=1, longest=131072, lengths_seed=0, state=True),
        # a packed batch of ragged prompts, an empty one and a single token among them; query and key heads
        # shared by four value heads, one constant decay a head
        dict(name="prefill ragged 29 H32/8", op="forward", dtype="bf16", heads=32, qk_heads=8, decay="head",
             seqs=29, longest=4096, lengths_seed=5, state=False),
        # the smallest prompt, in fp32: latency
        dict(name="prefill fp32 H2 T256", op="forward", dtype="f32", heads=2, qk_heads=2, decay="token",
             seqs=1, longest=256, lengths_seed=0, state=False),
        # the backward pass of a training step of one layer
        dict(name="backward H96 T8192", op="backward", dtype="bf16", heads=96, qk_heads=96, decay="token",
             seqs=1, longest=8192, lengths_seed=0, state=True),
        # the backward pass over packed documents, shared query and key heads, a learned constant decay a head
        dict(name="backward ragged 9 H16/4", op="backward", dtype="bf16", heads=16, qk_heads=4, decay="head",
             seqs=9, longest=2900, lengths_seed=2, state=False),
        # one decoding step of a full serving batch
        dict(name="decode N256 H96", op="decode", dtype="bf16", seqs=256, heads=96, qk_heads=96, decay="token"),
        # one decoding step of a single sequence: latency
        dict(name="decode N1 H32", op="decode", dtype="bf16", seqs=1, heads=32, qk_heads=32, decay="head"),
        # beam selection of a serving batch over a large vocabulary, rows of odd length
        dict(name="select B64 K8 V128003", op="select", dtype="bf16", groups=64, beams=8, vocab=128003,
             finished=True),
        # beam selection for one prompt: latency
        dict(name="select B1 K4 V32000", op="select", dtype="f32", groups=1, beams=4, vocab=32000, finished=False),
        # the beams' states of one layer follow their parents: fp32 states and two bf16 convolution histories
        dict(name="reorder B64 K4 H96", op="reorder", groups=64, beams=4, heads=96, history=True),
        # the same for two prompts on a few heads: latency
        dict(name="reorder B2 K5 H3", op="reorder", groups=2, beams=5, heads=3, history=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "decode", "select", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("forward", "backward"):
        shared = rng.choice([1, 1, 2, 4])
        heads = shared * _spread(rng, 1, 96 // shared)
        seqs = rng.choice([1, rng.randint(2, 40)])
        budget = 96 * 8192 // (4 if dtype == "f32" else 1)  # tokens x heads
        longest = _spread(rng, 60, max(64, min(65536, budget // heads)))
        while seqs > 1 and sum(_lengths(seqs, longest, 7)) * heads > budget:
            seqs -= 1
        return dict(op=op, dtype=dtype, heads=heads, qk_heads=heads // shared,
                    decay=rng.choice(["token", "token", "head"]), seqs=seqs, longest=longest,
                    lengths_seed=7 if seqs > 1 else 0, state=rng.random() < 0.5)
    if op == "decode":
        shared = rng.choice([1, 1, 2, 4])
        heads = shared * _spread(rng, 1, 96 // shared)
        return dict(op=op, dtype=dtype, seqs=_spread(rng, 1, 256), heads=heads, qk_heads=heads // shared,
                    decay=rng.choice(["token", "head"]))
    if op == "select":
        return dict(op=op, dtype=dtype, groups=_spread(rng, 1, 48), beams=rng.randint(1, 8),
                    vocab=_spread(rng, 500, 131000), finished=rng.random() < 0.5)
    return dict(op=op, groups=_spread(rng, 1, 48), beams=rng.randint(2, 8), heads=_spread(rng, 1, 48),
                history=rng.random() < 0.5)


def _lengths(seqs, longest, seed):
    """Lengths of a packed batch: one sequence of `longest`, or log-uniform up to it, with an empty sequence
    and a single token among eight or more."""
    if seqs == 1:
        return [longest]
    r = random.Random(1000003 * seed + 8191 * seqs + longest)
    n = [_spread(r, 1, longest) for _ in range(seqs)]
    n[r.randrange(seqs)] = longest
    if seqs >= 8:
        i = r.randrange(seqs - 1)
        n[i], n[i + 1] = 0, 1
    return n


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()


def _decay(g, tokens, heads, kind):
    """Per token: -rate_h softplus(N(0, 1)), rates from 1 down to 2^-8 over the heads (memories of about one
    token to several hundred).  Per head: the constant slopes -2^(-8 (h + 1) / H)."""
    h = torch.arange(heads, device="cuda", dtype=torch.float32)
    if kind == "head":
        return -torch.exp2(-8.0 * (h + 1) / heads)
    rate = torch.exp2(-8.0 * h / max(1, heads - 1))
    x = _normal(g, tokens, heads)
    return -rate * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "select":
        B, K, V = case["groups"], case["beams"], case["vocab"]
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s = dict(op=op, logits=(2.5 * _normal(g, B, K, V)).to(t),
                 scores=-20.0 * torch.rand((B, K), generator=g, device="cuda"), finished=None, end_token=None)
        s["scores"] = s["scores"].sort(-1, descending=True).values
        if case["finished"]:
            s["finished"] = torch.rand((B, K), generator=g, device="cuda") < 0.2
            s["end_token"] = 2
        return s
    if op == "reorder":
        B, K, H = case["groups"], case["beams"], case["heads"]
        states = [_normal(g, B * K, H, D, D)]
        if case["history"]:
            states += [_normal(g, B * K, 3, H, D).to(torch.bfloat16) for _ in range(2)]
        # selected beams mostly descend from the better ones
        u = torch.rand((B, K), generator=g, device="cuda")
        return dict(op=op, states=states, parents=(K * u * u).to(torch.int32).clamp(max=K - 1))
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    H, Hq, N = case["heads"], case["qk_heads"], case["seqs"]
    if op == "decode":
        return dict(op=op, q=_unit(_normal(g, N, Hq, D)).to(t), k=_unit(_normal(g, N, Hq, D)).to(t),
                    v=_normal(g, N, H, D).to(t), log_decay=_decay(g, N, H, case["decay"]),
                    state=0.3 * _normal(g, N, H, D, D))
    lengths = _lengths(N, case["longest"], case["lengths_seed"])
    T = sum(lengths)
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    s = dict(op=op, q=_unit(_normal(g, T, Hq, D)).to(t), k=_unit(_normal(g, T, Hq, D)).to(t),
             v=_normal(g, T, H, D).to(t), log_decay=_decay(g, T, H, case["decay"]), initial_state=None,
             cu_seqlens=None if N == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    if case["state"]:
        s["initial_state"] = 0.3 * _normal(g, N, H, D, D)
    if op == "backward":
        s["d_o"] = _normal(g, T, H, D).to(t)
        s["d_final_state"] = 0.3 * _normal(g, N, H, D, D) if case["state"] else None
    return s


def work(case):
    op = case["op"]
    if op == "select":
        n = case["groups"] * case["beams"] * case["vocab"]
        return dict(bytes=n * (2 if case["dtype"] == "bf16" else 4) + 17 * case["groups"] * case["beams"], flops=4 * n)
    if op == "reorder":
        B, K, H = case["groups"], case["beams"], case["heads"]
        row = H * D * D * 4 + (2 * 3 * H * D * 2 if case["history"] else 0)
        # with p_j = sqrt((j + 1) / K) - sqrt(j / K): rows that change, and rows read for them
        p = [math.sqrt((j + 1) / K) - math.sqrt(j / K) for j in range(K)]
        moved = sum(1 - x for x in p)
        read = sum(1 - (1 - x) ** (K - 1) for x in p)
        return dict(bytes=B * (moved + read) * row + B * K * 4, flops=0)
    es = 2 if case["dtype"] == "bf16" else 4
    H, Hq, N = case["heads"], case["qk_heads"], case["seqs"]
    if op == "decode":
        return dict(bytes=2 * N * H * D * D * 4 + N * (2 * Hq + 2 * H) * D * es + (N * H if case["decay"] == "token" else H) * 4,
                    flops=4 * N * H * D * D)
    T = sum(_lengths(N, case["longest"], case["lengths_seed"]))
    state = N * H * D * D * 4
    decays = 4 * (T * H if case["decay"] == "token" else H)
    if op == "forward":
        return dict(bytes=T * (2 * Hq + 2 * H) * D * es + decays + state * (2 if case["state"] else 1),
                    flops=4 * T * H * D * D)
    return dict(bytes=T * (4 * Hq + 3 * H) * D * es + 2 * decays + (3 * state if case["state"] else 0),
                flops=10 * T * H * D * D)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "forward":
        return _plain_forward(s)
    if s["op"] == "backward":
        return _plain_backward(s)
    if s["op"] == "decode":
        return _plain_decode(s)
    if s["op"] == "select":
        return _plain_select(s)
    return _plain_reorder(s)


def _run_own(s):
    import gated_delta_rule_25_amd as kda
    if s["op"] == "forward":
        o, final = kda.linear_chunk_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["initial_state"], s["cu_seqlens"])
        return dict(o=o, final_state=final)
    if s["op"] == "backward":
        with_state = s["initial_state"] is not None
        dq, dk, dv, dg, ds = kda.linear_chunk_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["d_o"],
                                                  s["initial_state"], s["cu_seqlens"], s["d_final_state"],
                                                  need_d_initial_state=with_state)
        r = dict(dq=dq, dk=dk, dv=dv, d_log_decay=dg)
        if with_state:
            r["d_initial_state"] = ds
        return r
    if s["op"] == "decode":
        o = kda.linear_decode_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"])
        return dict(o=o, state=s["state"])
    if s["op"] == "select":
        scores, tokens, parents, finished = kda.beam_select(s["logits"], s["scores"], s["finished"],
                                                            end_token=s["end_token"])
        r = dict(scores=scores, tokens=tokens, parents=parents)
        if finished is not None:
            r["finished"] = finished
        return r
    kda.beam_reorder(s["states"], s["parents"])
    return dict(states=list(s["states"]))


def _blocks(s):
    """The packed sequences cut into blocks of CHUNK tokens, each sequence's last block padded: the tensors as
    [blocks, heads, CHUNK, ...] in 32 bits, the decays' sums in 64."""
    q, k, v, la, cu = s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"]
    T, H = v.shape[0], v.shape[1]
    dev = v.device
    if cu is None:
        cu = torch.tensor([0, T], device=dev)
    cu = cu.long()
    N = cu.numel() - 1
    count = (cu[1:] - cu[:-1] + CHUNK - 1) // CHUNK
    first = torch.cat([count.new_zeros(1), count.cumsum(0)])
    nb = T // CHUNK + N  # no fewer than the blocks in use
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=N - 1)
    at = t - cu[seq]
    place = (first[seq] + at // CHUNK) * CHUNK + at % CHUNK
    block_seq = torch.searchsorted(first[1:].contiguous(), torch.arange(nb, device=dev), right=True)  # N: not in use

    def lay(x):
        heads = x.shape[1]
        x = x.float()
        if heads != H:
            x = x.repeat_interleave(H // heads, dim=1)
        y = x.new_zeros((nb * CHUNK, H, D))
        y[place] = x
        return y.view(nb, CHUNK, H, D).transpose(1, 2).contiguous()

    la = la.double()
    if la.dim() == 1:
        la = la.expand(T, H)
    g = torch.zeros((nb * CHUNK, H), dtype=torch.float64, device=dev)
    g[place] = la
    G = g.view(nb, CHUNK, H).transpose(1, 2).cumsum(-1)  # within the block, inclusive
    low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=dev).tril()
    pair = (G[..., :, None] - G[..., None, :]).masked_fill_(~low, -math.inf).exp_().float()
    total = G[..., -1]  # [nb, H]
    A = total.cumsum(0)
    before = A - total
    # [H, nb, nb]: what of the state that block c' adds is left where block c of the same sequence begins
    follows = (block_seq[:, None] == block_seq[None, :]) & (block_seq < N)[:, None]
    follows = follows.tril(-1)
    left = (before.t()[:, :, None] - A.t()[:, None, :]).masked_fill_(~follows, -math.inf).exp_().float()
    of = block_seq.clamp(max=N - 1)
    begin = before[first[:-1].clamp(max=nb - 1)]  # [N, H]
    since = (before - begin[of]).masked_fill((block_seq >= N)[:, None], -math.inf).exp().float()  # from the start
    return dict(N=N, T=T, H=H, nb=nb, place=place, lay=lay, G=G, pair=pair, total=total, A=A, before=before, left=left,
                count=count, first=first, block_seq=block_seq, of=of, since=since,
                row=G.exp().float(), weight=(total[..., None] - G).exp().float(), q=lay(q), k=lay(k), v=lay(v))


def _unlay(b, x):
    return x.transpose(1, 2).reshape(b["nb"] * CHUNK, b["H"], D)[b["place"]]


def _states(b, initial):
    """The state that each block begins with, and what the block adds to it."""
    add = torch.matmul((b["k"] * b["weight"][..., None]).transpose(-1, -2).contiguous(), b["v"])
    flat = add.transpose(0, 1).reshape(b["H"], b["nb"], D * D)
    S = torch.matmul(b["left"], flat).view(b["H"], b["nb"], D, D).transpose(0, 1)
    if initial is not None:
        S = S + b["since"][..., None, None] * initial[b["of"]]
    return S.contiguous(), add


def _plain_forward(s):
    b = _blocks(s)
    S, add = _states(b, s["initial_state"])
    P = torch.matmul(b["q"], b["k"].transpose(-1, -2).contiguous()) * b["pair"]
    o = torch.matmul(P, b["v"]) + b["row"][..., None] * torch.matmul(b["q"], S)
    end = b["total"].exp().float()[..., None, None] * S + add
    last = (b["first"][1:] - 1).clamp(min=0)
    empty = s["initial_state"] if s["initial_state"] is not None else torch.zeros_like(end[:1])
    final = torch.where((b["count"] > 0)[:, None, None, None], end[last], empty)
    return dict(o=_unlay(b, o).to(s["v"].dtype), final_state=final)


def _plain_backward(s):
    b = _blocks(s)
    N, H, nb = b["N"], b["H"], b["nb"]
    S, add = _states(b, s["initial_state"])
    q, k, v, d_o = b["q"], b["k"], b["v"], b["lay"](s["d_o"])
    P = torch.matmul(q, k.transpose(-1, -2).contiguous()) * b["pair"]
    dP = torch.matmul(d_o, v.transpose(-1, -2).contiguous())
    F = P * dP
    dP = dP * b["pair"]
    row, weight = b["row"][..., None], b["weight"][..., None]
    # the gradient that reaches each block's end
    back = torch.matmul((q * row).transpose(-1, -2).contiguous(), d_o)
    flat = back.transpose(0, 1).reshape(H, nb, D * D)
    dS = torch.matmul(b["left"].transpose(-1, -2).contiguous(), flat).view(H, nb, D, D).transpose(0, 1)
    final = b["A"][(b["first"][1:] - 1).clamp(min=0)]  # [N, H]
    if s["d_final_state"] is not None:
        rest = (final[b["of"]] - b["A"]).masked_fill((b["block_seq"] >= N)[:, None], -math.inf).exp().float()
        dS = dS + rest[..., None, None] * s["d_final_state"][b["of"]]
    dS = dS.contiguous()
    from_state = row * torch.matmul(d_o, S.transpose(-1, -2).contiguous())
    to_state = weight * torch.matmul(v, dS.transpose(-1, -2).contiguous())
    dq = torch.matmul(dP, k) + from_state
    dk = torch.matmul(dP.transpose(-1, -2).contiguous(), q) + to_state
    dv = torch.matmul(P.transpose(-1, -2).contiguous(), d_o) + weight * torch.matmul(k, dS)
    # what crosses from token t - 1 to token t: the block's end, and the pairs on the way there
    F = F.tril(-1)
    r = F.sum(-1) + (from_state * q).sum(-1)
    c = F.sum(-2) + (to_state * k).sum(-1)
    end = b["total"].exp().float()[..., None, None] * S + add
    cross = (end * dS).sum((-1, -2)).double()[..., None] + (r - c).double().flip(-1).cumsum(-1).flip(-1)
    dg = cross.transpose(1, 2).reshape(nb * CHUNK, H)[b["place"]]
    if s["log_decay"].dim() == 1:
        dg = dg.sum(0)
    Hq, t = s["q"].shape[1], s["q"].dtype
    share = lambda x: _unlay(b, x).view(b["T"], Hq, H // Hq, D).sum(2).to(t)  # noqa: E731
    out = dict(dq=share(dq), dk=share(dk), dv=_unlay(b, dv).to(t), d_log_decay=dg.float())
    if s["initial_state"] is not None:
        seen = torch.zeros((N, H, D, D), dtype=torch.float32, device=v.device)
        seen.index_add_(0, b["of"], b["since"][..., None, None] * back)
        if s["d_final_state"] is not None:
            whole = (final - b["before"][b["first"][:-1].clamp(max=nb - 1)]).exp().float()
            whole = torch.where((b["count"] > 0)[:, None], whole, torch.ones_like(whole))
            seen = seen + whole[..., None, None] * s["d_final_state"]
        out["d_initial_state"] = seen
    return out


def _plain_decode(s):
    S, q, k, v = s["state"], s["q"].float(), s["k"].float(), s["v"].float()
    share = v.shape[1] // q.shape[1]
    if share > 1:
        q, k = q.repeat_interleave(share, dim=1), k.repeat_interleave(share, dim=1)
    a = s["log_decay"].exp()
    S.mul_(a[..., None, None])
    S.add_(k[..., :, None] * v[..., None, :])
    o = (S * q[..., :, None]).sum(-2)
    return dict(o=o.to(s["v"].dtype), state=S)


def _plain_select(s):
    # in 64 bits: candidates next to each other decide which one is taken
    x = s["logits"].double()
    B, K, V = x.shape
    x = x - x.amax(-1, keepdim=True)
    c = s["scores"].double()[..., None] + (x - x.exp().sum(-1, keepdim=True).log())
    if s["finished"] is not None:
        only = torch.full_like(c, -math.inf)
        only[..., s["end_token"]] = s["scores"].double()
        c = torch.where(s["finished"][..., None], only, c)
    best, at = c.view(B, K * V).sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    r = dict(scores=best.float(), tokens=(at % V).int(), parents=(at // V).int())
    if s["finished"] is not None:
        r["finished"] = s["finished"].gather(1, at // V) | (at % V == s["end_token"])
    return r


def _plain_reorder(s):
    B, K = s["parents"].shape
    at = (torch.arange(B, device="cuda")[:, None] * K + s["parents"]).view(-1)
    for x in s["states"]:
        x.copy_(x[at])
    return dict(states=list(s["states"]))


# ---------------------------------------------------------------------------
# the definition, token by token in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "forward":
        return _exact_forward(s)
    if s["op"] == "backward":
        return _exact_backward(s)
    if s["op"] == "decode":
        share = s["v"].shape[1] // s["q"].shape[1]
        each = [x.double().repeat_interleave(share, 1) for x in (s["q"], s["k"])]
        S = s["state"].double() * s["log_decay"].double().exp()[..., None, None]
        S = torch.addcmul(S, each[1].unsqueeze(-1), s["v"].double().unsqueeze(-2))
        return dict(o=torch.matmul(each[0].unsqueeze(-2), S).squeeze(-2), state=S)
    if s["op"] == "select":
        c = s["scores"].double().unsqueeze(-1) + torch.log_softmax(s["logits"].double(), -1)
        if s["finished"] is not None:
            done = s["finished"].unsqueeze(-1)
            token = torch.arange(c.shape[-1], device=c.device)
            c = c.masked_fill(done & (token != s["end_token"]), -math.inf)
            c = torch.where(done & (token == s["end_token"]), s["scores"].double().unsqueeze(-1), c)
        r = dict(scores=c.flatten(1).topk(c.shape[1]).values, tokens=None, parents=None)
        if s["finished"] is not None:
            r["finished"] = None
        return r
    K = s["parents"].shape[1]
    moved = []
    for x in s["states"]:
        y = x.double()
        z = y.view(-1, K, y[0].numel())
        w = torch.gather(z, 1, s["parents"].long().unsqueeze(-1).expand(-1, -1, z.shape[-1]))
        moved.append(w.view(x.shape))
    return dict(states=moved)


def _walk(s):
    """The sequences side by side: token t of every sequence, in 64 bits."""
    T, H = s["v"].shape[0], s["v"].shape[1]
    cu = [0, T] if s["cu_seqlens"] is None else s["cu_seqlens"].tolist()
    begin = torch.tensor(cu[:-1], device="cuda")
    length = torch.tensor([e - a for a, e in zip(cu, cu[1:])], device="cuda")
    share = H // s["q"].shape[1]
    x = {n: s[n].double() for n in ("q", "k", "v", "d_o") if n in s}
    x["q"], x["k"] = x["q"].repeat_interleave(share, 1), x["k"].repeat_interleave(share, 1)
    la = s["log_decay"].double()
    x["a"] = (la if la.dim() == 2 else la.expand(T, H)).exp()
    zero = torch.zeros((len(cu) - 1, H, D, D), dtype=torch.float64, device="cuda")
    return T, H, begin, length, max(e - a for a, e in zip(cu, cu[1:])), x, zero


def _tokens(x, names, begin, length, t, last):
    """Rows of token t of each sequence; past a sequence's end zeros, and a decay of one."""
    if begin.numel() == 1:
        return [x[n][t:t + 1] for n in names], None
    live = t < length
    at = (begin + t).clamp(max=last)
    got = []
    for n in names:
        y = x[n][at]
        on = live.view(-1, *[1] * (y.dim() - 1))
        got.append(torch.where(on, y, torch.ones_like(y) if n == "a" else torch.zeros_like(y)))
    return got, at[live]


def _exact_forward(s):
    T, H, begin, length, most, x, zero = _walk(s)
    S = zero if s["initial_state"] is None else s["initial_state"].double()
    o = torch.zeros((T, H, D), dtype=torch.float64, device="cuda")
    for t in range(most):
        (q, k, v, a), at = _tokens(x, "qkva", begin, length, t, T - 1)
        S = torch.addcmul(S * a[..., None, None], k[..., :, None], v[..., None, :])
        y = torch.matmul(q[..., None, :], S)[..., 0, :]
        if at is None:
            o[t] = y[0]
        else:
            o[at] = y[t < length]
    return dict(o=o, final_state=S)


def _exact_backward(s):
    T, H, begin, length, most, x, zero = _walk(s)
    S = zero if s["initial_state"] is None else s["initial_state"].double()
    M = zero.clone() if s["d_final_state"] is None else s["d_final_state"].double()
    dq, dk, dv = (torch.zeros((T, H, D), dtype=torch.float64, device="cuda") for _ in range(3))

    def put(y, at, value, t):
        if at is None:
            y[t] = value[0]
        else:
            y[at] = value[t < length]

    names = ["q", "k", "v", "a", "d_o"]
    for t in range(most):
        (q, k, v, a, d), at = _tokens(x, names, begin, length, t, T - 1)
        S = torch.addcmul(S * a[..., None, None], k[..., :, None], v[..., None, :])
        put(dq, at, torch.matmul(S, d[..., :, None])[..., 0], t)
    cross = (S * M).sum((-1, -2))  # [N, H]: what is left at each sequence's end
    for t in reversed(range(most)):
        (q, k, v, a, d), at = _tokens(x, names, begin, length, t, T - 1)
        M = torch.addcmul(M, q[..., :, None], d[..., None, :])
        put(dk, at, torch.matmul(M, v[..., :, None])[..., 0], t)
        put(dv, at, torch.matmul(k[..., None, :], M)[..., 0, :], t)
        M = M * a[..., None, None]
    # d/d log a_t = <S_{t-1} a_t, dS_t>, which changes from token to token by q_t . dq_t - k_t . dk_t
    change = (x["q"] * dq).sum(-1) - (x["k"] * dk).sum(-1)
    dg = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for n, (a, e) in enumerate(zip(begin.tolist(), (begin + length).tolist())):
        dg[a:e] = cross[n] + change[a:e].flip(0).cumsum(0).flip(0)
    Hq = s["q"].shape[1]
    r = dict(dq=dq.view(T, Hq, -1, D).sum(2), dk=dk.view(T, Hq, -1, D).sum(2), dv=dv,
             d_log_decay=dg if s["log_decay"].dim() == 2 else dg.sum(0))
    if s["initial_state"] is not None:
        r["d_initial_state"] = M
    return r
