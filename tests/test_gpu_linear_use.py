"""Per-head-decay linear attention and beam search as a program uses them:
captured and replayed, on other streams and side by side, through autograd,
with padding, with many and skewed sequences, and all of it together.

Tolerances are those of tests/linear_testlib.py and tests/test_gpu_beam.py;
what runs the same kernels twice is compared bit for bit.
"""
import gc

import pytest
import torch

import kda_inputs
import linear_testlib as lt
import gated_delta_rule_25_amd as kda
from test_gpu_beam import oracle as beam_oracle
from test_gpu_linear import check_backward, check_forward

pytestmark = pytest.mark.gpu
DEV = "cuda"
REPLAYS = 3


def capture(fn):
    """Warm up fn on a side stream, then capture it."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    torch.cuda.synchronize()
    return g, out


def fwd(d, **kw):
    return kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["initial_state"], d["cu_seqlens"], **kw)


def bwd(d, **kw):
    return kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["initial_state"], d["cu_seqlens"],
                                d["d_final_state"], **kw)


# ---- more shapes ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_random_shapes(dtype):
    g = torch.Generator().manual_seed(40)

    def pick(n):
        return int(torch.randint(n, (1,), generator=g))

    for i in range(6):
        hq = 1 + pick(3)
        h = hq * (1 + pick(3))
        lengths = [pick(260) for _ in range(1 + pick(5))]
        decay = ["token", "head", "none", "strong", "reset"][pick(5)]
        seg = [0, -1, 64, 192, 320][pick(5)]
        d = lt.make(lengths, h, hq, dtype, decay, bool(pick(2)), 50 + i, DEV)
        if sum(lengths) == 0:
            continue
        print(i, lengths, h, hq, decay, seg, flush=True)
        check_forward(d, lengths, dtype, segment_tokens=seg)
        check_backward(d, lengths, dtype, segment_tokens=seg)


@pytest.mark.parametrize("seg", [0, 64])
def test_more_sequences_than_are_ranked(seg):
    # (sequences are ordered by length up to 256 of them)
    lengths = [(3 * i) % 16 for i in range(300)]
    d = lt.make(lengths, 1, 1, "bf16", "token", True, 41, DEV)
    check_forward(d, lengths, "bf16", segment_tokens=seg)
    check_backward(d, lengths, "bf16", segment_tokens=seg)


def test_more_chains_than_compute_units():
    # whole heads in one walk, forward and backward
    lengths = [70, 3, 130, 64, 1]
    d = lt.make(lengths, 70, 70, "bf16", "token", True, 42, DEV)
    check_forward(d, lengths, "bf16")
    check_backward(d, lengths, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_sequence_of_many_heads(dtype):
    lengths = [150]
    d = lt.make(lengths, 48, 16, dtype, "head", True, 43, DEV)
    check_forward(d, lengths, dtype)
    check_backward(d, lengths, dtype)


@pytest.mark.parametrize("need_dg", [True, False])
@pytest.mark.parametrize("h", [90, 128])
def test_backward_whose_last_walks_take_half_heads(h, need_dg):
    # (on 256 compute units: 76 heads' dv whole and 14 by halves, none whole)
    lengths = [70]
    check_backward(lt.make(lengths, h, h // 2, "bf16", "token", True, 49, DEV), lengths, "bf16", need_dg=need_dg)


def test_segments_that_the_gradient_cuts_further():
    # 1088 tokens hold no stretch of 512 tokens or fewer but 64 x 17's own divisors
    lengths = [1500]
    d = lt.make(lengths, 1, 1, "bf16", "head", True, 44, DEV)
    check_backward(d, lengths, "bf16", segment_tokens=1088)
    check_backward(lt.make(lengths, 1, 1, "bf16", "token", True, 44, DEV), lengths, "bf16", segment_tokens=1088)


def test_more_work_items_than_one_launch_takes():
    """20000 sequences of one token x 96 heads: each is its own pair, so
    o = (q . k) v and dq = (v . d_o) k, dk = (v . d_o) q, dv = (q . k) d_o."""
    n, h = 20000, 96
    g = torch.Generator(device=DEV).manual_seed(51)
    q, k, v, d_o = (torch.randn(n, h, 128, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(4))
    la = torch.full((h,), -0.5, device=DEV)
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    o, _ = kda.linear_chunk_fwd(q, k, v, la, None, cu, output_final_state=False)
    dq, dk, dv, dg, _ = kda.linear_chunk_bwd(q, k, v, la, d_o, None, cu, need_d_initial_state=False)
    torch.cuda.synchronize()
    for at in (0, 1, n // 2, n - 70, n - 1):
        s = slice(at, at + 70)
        x = [t[s].cpu().double() for t in (q, k, v, d_o)]
        qk, vo = (x[0] * x[1]).sum(-1, keepdim=True), (x[2] * x[3]).sum(-1, keepdim=True)
        mqk, mvo = (x[0] * x[1]).abs().sum(-1, keepdim=True), (x[2] * x[3]).abs().sum(-1, keepdim=True)
        for got, want, mag in ((o, qk * x[2], mqk * x[2].abs()), (dq, vo * x[1], mvo * x[1].abs()),
                               (dk, vo * x[0], mvo * x[0].abs()), (dv, qk * x[3], mqk * x[3].abs())):
            assert lt.excess(got[s], want, lt.bf16_bound(mag)) <= 1, at
    assert torch.equal(dg, torch.zeros_like(dg))  # a token's own pair does not pass a decay


def test_no_tokens():
    d = lt.make([0, 0], 2, 1, "bf16", "head", True, 45, DEV)
    o, fin = fwd(d)
    dq, dk, dv, dg, ds = bwd(d)
    torch.cuda.synchronize()
    assert o.shape == (0, 2, 128) and torch.equal(fin, d["initial_state"])
    assert dq.shape == (0, 1, 128) and dv.shape == (0, 2, 128) and torch.equal(ds, d["d_final_state"])
    assert torch.equal(dg, torch.zeros(2, device=DEV))


@pytest.mark.parametrize("seg", [-1, 64])
@pytest.mark.parametrize("hq", [4, 2])
def test_backward_leaves_rows_behind_the_last_sequence(hq, seg):
    lengths, pad = [130, 20], 40
    d = lt.make(lengths, 4, hq, "bf16", "token", True, 46, DEV)
    want = bwd(d, segment_tokens=seg)
    dd = dict(d)
    for n in ("q", "k", "v", "log_decay", "d_o"):
        dd[n] = torch.cat([d[n], torch.full((pad,) + d[n].shape[1:], float("nan"), dtype=d[n].dtype, device=DEV)])
    # the outputs come from the allocator: give it blocks that hold a pattern
    T = 150 + pad
    outs = [torch.full_like(dd["q"], 7.0), torch.full_like(dd["q"], 7.0), torch.full_like(dd["v"], 7.0),
            torch.full((T, 4), 7.0, device=DEV), torch.empty_like(d["initial_state"])]
    lib = kda._load()
    need = int(lib.kda_linear_chunk_bwd_workspace_bytes(2, T, 4, hq, 0, 1, 1, 128, 128, 1, seg))
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device=DEV)  # NaN wherever it is read unwritten
    P = kda._ptr
    rc = lib.kda_linear_chunk_bwd(P(dd["q"]), P(dd["k"]), P(dd["v"]), P(dd["log_decay"]), P(d["initial_state"]),
                                  P(d["cu_seqlens"]), P(dd["d_o"]), P(d["d_final_state"]), 2, T, 4, hq, 0, 128, 128, 1,
                                  seg, *(P(t) for t in outs), P(ws), need, kda._stream(d["q"].device))
    torch.cuda.synchronize()
    assert rc == kda.KDA_OK
    for got, ref in zip(outs[:4], want[:4]):
        assert torch.equal(got[:150], ref)
        assert bool((got[150:] == 7.0).all())
    assert torch.equal(outs[4], want[4])


@pytest.mark.parametrize("cu", [[0, 500, 200], [0, -5, 200], [300, 100, 0], [0, 100, 10 ** 9], [-3, 400, 250]])
def test_bad_cu_seqlens_stay_in_bounds(cu):
    """Outside the preconditions the results are undefined, and nothing behind
    the tensors is written (offsets are clamped to the tokens there are)."""
    d = lt.make([100, 100], 2, 1, "bf16", "token", True, 47, DEV)
    d["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    room = torch.full((400, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    for seg in (-1, 64):
        fwd(d, out=room[100:300], segment_tokens=seg)
        bwd(d, segment_tokens=seg)
    torch.cuda.synchronize()
    assert bool((room[:100] == 7.0).all()) and bool((room[300:] == 7.0).all())


def test_debug_checks(monkeypatch):
    monkeypatch.setenv("KDA_DEBUG_CHECKS", "1")
    d = lt.make([70, 30], 2, 2, "bf16", "token", True, 48, DEV)
    fwd(d)
    bwd(d)
    assert kda.last_precondition_flags() == 0
    out = torch.full_like(d["v"], 7.0)
    good = d["log_decay"]

    def refused(bits, call):
        with pytest.raises(kda.KDAError) as e:
            call()
        torch.cuda.synchronize()
        assert e.value.code == kda.KDA_ERR_PRECONDITION and kda.last_precondition_flags() == bits
        assert bool((out == 7.0).all())

    for bad in (0.25, float("nan"), float("inf")):
        d["log_decay"] = good.clone()
        d["log_decay"][99, 1] = bad
        refused(kda.CHECK_LOG_ALPHA, lambda: fwd(d, out=out))
        refused(kda.CHECK_LOG_ALPHA, lambda: bwd(d))
        S = torch.zeros(100, 2, 128, 128, device=DEV)
        refused(kda.CHECK_LOG_ALPHA, lambda: kda.linear_decode_step(S, d["q"], d["k"], d["v"], d["log_decay"], out))
    d["log_decay"] = good
    d["cu_seqlens"] = torch.tensor([0, 80, 70], dtype=torch.int32, device=DEV)
    refused(kda.CHECK_CU_SEQLENS, lambda: fwd(d, out=out))


# ---- captured, replayed, on streams ------------------------------------------

@pytest.mark.parametrize("seg", [-1, 64])
def test_forward_and_backward_graph(seg):
    d = lt.make([300, 37, 0, 129], 4, 2, "bf16", "token", True, 60, DEV)
    g, (o, fin, grads) = capture(lambda: (*fwd(d, segment_tokens=seg), bwd(d, segment_tokens=seg)))
    for i in range(REPLAYS):
        for n in ("q", "k", "v", "d_o"):
            d[n].copy_(d[n].roll(1, 0))
        for t in (o, fin, *grads):
            t.zero_()
        g.replay()
        we, fe = fwd(d, segment_tokens=seg)
        ge = bwd(d, segment_tokens=seg)
        torch.cuda.synchronize()
        assert torch.equal(o, we) and torch.equal(fin, fe), i
        assert all(torch.equal(x, y) for x, y in zip(grads, ge)), i


def test_two_graphs_with_one_workspace():
    d1 = lt.make([300], 3, 3, "bf16", "token", True, 61, DEV)
    d2 = lt.make([200, 150], 3, 3, "bf16", "token", True, 62, DEV)
    need = max(kda.linear_chunk_bwd_workspace_bytes(1, 300, 3, segment_tokens=64),
               kda.linear_chunk_bwd_workspace_bytes(2, 350, 3, segment_tokens=64),
               kda.linear_chunk_fwd_workspace_bytes(2, 350, 3, segment_tokens=64))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    g1, r1 = capture(lambda: bwd(d1, workspace=ws, segment_tokens=64))
    g2, r2 = capture(lambda: (*fwd(d2, workspace=ws, segment_tokens=64), *bwd(d2, workspace=ws, segment_tokens=64)))
    w1, w2 = bwd(d1, segment_tokens=64), (*fwd(d2, segment_tokens=64), *bwd(d2, segment_tokens=64))
    for i in range(REPLAYS):
        for t in (*r1, *r2):
            t.zero_()
        ws.fill_(255)
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(r1, w1)), i
        assert all(torch.equal(x, y) for x, y in zip(r2, w2)), i


def test_side_by_side_on_streams():
    ds = [lt.make([400, 90], 3, 3, "bf16", "token", True, 63 + i, DEV) for i in range(3)]
    want = [(*fwd(d, segment_tokens=64), *bwd(d, segment_tokens=64)) for d in ds]
    logits = torch.randn(6, 4, 5000, device=DEV)
    scores = torch.zeros(6, 4, device=DEV)
    sel = kda.beam_select(logits, scores)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(3):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append((*fwd(d, segment_tokens=64), *bwd(d, segment_tokens=64)))
        with torch.cuda.stream(streams[3]):
            s2 = kda.beam_select(logits, scores)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert all(torch.equal(x, y) for x, y in zip(s2[:3], sel[:3]))


def test_decoding_graph():
    """A beam search step over linear states, captured: decode, select, reorder."""
    B, K, H, V = 3, 4, 2, 700
    d = lt.make([B * K], H, 1, "bf16", "token", False, 67, DEV)
    W = torch.randn(H * 128, V, device=DEV)
    first = torch.randn(B * K, H, 128, 128, generator=torch.Generator().manual_seed(1)).to(DEV)
    S = first.clone()
    scores = torch.zeros(B, K, device=DEV)
    done = torch.zeros(B, K, dtype=torch.bool, device=DEV)

    def step(S, scores, done):
        o = kda.linear_decode_step(S, d["q"], d["k"], d["v"], d["log_decay"])
        logits = (o.view(B, K, H * 128).float() @ W).contiguous()
        s, t, p, f = kda.beam_select(logits, scores, done, end_token=5)
        kda.beam_reorder(S, p)
        scores.copy_(s)
        done.copy_(f)
        return t, p

    g, (t, p) = capture(lambda: step(S, scores, done))
    S.copy_(first)
    scores.zero_()
    done.zero_()
    Se, se, de = first.clone(), scores.clone(), done.clone()
    for i in range(REPLAYS):
        g.replay()
        te, pe = step(Se, se, de)
        torch.cuda.synchronize()
        assert torch.equal(t, te) and torch.equal(p, pe), i
        assert torch.equal(S, Se) and torch.equal(scores, se) and torch.equal(done, de), i


# ---- autograd ------------------------------------------------------------------

def leaves(d):
    names = [n for n in ("q", "k", "v", "log_decay", "initial_state") if d[n] is not None]
    return names, [d[n].detach().clone().requires_grad_() for n in names]


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_autograd_is_the_backward_call(dtype, decay):
    d = lt.make([100, 33], 4, 2, dtype, decay, True, 70, DEV)
    names, x = leaves(d)
    o, fin = kda.chunk_linear(*x, d["cu_seqlens"])
    torch.autograd.backward([o, fin], [d["d_o"], d["d_final_state"]])
    want = bwd(d)
    for n, t, w in zip(names, x, want):
        assert torch.equal(t.grad, w), n


def test_autograd_partial_gradients():
    d = lt.make([80], 2, 2, "f32", "token", True, 71, DEV)
    q = d["q"].clone().requires_grad_()
    o, fin = kda.chunk_linear(q, d["k"], d["v"], d["log_decay"], d["initial_state"])
    (o * d["d_o"]).sum().backward()          # no gradient reaches the final state
    d["d_final_state"] = None
    assert torch.equal(q.grad, bwd(d, need_d_log_decay=False)[0])
    q.grad = None
    o, fin = kda.chunk_linear(q, d["k"], d["v"], d["log_decay"], d["initial_state"])
    fin.sum().backward()                     # nor here the outputs: they do not depend on q then
    assert torch.equal(q.grad, torch.zeros_like(q))
    o, fin = kda.chunk_linear(q, d["k"], d["v"], d["log_decay"], d["initial_state"])
    o.sum().backward()                       # a broadcast (stride 0) gradient
    d["d_o"] = torch.ones_like(d["d_o"])
    assert torch.equal(q.grad, bwd(d, need_d_log_decay=False)[0])
    with pytest.raises(RuntimeError, match="once_differentiable"):
        o, fin = kda.chunk_linear(q, d["k"], d["v"], d["log_decay"], d["initial_state"])
        (gq,) = torch.autograd.grad(o.square().sum(), q, create_graph=True)
        gq.sum().backward()


@pytest.mark.parametrize("decay", ["token", "head"])
def test_gradients_against_differences(decay):
    """Central differences of the loss in fp32 I/O along random directions.
    The loss is evaluated in fp64 from fp32 outputs whose rounding is at most
    f32_bound of their magnitudes; divided by the step it is the bound of the
    difference, beside the third-order term of the step (h^2 of the loss's
    scale; products of unit vectors and decays below 1: each factor below 4)."""
    lengths = [70, 9]
    d = lt.make(lengths, 4, 2, "f32", decay, True, 72, DEV)
    grads = dict(zip(("q", "k", "v", "log_decay", "initial_state"), bwd(d)))
    do, ds = d["d_o"].double(), d["d_final_state"].double()

    def loss(x):
        o, fin = fwd(x)
        return float((o.double() * do).sum() + (fin.double() * ds).sum())

    mq, mk, mv, ms = lt.magnitudes(d["q"], d["k"], d["v"], d["initial_state"])
    mo, mf = lt.forward(mq, mk, mv, d["log_decay"], ms, lengths)
    # rounding of the outputs: independent from one to the next, so their
    # weighted sum is off by the root of the squares (6 of them)
    T = max(lengths)
    noise = 6 * ((lt.f32_bound(mo, T) * do.cpu()).square().sum() + (lt.f32_bound(mf, T) * ds.cpu()).square().sum()).sqrt()
    h = 1e-2
    g = torch.Generator().manual_seed(3)
    for name, grad in grads.items():
        x = torch.randn(grad.shape, generator=g).to(DEV)
        x = x / x.norm()
        up, down = dict(d), dict(d)
        up[name], down[name] = d[name] + h * x, d[name] - h * x
        if name == "log_decay":
            up[name], down[name] = up[name].clamp(max=0), down[name].clamp(max=0)
            # (a clamped step is not the full one: take the direction that was)
            x = (up[name].double() - down[name].double()) / (2 * h)
        want = float((grad.double() * x.double()).sum())
        got = (loss(up) - loss(down)) / (2 * h)
        scale = float(grad.double().norm())
        print(name, want, got, noise / h, flush=True)
        assert abs(got - want) <= float(noise) / h + 64 * h * h * scale, (name, got, want)


def test_captured_backward_refuses_accumulators_from_elsewhere(monkeypatch):
    """A gradient accumulator lives as long as some graph of its leaf and
    belongs to the stream it was made on; a capture on another stream must not
    run it.  (Nothing is captured here: the call is told that it is.)"""
    d = lt.make([40], 1, 1, "bf16", "token", True, 74, DEV)
    names, x = leaves(d)
    alive, _ = kda.chunk_linear(*x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, _ = kda.chunk_linear(*x)
        loss = o.float().sum()
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
            with pytest.raises(RuntimeError, match="outside the graph capture"):
                loss.backward()
    torch.cuda.synchronize()
    assert all(t.grad is None for t in x)
    del alive, o, loss, _
    gc.collect()  # the refusal's traceback holds its frames, and they the graph
    with torch.cuda.stream(side):
        o, _ = kda.chunk_linear(*x)
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
            o.float().sum().backward()
    torch.cuda.synchronize()
    assert all(t.grad is not None for t in x[:4])


def test_training_step_graph():
    d = lt.make([130, 40], 2, 2, "bf16", "token", True, 73, DEV)
    names, x = leaves(d)

    def step():
        for t in x:
            t.grad = None
        o, fin = kda.chunk_linear(*x, d["cu_seqlens"])
        loss = (o.float() * d["d_o"].float()).sum() + (fin * d["d_final_state"]).sum()
        loss.backward()
        return [t.grad for t in x]

    g, grads = capture(step)
    want = bwd(d)
    for i in range(REPLAYS):
        for t in grads:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        torch.zeros(1000, device=DEV).add_(1).sum().item()  # eager work in between
        for n, t, w in zip(names, grads, want):
            assert torch.equal(t, w), (i, n)


# ---- together ------------------------------------------------------------------

def test_prompts_to_beams():
    """Prompts of different lengths through one linear and one KDA layer, then a
    beam search over both layers' states: prefill, beams from each prompt's
    state, and steps of decode, select and reorder, against the recurrence in
    64 bits following the same choices."""
    lengths, K, H, V, steps = [70, 3, 128], 3, 2, 50, 4
    B = len(lengths)
    d = lt.make(lengths, H, H, "f32", "token", False, 80, DEV)
    a = kda_inputs.make_prefill(H, lengths, "f32", 0.02, False, DEV, seed=81)
    _, S1 = fwd(d)
    _, S2 = kda.chunk_fwd(a["q"], a["k"], a["v"], a["log_alpha"], a["beta"], None, a["cu_seqlens"],
                          output_final_state=True)
    S1 = S1.repeat_interleave(K, 0).contiguous()
    S2 = S2.repeat_interleave(K, 0).contiguous()
    r1 = lt.forward(d["q"], d["k"], d["v"], d["log_decay"], None, lengths)[1].repeat_interleave(K, 0)
    e2 = S2.clone()   # the KDA layer's states: rows that its own decode advances and plain indexing reorders
    g = torch.Generator().manual_seed(82)
    W = torch.randn(H * 128, V, generator=g)
    scores = torch.full((B, K), -float("inf"), device=DEV)
    scores[:, 0] = 0.0
    done = torch.zeros(B, K, dtype=torch.bool, device=DEV)
    for i in range(steps):
        t = lt.make([B * K], H, H, "f32", "token", False, 83 + i, "cpu")
        x = {n: t[n].to(DEV) for n in ("q", "k", "v", "log_decay")}
        kd = kda_inputs.make_decode(B * K, H, 1, "f32", 0.02, DEV, seed=90 + i)
        o1 = kda.linear_decode_step(S1, x["q"], x["k"], x["v"], x["log_decay"])
        o2 = kda.decode_step(S2, *(kd[n][0] for n in ("q", "k", "v", "log_alpha", "beta")))
        e2o = kda.decode_step(e2, *(kd[n][0] for n in ("q", "k", "v", "log_alpha", "beta")))
        assert torch.equal(o2, e2o)
        logits = ((o1 + o2).view(B, K, H * 128).cpu() @ W).to(DEV)
        ws, wt, wp, wf = beam_oracle(logits, scores, done, 7)
        scores, tokens, parents, done = kda.beam_select(logits, scores, done, end_token=7)
        kda.beam_reorder([S1, S2], parents)
        torch.cuda.synchronize()
        assert torch.equal(tokens.cpu().long(), wt) and torch.equal(parents.cpu().long(), wp), i
        assert torch.equal(done.cpu(), wf), i
        # the recurrence in 64 bits, and the same choices
        rows = (torch.arange(B)[:, None] * K + wp).view(-1)
        r1 = r1 * t["log_decay"].double().exp()[:, :, None, None] + t["k"].double()[..., None] * t["v"].double()[:, :, None]
        r1 = r1[rows]
        e2 = e2[rows.to(DEV)].contiguous()
        assert torch.equal(S2, e2), i
    mag = lt.forward(*lt.magnitudes(d["q"], d["k"], d["v"]), d["log_decay"], None, lengths)[1].amax() + 4 * steps
    assert lt.excess(S1, r1, lt.f32_bound(mag.expand_as(r1), max(lengths))) <= 1
