"""Beam selection and state reordering on the GPU against their definitions in
64 bits on the CPU.

Selection is compared exactly (tokens, parents, flags): the oracle's scores
are in fp64 and the tests' logits and scores are such that no two candidates
of different beams that matter are closer than 1e-5, or are exactly equal by
construction.  Scores: rounded to fp32 once (half a step, 2^-24 of the value),
and the sum of exponentials in fp32 (at most V terms a part, each off by two
roundings: 2^-20 is ample below V = 2^17; it enters the score absolutely).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


def kda():
    import gated_delta_rule_25_amd as m
    return m


def oracle(logits, scores, finished, end_token):
    x = logits.cpu().double()
    x = torch.where(x.isnan(), torch.full_like(x, -INF), x).clamp(max=torch.finfo(torch.float32).max)
    s = scores.cpu().double()
    B, K, V = x.shape
    m = x.amax(-1, keepdim=True)
    lse = torch.where(m > -INF, m + (x - m).exp().sum(-1, keepdim=True).log(), torch.zeros_like(m))
    c = torch.where(x > -INF, s[..., None] + (x - lse), torch.full_like(x, -INF))
    c = torch.where((s > -INF)[..., None], c, torch.full_like(c, -INF))
    if finished is not None:
        f = finished.cpu()
        only = torch.full_like(c, -INF)
        only[..., end_token] = s
        c = torch.where(f[..., None], only, c)
    best, at = c.view(B, K * V).sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    done = None if finished is None else f.gather(1, at // V) | (at % V == end_token)
    return best, at % V, at // V, done


def check(logits, scores, finished=None, end_token=None):
    s, t, p, f = kda().beam_select(logits, scores, finished, end_token=end_token)
    torch.cuda.synchronize()
    ws, wt, wp, wf = oracle(logits, scores, finished, end_token)
    assert t.dtype == torch.int32 and p.dtype == torch.int32
    assert torch.equal(p.cpu().long(), wp), (p, wp)
    assert torch.equal(t.cpu().long(), wt), (t, wt)
    assert (f is None) == (finished is None)
    if f is not None:
        assert torch.equal(f.cpu(), wf)
    s = s.cpu().double()
    low = ws == -INF
    assert torch.equal(s == -INF, low)
    err = (s - ws).abs()[~low]
    assert bool((err <= 2.0 ** -24 * ws[~low].abs() + 2.0 ** -20).all()), err.max()


def draw(B, K, V, dtype, seed, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    x = (scale * torch.randn(B, K, V, generator=g)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    s = (-20 * torch.rand(B, K, generator=g)).sort(-1, descending=True).values
    return x.cuda(), s.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (2, 3, 2), (1, 4, 3), (3, 2, 7), (2, 5, 17), (1, 16, 16), (4, 8, 1000),
                                   (2, 16, 4099), (1, 4, 32000), (2, 3, 65537), (1, 2, 131075)])
def test_select(dtype, B, K, V):
    x, s = draw(B, K, V, dtype, 100 + V + K)
    check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_rows_longer_than_the_parts_hold_in_one_vector(dtype):
    # more than 2048 vectors a row: several vectors a part
    x, s = draw(1, 3, 300001, dtype, 5)
    check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_finished(dtype):
    x, s = draw(6, 4, 999, dtype, 6)
    g = torch.Generator().manual_seed(7)
    f = (torch.rand(6, 4, generator=g) < 0.5).cuda()
    f[0] = True
    f[1] = False
    for end in (0, 2, 998):
        check(x, s, f, end)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_first_step(dtype):
    # one beam exists; its siblings have no score
    x, s = draw(3, 4, 501, dtype, 8)
    s[:, 1:] = -INF
    s[:, 0] = 0
    check(x, s)
    s[1] = -INF  # no beam at all
    check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_masked(dtype):
    x, s = draw(4, 3, 2050, dtype, 9)
    x[0, 0] = -INF                       # a row with nothing left
    x[1, :, 5:] = -INF                   # fewer tokens than candidates in some rows
    x[1, 1, :] = float("nan")
    x[2] = -INF                          # a group with nothing left
    x[3, 0, ::3] = float("nan")
    x[3, 1, 7] = INF
    x[3, 2] = torch.finfo(x.dtype).min   # a mask of the type's lowest value
    x[3, 2, 11] = 0
    check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_ties(dtype):
    # equal logits within a row, and equal rows with equal scores: the lowest index
    x, s = draw(3, 4, 3000, dtype, 10)
    x[0] = 0.5
    s[0] = -1.0
    x[1, :] = x[1, :1]
    s[1] = -2.0
    x[2, :, 100:2000:7] = 30.0
    check(x, s)
    x = torch.zeros(1, 3, 70000, dtype=x.dtype, device="cuda")
    x[0, :, 69999] = 1
    x[0, :, 0] = 1
    check(x, torch.zeros(1, 3, device="cuda"))


def test_select_descending_and_ascending_rows():
    # every later logit is better, and the reverse
    v = torch.arange(20000, dtype=torch.float32, device="cuda") * 1e-3
    x = torch.stack([v, v.flip(0)])[None].contiguous()
    check(x, torch.tensor([[0.0, -0.5]], device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_select_unaligned_logits(dtype, shift):
    x, s = draw(2, 3, 1003, dtype, 20 + shift)
    buf = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")
    y = buf[shift:].view(x.shape)
    y.copy_(x)
    check(y, s)


def test_select_in_place():
    x, s = draw(2, 4, 777, "f32", 30)
    f = torch.tensor([[True, False, False, False]] * 2, device="cuda")
    want = kda().beam_select(x, s, f, end_token=3)
    s2, f2 = s.clone(), f.clone()
    t, p = (torch.empty(2, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    got = kda().beam_select(x, s2, f2, end_token=3, out=(s2, t, p, f2))
    torch.cuda.synchronize()
    assert got[0] is s2 and got[3] is f2
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def states_of(n, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, 2, 16, 16, generator=g).cuda(),
            torch.randn(n, 3, 5, generator=g).to(torch.bfloat16).cuda(),   # 30-byte rows
            torch.randn(n, 7, generator=g).cuda(),                         # 28-byte rows
            torch.randint(0, 255, (n, 1), generator=g).to(torch.uint8).cuda()]


@pytest.mark.parametrize("B,K", [(1, 1), (1, 2), (3, 4), (5, 5), (2, 8), (2, 11), (1, 16)])
def test_reorder(B, K):
    g = torch.Generator().manual_seed(B * 100 + K)
    for parents in (torch.randint(0, K, (B, K), generator=g), torch.arange(K).flip(0).expand(B, K),
                    torch.arange(K).expand(B, K), torch.full((B, K), K - 1),
                    torch.arange(K).roll(1).expand(B, K)):
        p = parents.to(torch.int32).contiguous().cuda()
        st = states_of(B * K, 3)
        at = (torch.arange(B)[:, None] * K + parents).view(-1).cuda()
        want = [x[at].clone() for x in st]
        assert kda().beam_reorder(st, p) is st
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(st, want))


def test_reorder_parent_out_of_range_leaves_the_row():
    st = states_of(6, 4)
    p = torch.tensor([[0, -1, 0], [3, 1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, 0, 3, 4, 5], device="cuda")
    want = [x[at].clone() for x in st]
    kda().beam_reorder(st, p)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(st, want))


def test_reorder_more_tensors_than_one_call_takes():
    st = [torch.randn(4, 33, device="cuda") for _ in range(19)]
    p = torch.tensor([[1, 0], [1, 1]], dtype=torch.int32, device="cuda")
    want = [x[torch.tensor([1, 0, 3, 3], device="cuda")].clone() for x in st]
    kda().beam_reorder(st, p)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(st, want))


def test_reorder_offsets_past_32_bits():
    # 20 rows of 256 MiB: the last rows lie past 4 GiB
    n = 20
    x = torch.empty(n, 1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(n):
        x[i] = i
    p = torch.tensor([[9, 8, 7, 6, 5, 4, 3, 2, 1, 0]] * 2, dtype=torch.int32, device="cuda")
    kda().beam_reorder(x, p)
    torch.cuda.synchronize()
    for i in range(n):
        want = i // 10 * 10 + 9 - i % 10
        assert int(x[i].min()) == want and int(x[i].max()) == want


def test_reorder_leaves_what_lies_around_the_rows():
    buf = torch.arange(1000, dtype=torch.float32, device="cuda")
    x = buf[100:100 + 6 * 37].view(6, 37)
    before = buf.clone()
    p = torch.tensor([[2, 0, 0], [1, 1, 1]], dtype=torch.int32, device="cuda")
    kda().beam_reorder(x, p)
    torch.cuda.synchronize()
    assert torch.equal(buf[:100], before[:100]) and torch.equal(buf[322:], before[322:])
