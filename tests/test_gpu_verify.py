"""Verification of drafted tokens (qmm_verify) against the definition in 64 bits (torch on the CPU).  What is taken
and drawn has to be equal; prob is fp32, rounded once (half a step, 2^-24) from numbers good to 2^-37."""
import math

import numpy as np
import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def softmax(x, t):
    """Probabilities of one row in 64 bits, or None without a distribution."""
    x = x.double()
    if bool(x.isnan().any()) or bool((x == math.inf).any()) or bool((x == -math.inf).all()):
        return None
    if t == 0:
        p = torch.zeros_like(x)
        p[int(torch.nonzero(x == x.max())[0])] = 1.0
        return p
    return torch.softmax((x - x.max()) / t, -1)


def verify_ref(logits, draft, agent_rows, tokens, temperature, accept_u, sample_u):
    """accepted, token, prob of every sequence; and how near a decision is to its border, relative (those nearer than
    2^-32 are not compared: 2^-37 for each of the two probabilities, and what thousands of roundings at 2^-45 add up to)."""
    agents, n = len(agent_rows) - 1, logits.shape[1]
    prob = torch.full((logits.shape[0],), 7.0, dtype=torch.float64)
    accepted, token, near = [], [], []
    for a in range(agents):
        r0, r1 = agent_rows[a], agent_rows[a + 1]
        t = float(temperature[a])
        t = 0.0 if not t >= 2.0 ** -100 else t
        if r1 <= r0:
            accepted.append(0)
            token.append(-1)
            near.append(1.0)
            continue
        prob[r0] = 0.0
        refused, left, edge = None, None, 1.0
        for r in range(r0 + 1, r1):
            p, x = softmax(logits[r - 1], t), int(tokens[r])
            inside = 0 <= x < n
            if t == 0 or draft is None:
                q = torch.zeros(n, dtype=torch.float64)
                if inside:
                    q[x] = 1.0
            else:
                q = softmax(draft[r], t)
            if p is None:
                prob[r] = 0.0 if bool((logits[r - 1] == -math.inf).all()) else math.nan
                if t == 0 and not bool((logits[r - 1] == -math.inf).all()):
                    prob[r] = math.nan
                yes = False
            elif q is None:
                prob[r], yes = math.nan, False
            elif not inside:
                prob[r], yes = 0.0, False
            else:
                pt, qt, u = float(p[x]), float(q[x]), float(accept_u[r])
                prob[r] = 1.0 if pt >= qt and pt > 0 else (pt / qt if qt > 0 else 0.0)
                yes = u * qt < pt
                if refused is None and t > 0 and pt > 0:
                    edge = min(edge, abs(u * qt - pt) / pt)
            if not yes and refused is None:
                refused = r
                left = p
                if p is not None and q is not None:
                    left = (p - q).clamp(min=0.0)
                    if t == 0 or float(left.sum()) == 0.0:
                        left = p
        row = r1 - 1 if refused is None else refused - 1
        if refused is None:
            left = softmax(logits[row], t)
        accepted.append(row - r0)
        if left is None:
            token.append(-1)
        else:
            run = left.cumsum(-1)
            u = float(sample_u[a])
            u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1.0)
            target = u * float(run[-1])
            i = int((run <= target).sum())
            if i >= n:
                i = int(torch.nonzero(left)[-1])
            token.append(i)
            if t > 0:
                edge = min(edge, float((run - target).abs().min()) / float(run[-1]) if 0 < u < 1 else 1.0)
        near.append(edge)
    return accepted, token, prob, near


def call(logits, draft, agent_rows, tokens, temperature, accept_u, sample_u, plan=None, stride=0, stream=None):
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    rows, n = logits.shape

    def dev(x):
        if x is None or not stride:
            return None if x is None else x.cuda()
        wide = t.zeros(rows, n + stride, dtype=x.dtype, device="cuda")
        wide[:, stride:] = x.cuda()
        return wide[:, stride:]
    agents = len(agent_rows) - 1
    plan = plan or serve.VerifyPlan(agents=agents, max_rows=max(1, rows), columns=n)
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    acc, tok, prob = i32([9] * agents), i32([9] * agents), t.full((rows,), 7.0, device="cuda")
    plan.verify(dev(logits), i32(agent_rows), tokens.to(torch.int32).cuda(), accept_u.float().cuda(), sample_u.float().cuda(), acc, tok,
                draft_logits=dev(draft), temperature=None if temperature is None else torch.tensor(temperature).float().cuda(), prob=prob)
    t.cuda.synchronize()
    return acc.tolist(), tok.tolist(), prob.double().cpu(), plan.error()


def compare(logits, draft, agent_rows, tokens, temperature, accept_u, sample_u, **kw):
    acc, tok, prob, err = call(logits, draft, agent_rows, tokens, temperature, accept_u, sample_u, **kw)
    temps = torch.tensor(temperature).float().tolist() if temperature is not None else [1.0] * (len(agent_rows) - 1)
    wa, wt, wp, near = verify_ref(logits, draft, agent_rows, tokens, temps, accept_u.float(), sample_u.float())
    assert err == 0
    compared = 0
    for a in range(len(near)):
        if near[a] > 2.0 ** -32:
            assert (acc[a], tok[a]) == (wa[a], wt[a]), (a, acc[a], tok[a], wa[a], wt[a])
            compared += 1
    assert compared >= 0.9 * len(near)
    assert torch.equal(prob.isnan(), wp.isnan())
    d = (prob - wp).abs()[~wp.isnan()]
    assert bool((d <= 2.0 ** -23.9 * wp[~wp.isnan()].abs() + 1e-30).all()), float(d.max())
    return acc, tok


def make(agents, per, n, kind="f32", seed=0, noise=0.8, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    per = [per] * agents if isinstance(per, int) else per
    rows = sum(per)
    ar = np.concatenate([[0], np.cumsum(per)]).tolist()
    x = (torch.randn(rows, n, generator=g) * spread).to(TYPES[kind])
    d = torch.zeros(rows, n)
    d[1:] = x[:-1].float() + noise * torch.randn(max(0, rows - 1), n, generator=g)
    d = d.to(TYPES[kind])
    gumbel = -torch.log(-torch.log(torch.rand(rows, n, generator=g).clamp(1e-20, 1 - 1e-7)))
    tokens = (d.float() + gumbel).argmax(-1)
    return x, d, ar, tokens, torch.rand(rows, generator=g), torch.rand(agents, generator=g)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 100, 1023, 8191, 8192, 8193, 32001, 70000])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_widths(n, kind):
    x, d, ar, tok, au, su = make(9, [1, 2, 3, 4, 5, 0, 3, 3, 9], n, kind, seed=n)
    compare(x, d, ar, tok, [0.7, 1.0, 0.0, 1.3, 1.0, 1.0, 2.0, 0.25, 1.0], au, su)
    compare(x, None, ar, tok, [0.7, 1.0, 0.0, 1.3, 1.0, 1.0, 2.0, 0.25, 1.0], au, su)


@pytest.mark.parametrize("stride", [1, 2, 3, 4])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_strides(stride, kind):
    x, d, ar, tok, au, su = make(5, 3, 9001, kind, seed=stride)
    compare(x, d, ar, tok, None, au, su, stride=stride)


def test_vocabulary():
    x, d, ar, tok, au, su = make(12, 4, 151936, seed=5)
    compare(x, d, ar, tok, [0.8] * 12, au, su)
    compare(x, None, ar, tok, [1.0] * 12, au, su)


def test_most_columns():
    x, d, ar, tok, au, su = make(1, 2, 1 << 19, seed=6)
    compare(x, d, ar, tok, None, au, su)
    # (the sums' largest: all columns alike)
    compare(torch.zeros_like(x), torch.zeros_like(x), ar, tok, None, au, su)


@pytest.mark.parametrize("seed", range(6))
def test_many_small(seed):
    """Hundreds of sequences over few columns: refusals everywhere, every branch."""
    x, d, ar, tok, au, su = make(300, 5, 37, seed=seed, noise=2.0, spread=3.0)
    t = [(0.5, 1.0, 0.0, 3.0, 100.0)[i % 5] for i in range(300)]
    acc, _ = compare(x, d, ar, tok, t, au, su)
    assert len(set(acc)) == 5
    compare(x, None, ar, tok, t, au, su)


def test_the_next_token_is_distributed_as_the_target():
    """Drafts and next token together, over a grid of both numbers: the first token's frequencies are p.  (Each
    cell of the 64 x 64 grid stands for 2^-12 of the square; its border cuts at most 64 + 64 cells per column.)"""
    torch.manual_seed(0)
    n, k = 7, 64
    p, q = torch.randn(n) * 1.5, torch.randn(n) * 1.5
    pp, qq = torch.softmax(p.double(), -1), torch.softmax(q.double(), -1)
    got = torch.zeros(n, dtype=torch.float64)
    u = (torch.arange(k).float() + 0.5) / k
    for x in range(n):
        rows = 2 * k * k
        logits, draft = p.repeat(rows, 1), q.repeat(rows, 1)
        tokens = torch.full((rows,), x)
        acc, tok, _, err = call(logits, draft, list(range(0, rows + 1, 2)), tokens, None, u.repeat_interleave(2 * k), u.repeat(k))
        assert err == 0
        for a, t in zip(acc, tok):
            got[x if a == 1 else t] += float(qq[x]) / (k * k)
    assert float((got - pp).abs().max()) < 2 / k


def test_infinities_and_numbers_that_are_none():
    x, d, ar, tok, au, su = make(8, 3, 500, seed=8)
    x[0, 7] = math.nan       # sequence 0: its first draft's row
    x[5, 3] = math.inf       # sequence 1: the last row
    x[6] = -math.inf         # sequence 2: nothing
    x[9:12, 100:] = -math.inf  # sequence 3: masked by a grammar
    d[13, 9] = math.nan      # sequence 4: a drafter without a distribution
    d[16] = -math.inf        # sequence 5
    tok[19] = -1             # sequence 6: drafts that are no columns
    tok[22] = 500            # sequence 7
    au[3:6] = 0.0            # (sequence 1's drafts are taken)
    for t in ([1.0] * 8, [0.0] * 8):
        compare(x, d, ar, tok, t, au, su)
        compare(x, None, ar, tok, t, au, su)


def test_ties_steep_and_flat():
    x, d, ar, tok, au, su = make(6, 3, 3001, seed=9)
    x = x.round()
    x[:, 17] = x[:, 2900] = x.max() + 1
    tok[1::3] = 17
    compare(x, d.round(), ar, tok, [0.0, 1e-3, 1e-30, 1e6, math.inf, 0.0], au, su)
    compare(x * 1e4, None, ar, tok, [1.0, 0.01, 50.0, 1e5, 1.0, math.nan], au, su)
    compare(torch.full_like(x, -3e38), None, ar, tok, [1.0] * 6, au, su)


def test_numbers_at_the_ends():
    x, d, ar, tok, au, su = make(6, 3, 777, seed=10)
    su = torch.tensor([0.0, 1.0, 2.0, -1.0, math.nan, 1 - 2.0 ** -24])
    for u in (0.0, 1 - 2.0 ** -24):
        compare(x, d, ar, tok, None, torch.full((18,), u), su)


def test_drafter_equal_to_the_target():
    x, _, ar, tok, au, su = make(20, 4, 4000, seed=11)
    d = torch.zeros_like(x)
    d[1:] = x[:-1]
    acc, _ = compare(x, d, ar, tok, [0.9] * 20, au, su)
    assert acc == [3] * 20


def test_bad_agent_rows():
    x, d, ar, tok, au, su = make(3, 3, 300, seed=12)
    acc, tk, prob, err = call(x, d, [0, 6, 3, 9], tok, None, au, su)
    assert err == 4 and acc == [0, 0, 0] and tk == [-1, -1, -1] and bool((prob == 7).all())
    acc, tk, prob, err = call(x, d, [0, 3, 6, 10], tok, None, au, su)
    good = call(x, d, ar, tok, None, au, su)
    assert err == 4 and acc[:2] == good[0][:2] and tk[:2] == good[1][:2] and tk[2] == -1 and bool((prob[6:] == 7).all())
    acc, tk, prob, err = call(x, d, [-1, 3, 6, 9], tok, None, au, su)
    assert err == 4 and tk[0] == -1 and tk[1:] == good[1][1:]
    # rows of no sequence stay as they are
    acc, tk, prob, err = call(x, d, [1, 3, 6, 8], tok, None, au, su)
    assert err == 0 and prob[0] == 7 and prob[8] == 7


def test_no_rows_graphs_and_streams():
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    acc, tk, _, err = call(torch.zeros(0, 50), None, [0, 0, 0], torch.zeros(0), None, torch.zeros(0), torch.zeros(2))
    assert err == 0 and acc == [0, 0] and tk == [-1, -1]
    x, d, ar, tok, au, su = make(4, 3, 20000, seed=13)
    want = call(x, d, ar, tok, None, au, su)
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    plan = serve.VerifyPlan(agents=4, max_rows=12, columns=20000)
    args = [x.cuda(), i32(ar), tok.to(torch.int32).cuda(), au.cuda(), su.cuda()]
    a, b, dd = i32([0] * 4), i32([0] * 4), d.cuda()
    t.cuda.synchronize()
    s = t.cuda.Stream()
    plan.verify(*args, a, b, draft_logits=dd, stream=s.cuda_stream)
    s.synchronize()
    assert (a.tolist(), b.tolist()) == want[:2]
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        plan.verify(*args, a, b, draft_logits=dd)
    other = make(4, 3, 20000, seed=14)
    want2 = call(other[0], other[1], ar, other[3], None, other[4], other[5])
    for new, w in (((x, d, ar, tok, au, su), want), (other, want2)):
        args[0].copy_(new[0])
        dd.copy_(new[1])
        args[2].copy_(new[3])
        args[3].copy_(new[4])
        args[4].copy_(new[5])
        a.fill_(9)
        g.replay()
        t.cuda.synchronize()
        assert (a.tolist(), b.tolist()) == w[:2]


def test_refusals():
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    x, d, ar, tok, au, su = make(2, 2, 64, seed=15)
    plan = serve.VerifyPlan(agents=2, max_rows=4, columns=64)
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    good = dict(logits=x.cuda(), agent_rows=i32(ar), tokens=i32(tok.tolist()), accept_u=au.cuda(), sample_u=su.cuda(), accepted=i32([0, 0]),
                token=i32([0, 0]), draft_logits=d.cuda(), temperature=su.cuda(), prob=au.cuda().clone())
    plan.verify(**good)
    bad = dict(logits=x.cuda()[:, :63], agent_rows=i32(ar[:2]), tokens=tok.cuda(), accept_u=au.cuda()[:3], sample_u=su, accepted=i32([0]),
               token=i32([0, 0, 0]), draft_logits=d.cuda().half(), temperature=su.cuda().double(), prob=au.cuda()[:2])
    for name, value in bad.items():
        with pytest.raises(ValueError):
            plan.verify(**{**good, name: value})
    with pytest.raises(ValueError):
        plan.verify(**{**good, "logits": x.cuda().repeat(2, 1)})
    t.cuda.synchronize()
