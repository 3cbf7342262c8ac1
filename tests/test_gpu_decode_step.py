"""A decode step with drafts over a windowed cache, as a serving program runs it: qkv matmul -> rotate -> append -> windowed
attention -> o matmul -> lm_head -> verify, step after step, against the same step in PyTorch in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,window,sinks", [("q8_0", 40, 4), ("f16", 1000, 0), ("bf16", 17, 2)])
def test_steps_with_drafts(cache, window, sinks):
    t = torch_cuda()
    import synth
    from bit_weight_streaming_q4_gb300 import Qmm
    from bit_weight_streaming_q4_gb300.serve import KvPlan, VerifyPlan, rotate
    heads, kvh, dim, k, vocab, agents, drafts = 6, 2, 128, 512, 1500, 3, 2
    rows, page, pages = agents * (1 + drafts), 64, 4
    kind = torch.bfloat16 if cache == "bf16" else torch.float16

    def matrix(n, kk, tid):
        return Qmm(torch.from_numpy(synth.q4k_matrix(n, kk, seed=3, tensor_id=tid).reshape(-1)).cuda(), n, kk, m_max=128)
    qkv, o, head = matrix((heads + 2 * kvh) * dim, k, 1), matrix(k, heads * dim, 2), matrix(vocab, k, 3)
    g = torch.Generator().manual_seed(5)
    embed = torch.randn(vocab, k, generator=g).half().cuda()
    qw, kw = (1 + 0.2 * torch.randn(dim, generator=g)).cuda(), (1 + 0.2 * torch.randn(dim, generator=g)).cuda()
    inv = (1e4 ** (-torch.arange(dim // 2) / (dim // 2))).float().cuda()
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    table = torch.randperm(agents * pages, generator=g).to(torch.int32).view(agents, pages).cuda()
    plan = KvPlan(table, format=cache, heads=heads, kv_heads=kvh, head_dim=dim, page_tokens=page, pool_pages=agents * pages, max_rows=120,
                  max_agent_rows=40)
    judge = VerifyPlan(agents=agents, max_rows=rows, columns=vocab)
    pool = torch.zeros(agents * pages * kvh * 17408, dtype=torch.uint8, device="cuda") if cache == "q8_0" else \
        torch.zeros(agents * pages, kvh, 2, page, dim, dtype=kind, device="cuda")
    lens = [0] * agents
    history_k, history_v = [[] for _ in range(agents)], [[] for _ in range(agents)]  # what was appended, in 64 bits

    def forward(tokens, n):
        """Logits of n[a] next tokens of every sequence, and how far they may be off by the cache's rounding."""
        starts = np.concatenate([[0], np.cumsum(n)]).tolist()
        m = starts[-1]
        x = embed[torch.tensor(tokens, device="cuda")]
        y = torch.empty(m, (heads + 2 * kvh) * dim, device="cuda")
        qkv.run(x, y)
        q, kk, v = y.view(m, -1, dim).split((heads, kvh, kvh), 1)
        pos = i32([lens[a] + j for a in range(agents) for j in range(n[a])])
        q16, k32 = torch.empty(m, heads, dim, dtype=kind, device="cuda"), torch.empty(m, kvh, dim, device="cuda")
        rotate(q, kk, pos, inv, q16, k32, q_weight=qw, k_weight=kw)
        agent_rows = i32(starts)
        plan.append(pool, agent_rows, i32(lens), k32, v)
        out = torch.empty(m, heads, dim, dtype=torch.float16, device="cuda")
        row_len = [lens[a] + j + 1 for a in range(agents) for j in range(n[a])]
        plan.attend_window(pool, agent_rows, i32(row_len), q16, out, window=window, sinks=sinks)
        # the same in 64 bits from the matmul's output on
        yd = y.double().view(m, -1, dim)
        angle = pos.double()[:, None] * inv.double()

        def turned(z, w):
            z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-6) * w.double()
            a, b = z.chunk(2, -1)
            c, s = angle.cos()[:, None], angle.sin()[:, None]
            return torch.cat((a * c - b * s, a * s + b * c), -1)
        qd, kd, vd = turned(yd[:, :heads], qw), turned(yd[:, heads:heads + kvh], kw), yd[:, heads + kvh:]
        want = torch.empty(m, heads, dim, dtype=torch.float64, device="cuda")
        for a in range(agents):
            for j in range(n[a]):
                r = starts[a] + j
                history_k[a].append(kd[r])
                history_v[a].append(vd[r])
                ka, va = torch.stack(history_k[a]), torch.stack(history_v[a])
                slot = torch.arange(len(ka), device="cuda")
                see = (slot >= len(ka) - window) | (slot < sinks)
                for h in range(heads):
                    p = torch.softmax(ka[see, h // 3] @ qd[r, h] * dim ** -0.5, 0)
                    want[r, h] = p @ va[see, h // 3]
        # A query and a key are off by half a step each (q8_0: half a quant of its block's largest, 1 / 254), so a score by that
        # times sum |q k| / sqrt(dim) <= |q| |k| / sqrt(dim), about 1.2^2 sqrt(dim) here; a value by the same relative to its row's largest.
        step = {"q8_0": 2.0 ** -11 + 1 / 254, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}[cache]
        off = (out.double() - want).abs().max() / vd.abs().max()
        assert float(off) <= 2 * step * 1.5 * dim ** 0.5 + step, float(off)
        hidden = torch.empty(m, k, device="cuda")
        o.run(out.view(m, -1), hidden)
        logits = torch.empty(m, vocab, device="cuda")
        head.run((hidden * (4 / hidden.abs().max())).half(), logits)
        return logits, agent_rows

    tokens = torch.randint(0, vocab, (90,), generator=g).tolist()
    logits, _ = forward(tokens, [40, 30, 20])  # the prompts
    lens = [40, 30, 20]
    last = logits[[39, 69, 89]].argmax(-1).tolist()
    for step in range(4):
        # a sequence's last token and two drafts, drawn from distributions of the drafter's own
        fed, dl = [], torch.zeros(rows, vocab)
        for a in range(agents):
            fed += [last[a]]
            for j in range(drafts):
                dl[a * 3 + 1 + j] = torch.randn(vocab, generator=g) * 2
                fed.append(int(torch.multinomial(torch.softmax(dl[a * 3 + 1 + j], 0), 1, generator=g)))
        logits, agent_rows = forward(fed, [3] * agents)
        # (the target leans to the drafter, so that some drafts are taken)
        logits[:-1] += 4 * dl[1:].cuda() * (torch.arange(rows - 1) % 3 != 2).cuda()[:, None]
        au, su = torch.rand(rows, generator=g), torch.rand(agents, generator=g)
        acc, tok, prob = i32([9] * agents), i32([9] * agents), t.empty(rows, device="cuda")
        judge.verify(logits, agent_rows, i32(fed), au.cuda(), su.cuda(), acc, tok, draft_logits=dl.cuda(), prob=prob)
        assert plan.error() == 0 and judge.error() == 0
        p, qq = torch.softmax(logits.double().cpu(), -1), torch.softmax(dl.double(), -1)
        for a in range(agents):
            n = 0
            while n < drafts and float(au[3 * a + 1 + n]) * float(qq[3 * a + 1 + n, fed[3 * a + 1 + n]]) < float(p[3 * a + n, fed[3 * a + 1 + n]]):
                n += 1
            left = p[3 * a + n] if n == drafts else (p[3 * a + n] - qq[3 * a + n + 1]).clamp(min=0)
            run = left.cumsum(0)
            assert int(acc[a]) == n and int(tok[a]) == int((run <= float(su[a]) * float(run[-1])).sum())
            # what was refused leaves the cache: its slots are written again
            lens[a] += 1 + n
            del history_k[a][lens[a]:], history_v[a][lens[a]:]
            last[a] = int(tok[a])
    for m in (qkv, o, head):
        m.close()
