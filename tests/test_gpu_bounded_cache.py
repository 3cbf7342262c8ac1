"""The serving operators and the matmuls as one loop (examples/bounded_cache.py), at a small size."""
import importlib.util
import os
import sys

import pytest

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "bounded_cache.py")


@pytest.fixture(scope="module")
def example():
    torch_cuda()
    spec = importlib.util.spec_from_file_location("bounded_cache", PATH)
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod  # (its dataclasses look themselves up there)
    spec.loader.exec_module(mod)
    return mod


def shape(example):
    return example.Shape(layers=2, dim=512, heads=12, kv_heads=2, vocab=1500)


def prompts(torch, shape, lens, seed=3):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(shape.vocab, (n,), generator=g).tolist() for n in lens]


def row_by_row(server):
    """Norms that do not depend on how many rows a call has (a library reduction's order may)."""
    import torch
    norm = type(server)._norm
    server._norm = lambda x: torch.cat([norm(server, x[i:i + 1].clone()) for i in range(len(x))])
    return server


@pytest.mark.parametrize("cache", ["q8_0", "f16", "bf16"])
def test_sequences_do_not_depend_on_each_other(example, cache):
    """Three sequences together, with evictions, answer bit for bit what each answers beside idle ones."""
    torch = torch_cuda()
    s = shape(example)
    ps = prompts(torch, s, (150, 5, 70))

    def run(which):
        server = row_by_row(example.Server(s, 3, cache=cache, budget=60, slack=9, recent=16, piece=8))
        res = server.generate([p if a in which else [] for a, p in enumerate(ps)], 24)
        lens = list(server.lens)
        server.close()
        return res, lens

    together, lens = run({0, 1, 2})
    for a in range(3):
        alone, n = run({a})
        assert alone[a] == together[a] and n[a] == lens[a], a
        assert len(alone[a]["token"]) == 24 and len(alone[a]["prompt_logprob"]) == len(ps[a]) - 1


@pytest.mark.parametrize("cache", ["q8_0", "bf16"])
def test_budget_positions_and_weights(example, cache):
    torch = torch_cuda()
    s = shape(example)
    ps = prompts(torch, s, (150, 5, 70))
    server = example.Server(s, 3, cache=cache, budget=60, slack=9, recent=16, piece=8)
    server.generate(ps, 24)
    for a, p in enumerate(ps):
        assert server.seen[a] == len(p) + 23 and server.lens[a] <= 69 + 8
        assert server.lens[a] == (server.seen[a] if server.seen[a] <= 69 else server.lens[a])
        for layer in server.layers:
            for g in range(s.kv_heads):
                pos = layer.pos[a, g, :server.lens[a]].tolist()
                assert len(set(pos)) == len(pos) and 0 <= min(pos) and max(pos) < server.seen[a]
                # the first tokens, and those that the last cut protected and the ones since then
                assert {0, 1, 2, 3} <= set(pos) and set(range(server.seen[a] - min(16, server.seen[a]), server.seen[a])) <= set(pos)
                assert bool((layer.weight[a, g, :server.lens[a]] >= 0).all())
    server.close()


def test_weights_of_an_uncut_cache_add_up(example):
    """Each row gives its group's heads a weight of 1 each: heads / kv_heads per row and KV head.  A
    weight is good to some 2^-15 of itself (a 2^-11 relative rounding would show at 128 times the bound)."""
    torch = torch_cuda()
    s = shape(example)
    server = example.Server(s, 2, cache="f16", budget=200, piece=8)
    server.generate(prompts(torch, s, (90, 33)), 10)
    for layer in server.layers:
        for a in range(2):
            got = layer.weight[a, :, :server.lens[a]].double().sum(-1)
            want = s.heads // s.kv_heads * server.seen[a]
            assert server.lens[a] == server.seen[a]
            assert float((got - want).abs().max()) <= want * 2.0 ** -15, (a, got, want)
    server.close()


def test_reported_logprobs_are_those_of_the_logits(example):
    """|error| of fp32 sums over 1,500 columns: some 2^-20 of the row's span, which is below 2^8."""
    torch = torch_cuda()
    s = shape(example)
    ps = prompts(torch, s, (40, 17), seed=9)
    server = example.Server(s, 2, cache="f16", budget=200, piece=8)
    seen = []
    step = server.step
    server.step = lambda t: seen.append((t, step(t))) or seen[-1][1]
    res = server.generate(ps, 6)
    rows = [[], []]
    for t, y in seen:
        at = 0
        for a, part in enumerate(t):
            rows[a] += list(y[at:at + len(part)].double().cpu())
            at += len(part)
    for a, p in enumerate(ps):
        r = res[a]
        fed = p + r["token"][:-1]
        assert len(rows[a]) == len(fed)
        lp = torch.stack(rows[a]).log_softmax(-1)
        want = [float(lp[i, t]) for i, t in enumerate((p + r["token"])[1:])]
        assert max(abs(x - y) for x, y in zip(r["prompt_logprob"] + r["logprob"], want)) <= 2.0 ** -12
        tail = lp[len(p) - 1:]
        ent = (-(tail.exp() * tail).sum(-1)).tolist()
        assert max(abs(x - y) for x, y in zip(r["entropy"], ent)) <= 2.0 ** -12
        assert r["token"] == tail.argmax(-1).tolist()
        for i, top in enumerate(r["top"]):
            assert [t for t, _ in top] == tail[i].topk(len(top)).indices.tolist()
    server.close()


@pytest.mark.parametrize("name,bad", [
    ("q", dict(q=(3, 12, 64))), ("q", dict(q=(3, 11, 128))), ("q", dict(qtype="float32")), ("q", dict(rows=5)),
    ("out", dict(out=(2, 12, 128))), ("out", dict(otype="float64")), ("pool", dict(pool=-1)), ("row_len", dict(row_len=2)),
    ("agent_rows", dict(agent_rows=2)), ("lse", dict(lse=7)), ("weight_out", dict(weight=3))])
def test_binding_refuses_what_does_not_fit(example, name, bad):
    torch = torch_cuda()
    from bit_weight_streaming_q4_gb300.serve import KvPlan
    plan = KvPlan(torch.zeros(2, 1, dtype=torch.int32, device="cuda"), format="f16", heads=12, kv_heads=2, head_dim=128,
                  page_tokens=64, pool_pages=2, max_rows=4)
    rows = bad.get("rows", 3)
    new = lambda n, t: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    q = new(bad.get("q", (rows, 12, 128)), getattr(torch, bad.get("qtype", "float16")))
    out = new(bad.get("out", (rows, 12, 128)), getattr(torch, bad.get("otype", "float32")))
    pool = new(2 * 2 * 2 * 64 * 128 + bad.get("pool", 0), torch.float16)
    kw = dict(lse=new(bad["lse"], torch.float32)) if "lse" in bad else {}
    if "weight" in bad:
        kw["weight_out"] = new(bad["weight"], torch.float32)
    with pytest.raises(ValueError, match=f"^{name}:"):
        plan.attend(pool, new(bad.get("agent_rows", 3), torch.int32), new(bad.get("row_len", rows), torch.int32), q, out, **kw)
