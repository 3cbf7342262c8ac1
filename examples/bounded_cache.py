"""Serving sequences with a bounded KV cache and reported log probabilities: the library's matmuls and
serving operators as one loop.

Each step takes the next rows of every sequence (a piece of its prompt, or the token it answered with) and,
layer by layer, multiplies by the qkv matrix, appends K and V to the paged cache, attends over it while
adding up what weight each cached token received, and multiplies by the o matrix.  A sequence that has
outgrown its budget by `slack` tokens is cut back to it: the first `sink` and the last `recent` tokens stay,
then those with the most weight.  The lm_head's rows give the prompt tokens' log probabilities, and each
answered token with its own, the distribution's entropy and the alternatives.

The weights are random (Q4_K, seeded), so the answers mean nothing; shapes, types and calls are those
of a real model.  PyTorch does the embedding, the norms and the rotation of q and k.

    python examples/bounded_cache.py --cache q8_0 --prompts 700 90 333 --new 32 --budget 256
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import synth  # noqa: E402
from bit_weight_streaming_q4_gb300 import Qmm  # noqa: E402
from bit_weight_streaming_q4_gb300.serve import KvPlan, logprobs  # noqa: E402

TOP = 5


@dataclass
class Shape:
    layers: int = 2
    dim: int = 5120
    heads: int = 48
    kv_heads: int = 8
    head_dim: int = 128
    vocab: int = 151936


@dataclass
class Layer:
    qkv: Qmm
    o: Qmm
    pool: torch.Tensor
    weight: torch.Tensor  # [sequences][kv_heads][slots]: attention received so far
    pos: torch.Tensor     # the slots' positions


class Server:
    """Weights, caches and lengths of a fixed set of sequences.

    piece: rows of one sequence per step.  A sequence never holds more than budget + slack + piece tokens."""

    def __init__(self, shape: Shape, sequences: int, *, cache: str = "q8_0", budget: int = 256, slack: int = 32,
                 sink: int = 4, recent: int = 64, piece: int = 16, seed: int = 0):
        s = self.shape = shape
        self.budget, self.slack, self.sink, self.recent, self.piece = budget, slack, sink, recent, piece
        page = 64
        pages = -(-(budget + slack + piece) // page)
        order = torch.randperm(sequences * pages, generator=torch.Generator().manual_seed(seed))
        self.plan = KvPlan(order.to(torch.int32).view(sequences, pages).cuda(), format=cache, heads=s.heads,
                           kv_heads=s.kv_heads, head_dim=s.head_dim, page_tokens=page, pool_pages=sequences * pages,
                           max_rows=sequences * piece, max_agent_rows=piece)
        self.q_type = torch.bfloat16 if cache == "bf16" else torch.float16

        def matrix(n, k, tensor_id):
            blocks = torch.from_numpy(synth.q4k_matrix(n, k, seed=seed, tensor_id=tensor_id).reshape(-1)).cuda()
            return Qmm(blocks, n, k, m_max=sequences * piece)

        self.layers = []
        slots = (sequences, s.kv_heads, pages * page)
        for i in range(s.layers):
            if cache == "q8_0":
                pool = torch.zeros(sequences * pages * s.kv_heads * 17408, dtype=torch.uint8, device="cuda")
            else:
                pool = torch.zeros(sequences * pages, s.kv_heads, 2, page, s.head_dim, dtype=self.q_type, device="cuda")
            self.layers.append(Layer(matrix((s.heads + 2 * s.kv_heads) * s.head_dim, s.dim, 10 * i + 1),
                                     matrix(s.dim, s.heads * s.head_dim, 10 * i + 2), pool,
                                     torch.zeros(slots, device="cuda"), torch.zeros(slots, dtype=torch.int32, device="cuda")))
        self.head = matrix(s.vocab, s.dim, 9)
        self.embed = torch.randn(s.vocab, s.dim, generator=torch.Generator().manual_seed(seed)).half().cuda()
        self.lens = [0] * sequences    # tokens in the cache
        self.seen = [0] * sequences    # tokens that went through it
        self.freq = 10000.0 ** (-torch.arange(0, s.head_dim, 2, device="cuda").float() / s.head_dim)

    def _norm(self, x):
        # (centred: the random weights' mean is not 0; the gain brings products to a spread of about 2)
        x = x - x.mean(-1, keepdim=True)
        return (x * (x.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * 8 * self.shape.dim ** -0.5).half()

    def _rotate(self, x, angle):
        a, b = x.chunk(2, -1)
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    def _i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def step(self, tokens: list[list[int]]) -> torch.Tensor:
        """Logits [rows, vocab] of every sequence's next tokens, which enter the cache."""
        s, n = self.shape, [len(t) for t in tokens]
        starts = [sum(n[:i]) for i in range(len(n) + 1)]
        rows = starts[-1]
        agent_rows, cache_len = self._i32(starts), self._i32(self.lens)
        row_len = self._i32([self.lens[a] + j + 1 for a in range(len(n)) for j in range(n[a])])
        row_pos = self._i32([self.seen[a] + j for a in range(len(n)) for j in range(n[a])])
        angle = row_pos[:, None] * self.freq
        h = self.embed[torch.tensor(sum(tokens, []), device="cuda")].float()
        qkv = torch.empty(rows, (s.heads + 2 * s.kv_heads) * s.head_dim, device="cuda")
        out = torch.empty(rows, s.heads, s.head_dim, dtype=torch.float16, device="cuda")
        o = torch.empty(rows, s.dim, device="cuda")
        lens = [a + b for a, b in zip(self.lens, n)]
        cut = [self.budget if x > self.budget + self.slack else -1 for x in lens]
        self.seen = [a + b for a, b in zip(self.seen, n)]
        for layer in self.layers:
            layer.qkv.run(self._norm(h), qkv)
            q, k, v = qkv.view(rows, -1, s.head_dim).split((s.heads, s.kv_heads, s.kv_heads), 1)
            q, k = self._rotate(q, angle).to(self.q_type), self._rotate(k, angle)
            self.plan.append(layer.pool, agent_rows, cache_len, k, v, weight=layer.weight, pos=layer.pos, row_pos=row_pos)
            self.plan.attend(layer.pool, agent_rows, row_len, q, out, weight_in=layer.weight, weight_out=layer.weight)
            layer.o.run(out.view(rows, -1), o)
            h = h + o * (s.heads * s.head_dim) ** -0.5
            if max(cut) >= 0:
                self.plan.evict(layer.pool, self._i32(lens), self._i32(cut), layer.weight, layer.pos,
                                weight_out=layer.weight, pos_out=layer.pos, len_out=torch.empty_like(cache_len),
                                sink=self.sink, protect_from=self._i32([x - self.recent for x in self.seen]))
        self.lens = [x if c < 0 else min(x, c) for x, c in zip(lens, cut)]
        y = torch.empty(rows, s.vocab, device="cuda")
        self.head.run(self._norm(h), y)
        return y

    def generate(self, prompts: list[list[int]], new: int) -> list[dict]:
        """Greedy answers of `new` tokens.  Per sequence: `prompt_logprob` of the prompt's tokens but the
        first, and per answered token `token`, `logprob`, `entropy` and the `top` alternatives."""
        todo = [list(p) for p in prompts]
        res = [{"prompt_logprob": [], "token": [], "logprob": [], "entropy": [], "top": []} for _ in prompts]
        while any(todo):
            part = [t[:self.piece] for t in todo]
            todo = [t[self.piece:] for t in todo]
            y = self.step(part)
            rows = y.shape[0]
            # the token that follows each row, where the prompt has it (-1: none is known)
            nxt = self._i32([x for p, t in zip(part, todo) for x in p[1:] + (t[:1] or [-1])[:len(p)]]).view(rows, 1)
            given, entropy = torch.empty(rows, 1, device="cuda"), torch.empty(rows, device="cuda")
            top, top_lp = torch.empty(rows, TOP, dtype=torch.int32, device="cuda"), torch.empty(rows, TOP, device="cuda")
            logprobs(y, tokens=nxt, logprob=given, entropy=entropy, top_index=top, top_logprob=top_lp)
            given, entropy, top, top_lp = given.view(-1).tolist(), entropy.tolist(), top.tolist(), top_lp.tolist()
            at = 0
            for a, p in enumerate(part):
                if not p:
                    continue
                last = at + len(p) - 1
                r = res[a]
                if not r["token"]:  # rows of the prompt
                    r["prompt_logprob"] += given[at:last + (1 if todo[a] else 0)]
                if not todo[a] and len(r["token"]) < new:
                    r["token"].append(top[last][0])
                    r["logprob"].append(top_lp[last][0])
                    r["entropy"].append(entropy[last])
                    r["top"].append(list(zip(top[last], top_lp[last])))
                    if len(r["token"]) < new:
                        todo[a].append(top[last][0])
                at += len(p)
        if self.plan.error():
            raise RuntimeError(f"error word {self.plan.error()}")
        return res

    def close(self):
        for m in [self.head] + [x for layer in self.layers for x in (layer.qkv, layer.o)]:
            m.close()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--cache", default="q8_0", choices=["q8_0", "f16", "bf16"])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 90, 333], help="their lengths")
    ap.add_argument("--new", type=int, default=32)
    ap.add_argument("--budget", type=int, default=256)
    args = ap.parse_args()
    shape = Shape(layers=args.layers)
    server = Server(shape, len(args.prompts), cache=args.cache, budget=args.budget)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(shape.vocab, (n,), generator=g).tolist() for n in args.prompts]
    for a, r in enumerate(server.generate(prompts, args.new)):
        print(f"sequence {a}: {server.seen[a]} tokens seen, {server.lens[a]} cached; "
              f"prompt's mean log probability {sum(r['prompt_logprob']) / max(1, len(r['prompt_logprob'])):.3f}")
        for t, lp, e, top in list(zip(r["token"], r["logprob"], r["entropy"], r["top"]))[:4]:
            print(f"  {t:7d}  log p {lp:8.4f}  entropy {e:7.4f}  then " + ", ".join(f"{i} {p:.3f}" for i, p in top[1:]))
    server.close()


if __name__ == "__main__":
    main()
