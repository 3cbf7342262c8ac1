"""Cases of the serving operators around a decode step's matmuls: appending to a paged KV cache,
attention of new tokens over it with accumulated attention weights, eviction by those weights, and
log probabilities of tokens with entropy and top alternatives.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own``
is set, with the framework's operators.  ``exact`` is the definition in 64 bits."""
import math

import torch

own = False

# The 27B-shaped stack of this repository: 48 query heads over 8 KV heads of 128, an lm_head of
# 151,936 columns, 4 sequences of 23,000 cached tokens with 1 token and 2 drafts each, 8 of 16,000
# with 1 and 7, a pool of about 132K tokens, and chunks of 524 rows.
HEADS, KV_HEADS, DIM, VOCAB = 48, 8, 128, 151936
Q8_REC = 17408  # bytes of a q8_0 record: 64 tokens of one KV head


def _attend(name, fmt, agents, lo, hi, rows, heads=HEADS, kvh=KV_HEADS, dim=DIM, page=64):
    return {"name": name, "op": "attend", "fmt": fmt, "agents": agents, "lo": lo, "hi": hi, "rows": rows,
            "heads": heads, "kvh": kvh, "dim": dim, "page": page}


def _evict(name, fmt, agents, lo, hi, keep, sink, recent, kvh=KV_HEADS, dim=DIM, page=64):
    return {"name": name, "op": "evict", "fmt": fmt, "agents": agents, "lo": lo, "hi": hi, "keep": keep,
            "sink": sink, "recent": recent, "kvh": kvh, "dim": dim, "page": page}


def _append(name, fmt, src, agents, lo, hi, rows, heads=HEADS, kvh=KV_HEADS, dim=DIM, page=64):
    return {"name": name, "op": "append", "fmt": fmt, "src": src, "agents": agents, "lo": lo, "hi": hi, "rows": rows,
            "heads": heads, "kvh": kvh, "dim": dim, "page": page}


def _logprobs(name, m, n, top, given=1, kind="f32", masked=0.0):
    return {"name": name, "op": "logprobs", "m": m, "n": n, "top": top, "given": given, "kind": kind, "masked": masked}


def listed():
    return [
        # a conversation's first turn: one token over a short prompt, where latency counts
        _attend("attend f16 1x70", "f16", 1, 70, 70, 1, page=16),
        # the decode step: 4 long conversations, a token and two drafts each, on the q8_0 pool
        _attend("attend q8_0 4x23000 r3", "q8_0", 4, 23000, 23003, 3),
        # one sequence that holds the whole pool, one token
        _attend("attend f16 1x131071", "f16", 1, 131071, 131071, 1),
        # many short and middling conversations of ragged lengths, small heads
        _attend("attend bf16 61 ragged d64", "bf16", 61, 1, 4099, 1, heads=32, kvh=8, dim=64, page=32),
        # the wide verify step: 8 sequences, a token and seven drafts each
        _attend("attend bf16 8x16000 r8", "bf16", 8, 16000, 16008, 8),
        # a small cache trimmed by a few tokens
        _evict("evict f16 1x333", "f16", 1, 333, 333, 256, 4, 32, page=16),
        # the decode step's caches cut to half
        _evict("evict f16 4x23003", "f16", 4, 23003, 23003, 11500, 4, 1024),
        # ragged caches of a shared q8_0 pool, some of them under the budget already
        _evict("evict q8_0 8 ragged", "q8_0", 8, 3000, 16008, 8000, 16, 500),
        # the decode step's twelve rows, from the qkv projection's output
        _append("append q8_0 4x3", "q8_0", "f32", 4, 22990, 23000, 3),
        # a prompt, from the same
        _append("append f16 1x8191", "f16", "f32", 1, 77, 77, 8191),
        # the lm_head's rows of a decode step
        _logprobs("logprobs 12 top 20", 12, VOCAB, 20),
        # the rows of a prompt's chunk: every prompt token's probability
        _logprobs("logprobs 524 top 5", 524, VOCAB, 5),
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "evict", "append", "logprobs"])
    if op == "logprobs":
        m = _log_between(rng, 1, 500)
        kind = rng.choice(["f32", "f32", "f16", "bf16"])
        n = rng.choice([VOCAB, _log_between(rng, 50, 200000)])
        c = _logprobs("", m, n, rng.randint(0, min(32, n)), rng.choice([0, 1, 1, 3]), kind, rng.choice([0.0, 0.0, 0.4]))
    else:
        fmt = rng.choice(["q8_0", "f16", "bf16"])
        dim = 128 if fmt == "q8_0" else rng.choice([64, 128, 128, 256])
        page = 64 if fmt == "q8_0" else rng.choice([16, 32, 64, 128])
        kvh = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 6])
        most = min(128000, 128000 * 8 * 128 // (kvh * dim))
        hi = _log_between(rng, 2, most)
        agents = max(1, min(64, _log_between(rng, 1, 64), most // hi))
        lo = rng.choice([hi, rng.randint(1, hi)])
        if op == "attend":
            c = _attend("", fmt, agents, lo, hi, rng.choice([1, 1, 3, 5, 8]), group * kvh, kvh, dim, page)
        elif op == "evict":
            keep = rng.randint(1, hi)
            sink = rng.randint(0, 16)
            c = _evict("", fmt, agents, lo, hi, keep, sink, rng.randint(0, max(1, keep // 2)), kvh, dim, page)
        else:
            rows = _log_between(rng, 1, max(1, min(2048, 8191 // agents)))
            c = _append("", fmt, rng.choice(["f32", "f32", "f16", "bf16"]), agents, 0, min(hi, 20000), rows, group * kvh, kvh, dim, page)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs
KINDS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def lengths(case):
    """The sequences' cached tokens: spread over lo .. hi, the last one hi."""
    a, lo, hi = case["agents"], case["lo"], case["hi"]
    return [lo + round((hi - lo) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(a - 1)] + [hi]


def _totals(case):
    """Tokens that a sequence's pages have to hold."""
    more = case["rows"] if case["op"] == "append" else 0
    return [n + more for n in lengths(case)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(case, g):
    """A shared pool whose pages are dealt out in a random order, and the page table."""
    page, kvh, dim = case["page"], case["kvh"], case["dim"]
    need = [-(-max(n, 1) // page) for n in _totals(case)]
    total, width = sum(need), max(need)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(len(need), width, dtype=torch.int32)
    at = 0
    for a, n in enumerate(need):
        table[a, :n] = order[at:at + n]
        at += n
    if case["fmt"] == "q8_0":
        # quants of the whole range, scales that give values of order one
        pool = torch.randint(0, 256, (total, kvh, Q8_REC), generator=g, device="cuda", dtype=torch.uint8)
        for at in (8192, 16896):
            d = (torch.randn(total, kvh, 256, generator=g, device="cuda").abs() / 64).half()
            pool[:, :, at:at + 512] = d.view(torch.uint8)
    else:
        pool = torch.empty(total, kvh, 2, page, dim, dtype=KINDS[case["fmt"]], device="cuda")
        pool.normal_(generator=g)
    return pool, table.cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "logprobs":
        m, n = case["m"], case["n"]
        x = torch.randn(m, n, generator=g, device="cuda") * 2.5
        if case["masked"]:  # an answer held to a grammar
            x.masked_fill_(torch.rand(m, n, generator=g, device="cuda") < case["masked"], -math.inf)
            x[:, 0] = 0.5
        s["logits"] = x.to(KINDS[case["kind"]])
        s["tokens"] = torch.randint(0, n, (m, case["given"]), generator=g, device="cuda").to(torch.int32)
        f32 = dict(dtype=torch.float32, device="cuda")
        s["out"] = {"lse": torch.empty(m, **f32), "entropy": torch.empty(m, **f32),
                    "logprob": torch.empty(m, case["given"], **f32), "top_logprob": torch.empty(m, case["top"], **f32),
                    "top_index": torch.empty(m, case["top"], dtype=torch.int32, device="cuda")}
        return s
    pool, table = _cache(case, g)
    agents, kvh, dim = case["agents"], case["kvh"], case["dim"]
    cap = table.shape[1] * case["page"]
    lens = lengths(case)
    s.update(pool=pool, table=table, cap=cap, lens=_i32(lens))
    slots = torch.arange(cap, device="cuda")
    if op == "attend":
        r = case["rows"]
        s["agent_rows"] = _i32([a * r for a in range(agents + 1)])
        # a token and its drafts: each row sees one token more than the one before it
        s["row_len"] = _i32([max(0, n - (r - 1 - j)) for n in lens for j in range(r)])
        kind = torch.bfloat16 if case["fmt"] == "bf16" else torch.float16
        s["q"] = torch.randn(agents * r, case["heads"], dim, generator=g, device="cuda").to(kind)
        s["weight_in"] = torch.rand(agents, kvh, cap, generator=g, device="cuda")
        s["weight_out"] = torch.zeros(agents, kvh, cap, device="cuda")
        s["out"] = torch.empty(agents * r, case["heads"], dim, dtype=kind, device="cuda")
        s["lse"] = torch.empty(agents * r, case["heads"], device="cuda")
    elif op == "evict":
        # accumulated weights fall off steeply, and an earlier eviction has mixed the older slots
        s["weight"] = torch.rand(agents, kvh, cap, generator=g, device="cuda").pow(4) * 30
        mixed = torch.rand(agents, kvh, cap, generator=g, device="cuda")
        s["pos"] = torch.where(slots < (s["lens"] // 2)[:, None, None], mixed, slots + 1.0).argsort(-1).to(torch.int32)
        s["keep"] = _i32([case["keep"]] * agents)
        s["protect_from"] = _i32([n - case["recent"] for n in lens])
        s["weight_out"] = torch.zeros(agents, kvh, cap, device="cuda")
        s["pos_out"] = torch.zeros(agents, kvh, cap, dtype=torch.int32, device="cuda")
        s["len_out"] = torch.zeros(agents, dtype=torch.int32, device="cuda")
    else:
        r, heads = case["rows"], case["heads"]
        # the qkv projection's output, K and V being columns of it
        y = torch.randn(agents * r, (heads + 2 * kvh) * dim, generator=g, device="cuda").to(KINDS[case["src"]])
        s["y"] = y
        s["k"] = y[:, heads * dim:(heads + kvh) * dim].unflatten(1, (kvh, dim))
        s["v"] = y[:, (heads + kvh) * dim:].unflatten(1, (kvh, dim))
        s["agent_rows"] = _i32([a * r for a in range(agents + 1)])
        s["row_pos"] = _i32([n + j for n in lens for j in range(r)])
        s["weight"] = torch.rand(agents, kvh, cap, generator=g, device="cuda")
        s["pos"] = slots.expand(agents, kvh, cap).to(torch.int32).contiguous()
    if own:  # what a serving program sets up once: the plan with its workspace and error word
        from bit_weight_streaming_q4_gb300 import serve
        s["plan"] = serve.KvPlan(s["table"], format=case["fmt"], heads=case.get("heads", kvh), kv_heads=kvh, head_dim=dim,
                                 page_tokens=case["page"], pool_pages=pool.shape[0], max_rows=agents * case.get("rows", 1),
                                 max_agent_rows=case.get("rows", 1))
    return s


# ------------------------------------------------------------------------------ the passes
def run(s):
    return {"attend": _run_attend, "evict": _run_evict, "append": _run_append, "logprobs": _run_logprobs}[s["case"]["op"]](s)


def _pool_parts(s):
    """The cache's contents as numbers (views of the pool): quants and scales, or the values."""
    p = s["pool"]
    if s["case"]["fmt"] != "q8_0":
        return {"pool": p}
    return {"k_quant": p[:, :, :8192].view(torch.int8), "k_scale": p[:, :, 8192:8704].view(torch.float16),
            "v_quant": p[:, :, 8704:16896].view(torch.int8), "v_scale": p[:, :, 16896:].view(torch.float16)}


def _k_place(slot, dim):
    """Byte of K quant `dim` of the token in slot `slot` of a q8_0 record."""
    return slot * 128 + 16 * ((dim // 16) ^ (2 * (slot % 4) + (slot // 4) % 2)) + dim % 16


def _values(s):
    """K and V of all cached tokens in 32 bits, [agents, kv_heads, cap, dim] each."""
    c, table = s["case"], s["table"].long()
    a, w = table.shape
    kvh, page, dim = c["kvh"], c["page"], c["dim"]
    if c["fmt"] != "q8_0":
        rec = s["pool"][table]  # [a, w, kvh, 2, page, dim]
        k, v = (rec[:, :, :, i].permute(0, 2, 1, 3, 4).reshape(a, kvh, w * page, dim).float() for i in (0, 1))
        return k, v
    part = {n: x[table] for n, x in _pool_parts(s).items()}  # [a, w, kvh, ...]
    t = torch.arange(64, device="cuda")[:, None]
    place = _k_place(t, torch.arange(128, device="cuda")).reshape(-1)
    k = part["k_quant"][..., place].unflatten(-1, (64, 4, 32)).float() * part["k_scale"].unflatten(-1, (64, 4)).float()[..., None]
    v = part["v_quant"].unflatten(-1, (4, 32, 64)).float() * part["v_scale"].unflatten(-1, (4, 1, 64)).float()
    k = k.flatten(-2).permute(0, 2, 1, 3, 4).reshape(a, kvh, w * 64, 128)
    v = v.flatten(-3, -2).transpose(-1, -2).permute(0, 2, 1, 3, 4).reshape(a, kvh, w * 64, 128)
    return k, v


def _run_attend(s):
    if own:
        s["plan"].attend(s["pool"], s["agent_rows"], s["row_len"], s["q"], s["out"], lse=s["lse"],
                         weight_in=s["weight_in"], weight_out=s["weight_out"])
        return {"out": s["out"], "lse": s["lse"], "weight": s["weight_out"]}
    c = s["case"]
    a, r, kvh, dim, cap = c["agents"], c["rows"], c["kvh"], c["dim"], s["cap"]
    grp = c["heads"] // kvh
    k, v = _values(s)
    q = s["q"].float().view(a, r, kvh, grp, dim).permute(0, 2, 1, 3, 4).reshape(a, kvh, r * grp, dim)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(dim))
    n = s["row_len"].view(a, r).repeat_interleave(grp, 1)  # tokens that a query sees
    slot = torch.arange(cap, device="cuda")
    x = x.masked_fill_((slot >= n[..., None])[:, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    p = e / z.clamp(min=1e-38)
    seen = (slot < s["lens"][:, None])[:, None, :]
    v = v.masked_fill_(~seen[..., None], 0.0)
    out = torch.matmul(p, v)
    out = out.view(a, kvh, r, grp, dim).permute(0, 2, 1, 3, 4).reshape(a * r, c["heads"], dim)
    lse = (top + torch.log(z))[..., 0].view(a, kvh, r, grp).permute(0, 2, 1, 3).reshape(a * r, c["heads"])
    weight = torch.where(seen, s["weight_in"] + p.sum(2), s["weight_out"])
    return {"out": out.to(s["q"].dtype), "lse": lse, "weight": weight}


def _run_evict(s):
    c = s["case"]
    if own:
        s["plan"].evict(s["pool"], s["lens"], s["keep"], s["weight"], s["pos"], weight_out=s["weight_out"],
                        pos_out=s["pos_out"], len_out=s["len_out"], sink=c["sink"], protect_from=s["protect_from"])
        return {**_pool_parts(s), "weight": s["weight_out"], "pos": s["pos_out"], "len": s["len_out"]}
    kvh, page = c["kvh"], c["page"]
    slot = torch.arange(s["cap"], device="cuda")
    n = s["lens"].long()[:, None, None]
    budget = torch.minimum(n, s["keep"].long()[:, None, None])
    safe = (s["pos"] < c["sink"]) | (s["pos"] >= s["protect_from"][:, None, None])
    key = torch.where(safe, math.inf, s["weight"]).masked_fill(slot >= n, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.empty_like(safe).scatter_(-1, order, (slot < budget).expand_as(safe))
    holes = (~kept & (slot < budget)).nonzero()
    moved = (kept & (slot >= budget)).nonzero()
    a, g, at, src = moved[:, 0], moved[:, 1], holes[:, 2], moved[:, 2]
    new = slot < budget
    weight = torch.where(new, s["weight"], s["weight_out"])
    pos = torch.where(new, s["pos"], s["pos_out"])
    weight[a, g, at] = s["weight"][a, g, src]
    pos[a, g, at] = s["pos"][a, g, src]
    to, frm = (s["table"].long()[a, x // page] for x in (at, src))
    at, src = at % page, src % page
    p = s["pool"]
    if c["fmt"] != "q8_0":
        p[to, g, :, at] = p[frm, g, :, src]
    else:
        d = torch.arange(128, device="cuda")
        byte = torch.arange(8, device="cuda")
        blk = torch.arange(4, device="cuda").repeat_interleave(2)
        low = torch.arange(2, device="cuda").repeat(4)

        def places(t):
            t = t[:, None]
            return torch.cat([_k_place(t, d), 8192 + t * 8 + byte, 8704 + d * 64 + t, 16896 + (blk * 64 + t) * 2 + low], 1)
        p[to[:, None], g[:, None], places(at)] = p[frm[:, None], g[:, None], places(src)]
    return {**_pool_parts(s), "weight": weight, "pos": pos, "len": budget[:, 0, 0].to(torch.int32)}


def _run_append(s):
    c = s["case"]
    if own:
        s["plan"].append(s["pool"], s["agent_rows"], s["lens"], s["k"], s["v"], weight=s["weight"], pos=s["pos"], row_pos=s["row_pos"])
        return {**_pool_parts(s), "weight": s["weight"], "pos": s["pos"]}
    a, r, kvh, dim, page = c["agents"], c["rows"], c["kvh"], c["dim"], c["page"]
    seq = torch.arange(a, device="cuda").repeat_interleave(r)
    slot = s["lens"].long()[seq] + torch.arange(r, device="cuda").repeat(a)
    to, at = s["table"].long()[seq, slot // page], slot % page
    s["weight"][seq, :, slot] = 0.0
    s["pos"][seq, :, slot] = s["row_pos"][:, None].expand(-1, kvh)
    k, v = s["k"].float(), s["v"].float()
    p = s["pool"]
    if c["fmt"] != "q8_0":
        p[to, :, 0, at] = k.to(p.dtype)
        p[to, :, 1, at] = v.to(p.dtype)
        return {**_pool_parts(s), "weight": s["weight"], "pos": s["pos"]}

    def quantise(x):
        x = x.unflatten(-1, (4, 32))
        big = x.abs().amax(-1)
        d = torch.div(big, torch.full_like(big, 127.0)).clamp(max=65504.0).half()
        inv = torch.where(d == 0, 0.0, torch.reciprocal(d.float()))
        return d, torch.round(x * inv[..., None]).clamp_(-127, 127).to(torch.int8).flatten(-2)

    g = torch.arange(kvh, device="cuda")[:, None]
    dims, blk = torch.arange(128, device="cuda"), torch.arange(4, device="cuda")
    to, at = to[:, None, None], at[:, None, None]
    part = _pool_parts(s)
    d, x = quantise(k)
    part["k_quant"][to, g, _k_place(at, dims)] = x
    part["k_scale"][to, g, at * 4 + blk] = d
    d, x = quantise(v)
    part["v_quant"][to, g, dims * 64 + at] = x
    part["v_scale"][to, g, blk * 64 + at] = d
    return {**part, "weight": s["weight"], "pos": s["pos"]}


def _run_logprobs(s):
    c = s["case"]
    if own:
        from bit_weight_streaming_q4_gb300 import serve
        o = s["out"]
        serve.logprobs(s["logits"], s["tokens"], o["lse"], o["logprob"], o["entropy"], o["top_index"], o["top_logprob"])
        return o
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    y = x - top
    e = torch.exp(y)
    z = e.sum(-1, keepdim=True)
    lse = top + torch.log(z)
    entropy = torch.log(z)[:, 0] - torch.where(e > 0, e * y, 0.0).sum(-1) / z[:, 0]
    value, index = torch.sort(x, dim=-1, descending=True, stable=True)
    return {"lse": lse[:, 0], "entropy": entropy, "logprob": x.gather(1, s["tokens"].long()) - lse,
            "top_logprob": value[:, :c["top"]] - lse, "top_index": index[:, :c["top"]].to(torch.int32)}


# ------------------------------------------------------------------------------ what a pass cannot do without
def _token_bytes(case):
    """Bytes of one token's K and V of one KV head."""
    return 272 if case["fmt"] == "q8_0" else 4 * case["dim"]


def work(case):
    if case["op"] == "logprobs":
        m, n = case["m"], case["n"]
        return {"bytes": m * n * torch.empty(0, dtype=KINDS[case["kind"]]).element_size() + m * (8 + 8 * case["given"] + 8 * case["top"]),
                "flops": 5 * m * n}
    tok, kvh, a = _token_bytes(case), case["kvh"], case["agents"]
    lens = lengths(case)
    if case["op"] == "attend":
        rows, heads, dim = a * case["rows"], case["heads"], case["dim"]
        seen = sum(max(0, n - j) for n in lens for j in range(case["rows"]))
        return {"bytes": sum(lens) * kvh * (tok + 8) + rows * heads * (4 * dim + 4), "flops": 4 * seen * heads * dim}
    if case["op"] == "append":
        rows = a * case["rows"]
        size = torch.empty(0, dtype=KINDS[case["src"]]).element_size()
        return {"bytes": rows * kvh * (2 * case["dim"] * size + tok + 8), "flops": rows * kvh * 2 * case["dim"]}
    moved = kept = 0.0
    for n in lens:
        b = min(n, case["keep"])
        safe = min(b, case["sink"] + case["recent"])
        late = min(n - b, case["recent"], b)  # protected ones past the budget, and the even share of the rest
        kept += b
        moved += late + max(0, n - b - late) * max(0, b - safe) / max(1, n - safe)
    return {"bytes": kvh * (8 * sum(lens) + 8 * kept + 2 * tok * moved), "flops": 4 * kvh * sum(lens)}


# ------------------------------------------------------------------------------ the definition in 64 bits
def _token(s, a, g, n):
    """K and V [n, dim] of the first n tokens of sequence a, KV head g, token by token's place."""
    c = s["case"]
    t = torch.arange(n, device="cuda")
    page, at = s["table"][a].long()[t // c["page"]], t % c["page"]
    p = s["pool"]
    if c["fmt"] != "q8_0":
        return p[page, g, 0, at].double(), p[page, g, 1, at].double()
    rec = p[page, g]  # [n, 17408]
    dim = torch.arange(128, device="cuda").expand(n, 128)
    tt = at[:, None]
    kb = tt * 128 + 16 * torch.bitwise_xor(dim // 16, 2 * (tt % 4) + (tt // 4) % 2) + dim % 16
    half = rec.view(torch.float16)
    k = rec.gather(1, kb).view(torch.int8).double() * half.gather(1, 4096 + tt * 4 + dim // 32).double()
    v = rec.gather(1, 8704 + dim * 64 + tt).view(torch.int8).double() * half.gather(1, 8448 + dim // 32 * 64 + tt).double()
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        x = s["logits"].double()
        lse = torch.logsumexp(x, -1)
        lp = x - lse[:, None]
        entropy = -torch.special.xlogy(lp.exp(), lp.exp()).sum(-1)
        best = torch.topk(lp, case["top"], dim=-1).values if case["top"] else lp[:, :0]
        return {"lse": lse, "entropy": entropy, "logprob": lp.gather(1, s["tokens"].long()), "top_logprob": best, "top_index": None}
    lens = lengths(case)
    if case["op"] == "attend":
        grp, r = case["heads"] // case["kvh"], case["rows"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        weight = s["weight_out"].double()
        for a in range(case["agents"]):
            for g in range(case["kvh"]):
                k, v = _token(s, a, g, lens[a])
                w = s["weight_in"][a, g, :lens[a]].double()
                for j in range(r):
                    n = max(0, lens[a] - (r - 1 - j))
                    if n:
                        x = s["q"][a * r + j, g * grp:(g + 1) * grp].double() @ k[:n].T / math.sqrt(case["dim"])
                        p = torch.softmax(x, -1)
                        out[a * r + j, g * grp:(g + 1) * grp] = p @ v[:n]
                        lse[a * r + j, g * grp:(g + 1) * grp] = torch.logsumexp(x, -1)
                        w[:n] += p.sum(0)
                weight[a, g, :lens[a]] = w
        return {"out": out, "lse": lse, "weight": weight}
    if case["op"] == "evict":
        weight, pos = s["weight_out"].double(), None
        parts = {n: None for n in _pool_parts(s)}
        for a in range(case["agents"]):
            n = lens[a]
            b = min(n, case["keep"])
            for g in range(case["kvh"]):
                w, at = s["weight"][a, g, :n].double(), s["pos"][a, g, :n]
                rank = torch.where((at < case["sink"]) | (at >= n - case["recent"]), math.inf, w)
                keep = torch.sort(torch.argsort(rank, descending=True, stable=True)[:b]).values
                stay, go = keep[keep < b], keep[keep >= b]
                free = torch.ones(b, dtype=torch.bool, device="cuda")
                free[stay] = False
                weight[a, g, stay] = w[stay]
                weight[a, g, free.nonzero()[:, 0]] = w[go]
        return {**parts, "weight": weight, "pos": pos, "len": None}
    out = {n: None for n in _pool_parts(s)}
    weight = s["weight"].double()
    pool = s["pool"].double() if case["fmt"] != "q8_0" else None
    scales = {n: x.double() for n, x in _pool_parts(s).items() if n.endswith("scale")}
    for a in range(case["agents"]):
        for j0 in range(0, case["rows"], 512):
            rows = torch.arange(j0, min(j0 + 512, case["rows"]), device="cuda")
            t = lens[a] + rows
            weight[a][:, t] = 0.0
            page, at, i = s["table"][a].long()[t // case["page"]], t % case["page"], a * case["rows"] + rows
            for g in range(case["kvh"]):
                k, v = s["k"][i, g].double(), s["v"][i, g].double()
                if pool is not None:
                    pool[page, g, 0, at], pool[page, g, 1, at] = k, v
                    continue
                for b in range(4):
                    scales["k_scale"][page, g, at * 4 + b] = k[:, 32 * b:32 * b + 32].abs().amax(-1) / 127
                    scales["v_scale"][page, g, b * 64 + at] = v[:, 32 * b:32 * b + 32].abs().amax(-1) / 127
    return {**out, **({"pool": pool} if pool is not None else scales), "weight": weight, "pos": None}
