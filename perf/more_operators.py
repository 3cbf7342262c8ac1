"""Cases of the operators that a decode step with drafts needs between its matmuls: norms and position
rotation of queries and keys, attention with a sliding window and visible first tokens over the paged
cache, and verification of drafted tokens against the target's probabilities.

``run`` computes a case in its plain form (elementary torch operations) or, where ``own`` is set, with
the framework's operators.  ``exact`` is the definition in 64 bits."""
import math

import torch

own = False

# The 27B-shaped stack of this repository: 48 query heads over 8 KV heads of 128, an lm_head of
# 151,936 columns, 4 sequences of 23,000 cached tokens with 1 token and 2 drafts each, 8 of 16,000
# with 1 and 7, chunks of 524 rows.
HEADS, KV_HEADS, DIM, VOCAB = 48, 8, 128, 151936
Q8_REC = 17408  # bytes of a q8_0 record: 64 tokens of one KV head


def _window(name, fmt, agents, lo, hi, rows, window, sinks, heads=HEADS, kvh=KV_HEADS, dim=DIM, page=64):
    return {"name": name, "op": "window", "fmt": fmt, "agents": agents, "lo": lo, "hi": hi, "rows": rows, "window": window,
            "sinks": sinks, "heads": heads, "kvh": kvh, "dim": dim, "page": page}


def _rotate(name, src, dst, rows, start, heads=HEADS, kvh=KV_HEADS, dim=DIM, rot=DIM, axes=1, interleaved=False, norm=True):
    return {"name": name, "op": "rotate", "src": src, "dst": dst, "rows": rows, "start": start, "heads": heads, "kvh": kvh,
            "dim": dim, "rot": rot, "axes": axes, "interleaved": interleaved, "norm": norm}


def _verify(name, agents, rows, n, kind="f32", drafter=True, temperature="mixed"):
    return {"name": name, "op": "verify", "agents": agents, "rows": rows, "n": n, "kind": kind, "drafter": drafter,
            "temperature": temperature}


def listed():
    return [
        # a conversation's first turn on a layer with a short window: one token, where latency counts
        _window("window f16 1x70", "f16", 1, 70, 70, 1, 64, 4, page=16),
        # the decode step: 4 long conversations, a token and two drafts each, on the q8_0 pool
        _window("window q8_0 4x23000 r3", "q8_0", 4, 23000, 23003, 3, 4096, 4),
        # many short and middling conversations of ragged lengths, small heads
        _window("window bf16 61 ragged d64", "bf16", 61, 1, 4099, 1, 1024, 4, heads=32, kvh=8, dim=64, page=32),
        # a long prompt's next piece, the tokens before it cached
        _window("window f16 prompt 2048 of 23000", "f16", 1, 23000, 23000, 2048, 4096, 4),
        # chunks of four prompts at once, beginnings and later pieces, on the q8_0 pool
        _window("window q8_0 prompts 4x524", "q8_0", 4, 500, 9001, 524, 1024, 16),
        # wide heads, odd lengths, no window: plain causal attention of prompts
        _window("window bf16 prompts 3x777 d256", "bf16", 3, 777, 2501, 777, 1 << 30, 0, heads=8, kvh=2, dim=256, page=32),
        # the decode step's twelve rows, from the qkv projection's output
        _rotate("rotate 4x3", "f32", "f16", 12, 23000),
        # a prompt, from the same
        _rotate("rotate 8191", "f32", "f16", 8191, 0),
        # an image's patches among text: time, height and width, part of a wide head rotated
        _rotate("rotate 3 axes 2345", "bf16", "bf16", 2345, 5000, heads=16, kvh=2, dim=256, rot=64, axes=3),
        # the decode step's drafts by a draft head, judged from the lm_head's rows
        _verify("verify 4x3", 4, 3, VOCAB),
        # the wide verify step, drafts by a block drafter
        _verify("verify 8x8", 8, 8, VOCAB),
        # drafts looked up in the text, many short sequences, 16-bit logits of a small vocabulary
        _verify("verify lookup 33x5 bf16", 33, 5, 32001, kind="bf16", drafter=False),
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "rotate", "verify", "verify"])
    if op == "verify":
        n = rng.choice([VOCAB, _log_between(rng, 50, 200000)])
        rows = rng.randint(1, 9)
        agents = _log_between(rng, 1, max(1, 64 * VOCAB // (rows * max(n, 4000))))
        c = _verify("", agents, rows, n, rng.choice(["f32", "f32", "f16", "bf16"]), rng.random() < 0.7,
                    rng.choice(["mixed", "one", "greedy"]))
    elif op == "rotate":
        dim = rng.choice([64, 128, 128, 256])
        kvh = rng.choice([1, 2, 4, 8])
        heads = kvh * rng.choice([1, 2, 4, 6])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        rows = _log_between(rng, 1, 8191 * HEADS * DIM // max(HEADS * DIM, heads * dim))
        c = _rotate("", rng.choice(["f32", "f32", "f16", "bf16"]), rng.choice(["f16", "bf16"]), rows,
                    rng.choice([0, rng.randint(0, 120000)]), heads, kvh, dim, rot, rng.choice([1, 1, 2, 3]),
                    rng.random() < 0.3, rng.random() < 0.7)
    else:
        fmt = rng.choice(["q8_0", "f16", "bf16"])
        dim = 128 if fmt == "q8_0" else rng.choice([64, 128, 128, 256])
        page = 64 if fmt == "q8_0" else rng.choice([16, 32, 64, 128])
        kvh = rng.choice([1, 2, 4, 8])
        heads = kvh * rng.choice([1, 2, 4, 6])
        most = min(128000, 128000 * 8 * 128 // (kvh * dim))
        hi = _log_between(rng, 2, most)
        window = rng.choice([1 << 30, _log_between(rng, 1, 8192), _log_between(rng, 64, 8192)])
        agents = max(1, min(64, _log_between(rng, 1, 64), most // hi))
        seen = min(window, hi)
        rows = max(1, min(2048, hi, 200_000_000_000 // (agents * seen * heads * dim * 4)))
        # (a sequence's scores in 32 bits: at most 4 GB)
        while rows > 1 and rows * heads * min(hi, seen + rows) > 1 << 30:
            rows //= 2
        rows = rng.choice([min(rows, rng.choice([1, 1, 3, 5, 8])), _log_between(rng, 1, rows)])
        c = _window("", fmt, agents, rng.choice([hi, rng.randint(1, hi)]), hi, rows, window, rng.choice([0, 0, 1, 4, 64, 129]),
                    heads, kvh, dim, page)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs
KINDS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def lengths(case):
    """The sequences' tokens, the call's rows among them: spread over lo .. hi, the last one hi."""
    a, lo, hi = case["agents"], case["lo"], case["hi"]
    return [lo + round((hi - lo) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(a - 1)] + [hi]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(case, g):
    """A shared pool whose pages are dealt out in a random order, and the page table."""
    page, kvh, dim = case["page"], case["kvh"], case["dim"]
    need = [-(-max(n, 1) // page) for n in lengths(case)]
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


def _temperatures(case):
    a = case["agents"]
    if case["temperature"] == "greedy":
        return [0.0] * a
    if case["temperature"] == "one":
        return [1.0] * a
    return [(0.7, 1.0, 0.0, 1.3)[i % 4] for i in range(a)]


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "verify":
        return _prepare_verify(s, g)
    if case["op"] == "rotate":
        return _prepare_rotate(s, g)
    pool, table = _cache(case, g)
    agents, r, kvh, dim = case["agents"], case["rows"], case["kvh"], case["dim"]
    lens = lengths(case)
    s.update(pool=pool, table=table, lens=lens)
    s["agent_rows"] = _i32([a * r for a in range(agents + 1)])
    # each row sees one token more than the one before it
    s["row_len"] = _i32([max(0, n - (r - 1 - j)) for n in lens for j in range(r)])
    kind = torch.bfloat16 if case["fmt"] == "bf16" else torch.float16
    s["q"] = torch.randn(agents * r, case["heads"], dim, generator=g, device="cuda").to(kind)
    s["out"] = torch.empty(agents * r, case["heads"], dim, dtype=kind, device="cuda")
    s["lse"] = torch.empty(agents * r, case["heads"], device="cuda")
    if own:  # what a serving program sets up once: the plan with its workspace and error word
        from bit_weight_streaming_q4_gb300 import serve
        s["plan"] = serve.KvPlan(table, format=case["fmt"], heads=case["heads"], kv_heads=kvh, head_dim=dim, page_tokens=case["page"],
                                 pool_pages=pool.shape[0], max_rows=agents * r, max_agent_rows=r)
    return s


def _prepare_rotate(s, g):
    c = s["case"]
    rows, heads, kvh, dim, half = c["rows"], c["heads"], c["kvh"], c["dim"], c["rot"] // 2
    # the qkv projection's output, q and k being columns of it
    s["y"] = (torch.randn(rows, (heads + 2 * kvh) * dim, generator=g, device="cuda") * 3).to(KINDS[c["src"]])
    s["q"] = s["y"][:, :heads * dim].unflatten(1, (heads, dim))
    s["k"] = s["y"][:, heads * dim:(heads + kvh) * dim].unflatten(1, (kvh, dim))
    s["q_weight"] = s["k_weight"] = None
    if c["norm"]:
        s["q_weight"] = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
        s["k_weight"] = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
    s["inv_freq"] = (1e6 ** (-torch.arange(half, device="cuda").double() / half)).float()
    t = torch.arange(rows, device="cuda")
    if c["axes"] == 1:
        s["pos"] = (c["start"] + t).to(torch.int32)
        s["axis"] = None
    else:  # patches in rows of 37: time, height, width
        p = torch.stack([t // 1369, t // 37 % 37, t % 37])[:c["axes"]]
        s["pos"] = (c["start"] + p).to(torch.int32).contiguous()
        s["axis"] = (torch.arange(half, device="cuda") * c["axes"] // half).to(torch.int32)
    s["q_out"] = torch.empty(rows, heads, dim, dtype=KINDS[c["dst"]], device="cuda")
    s["k_out"] = torch.empty(rows, kvh, dim, dtype=KINDS[c["dst"]], device="cuda")
    return s


def _prepare_verify(s, g):
    c = s["case"]
    a, r, n = c["agents"], c["rows"], c["n"]
    # a few tokens of each row are likely, and the drafter mostly knows which
    x = torch.randn(a, r, n, generator=g, device="cuda") * 2
    x.scatter_add_(2, torch.randint(0, n, (a, r, 6), generator=g, device="cuda"), torch.rand(a, r, 6, generator=g, device="cuda") * 6 + 7)
    s["logits"] = x.view(a * r, n).to(KINDS[c["kind"]])
    temps = _temperatures(c)
    s["temperature"] = torch.tensor(temps, dtype=torch.float32, device="cuda")
    d = torch.zeros(a, r, n, device="cuda")  # row j: what token j was drafted from; row 0 has no draft
    d[:, 1:] = x[:, :-1] + 0.8 * torch.randn(a, r - 1, n, generator=g, device="cuda")
    d = d.to(KINDS[c["kind"]])
    noise = -torch.log(torch.rand(a, r, n, generator=g, device="cuda").clamp_(min=1e-30)).log_()
    tokens = (d.float() + noise.neg_() * s["temperature"][:, None, None]).argmax(-1)
    s["tokens"] = tokens.to(torch.int32).view(-1).contiguous()
    s["draft_logits"] = d.view(a * r, n) if c["drafter"] else None
    s["agent_rows"] = _i32([i * r for i in range(a + 1)])
    s["accept_u"] = torch.rand(a * r, generator=g, device="cuda")
    s["sample_u"] = torch.rand(a, generator=g, device="cuda")
    s["accepted"] = torch.empty(a, dtype=torch.int32, device="cuda")
    s["token"] = torch.empty(a, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(a * r, device="cuda")
    if own:
        from bit_weight_streaming_q4_gb300 import serve
        s["plan"] = serve.VerifyPlan(agents=a, max_rows=a * r, columns=n, device=s["logits"].device)
    return s


# ------------------------------------------------------------------------------ the passes
def run(s):
    return {"window": _run_window, "rotate": _run_rotate, "verify": _run_verify}[s["case"]["op"]](s)


def _k_place(slot, dim):
    """Byte of K quant `dim` of the token in slot `slot` of a q8_0 record."""
    return slot * 128 + 16 * ((dim // 16) ^ (2 * (slot % 4) + (slot // 4) % 2)) + dim % 16


def _values(s, pages):
    """K and V of some pages of the pool in 32 bits, [kv_heads, tokens, dim] each."""
    c = s["case"]
    kvh, dim = c["kvh"], c["dim"]
    rec = s["pool"][pages]
    if c["fmt"] != "q8_0":
        return [rec[:, :, i].transpose(0, 1).reshape(kvh, -1, dim).float() for i in (0, 1)]
    t = torch.arange(64, device="cuda")[:, None]
    place = _k_place(t, torch.arange(128, device="cuda")).reshape(-1)
    k = rec[:, :, :8192].view(torch.int8)[..., place].unflatten(-1, (64, 4, 32)).float()
    k = k * rec[:, :, 8192:8704].contiguous().view(torch.float16).unflatten(-1, (64, 4)).float()[..., None]
    v = rec[:, :, 8704:16896].view(torch.int8).unflatten(-1, (4, 32, 64)).float()
    v = v * rec[:, :, 16896:].contiguous().view(torch.float16).unflatten(-1, (4, 1, 64)).float()
    return k.flatten(-2).transpose(0, 1).reshape(kvh, -1, 128), v.flatten(-3, -2).transpose(-1, -2).transpose(0, 1).reshape(kvh, -1, 128)


def _run_window(s):
    c = s["case"]
    if own:
        s["plan"].attend_window(s["pool"], s["agent_rows"], s["row_len"], s["q"], s["out"], window=c["window"], sinks=c["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    r, kvh, dim, page, w, sinks = c["rows"], c["kvh"], c["dim"], c["page"], c["window"], c["sinks"]
    grp = c["heads"] // kvh
    out, lse = [], []
    for a, n in enumerate(s["lens"]):
        # the pages that some row sees
        first = max(0, n - r + 1 - w) // page
        some = list(range(min(first, -(-sinks // page)))) + list(range(first, -(-n // page)))
        at = torch.tensor(some, device="cuda")
        slot = (at[:, None] * page + torch.arange(page, device="cuda")).view(-1)
        k, v = _values(s, s["table"][a].long()[at])
        seen = s["row_len"][a * r:(a + 1) * r, None]
        mask = (slot < seen) & ((slot < sinks) | (slot >= seen - w))  # [r, slots]
        q = s["q"][a * r:(a + 1) * r].float().view(r, kvh, grp, dim).permute(1, 2, 0, 3).reshape(kvh, grp * r, dim)
        x = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(dim)).view(kvh, grp, r, -1)
        x.masked_fill_(~mask, -math.inf)
        top = x.amax(-1, keepdim=True).clamp_(min=-3e38)
        x = x.sub_(top).exp_()
        z = x.sum(-1, keepdim=True)
        o = torch.matmul(x.view(kvh, grp * r, -1), v).view(kvh, grp, r, dim) / z.clamp(min=1e-38)
        out.append(o.permute(2, 0, 1, 3).reshape(r, c["heads"], dim))
        lse.append((top + torch.log(z))[..., 0].permute(2, 0, 1).reshape(r, c["heads"]))
    return {"out": torch.cat(out).to(s["q"].dtype), "lse": torch.cat(lse)}


def _run_rotate(s):
    c = s["case"]
    if own:
        from bit_weight_streaming_q4_gb300 import serve
        serve.rotate(s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                     axis=s["axis"], interleaved=c["interleaved"], eps=1e-6)
        return {"q": s["q_out"], "k": s["k_out"]}
    half, rot = c["rot"] // 2, c["rot"]
    pos = s["pos"][None] if c["axes"] == 1 else s["pos"]
    axis = torch.zeros(half, dtype=torch.int64, device="cuda") if s["axis"] is None else s["axis"].long()
    angle = pos.double().T[:, axis] * s["inv_freq"].double()  # [rows, half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    res = {}
    for name in ("q", "k"):
        x = s[name].float()
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s[name + "_weight"]
        if c["interleaved"]:
            p, q = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([p * cos - q * sin, p * sin + q * cos], -1).flatten(-2)
        else:
            p, q = x[..., :half], x[..., half:rot]
            y = torch.cat([p * cos - q * sin, p * sin + q * cos], -1)
        res[name] = torch.cat([y, x[..., rot:]], -1).to(KINDS[c["dst"]])
    return res


def _softmax(x, temperature):
    """Probabilities in 64 bits; at temperature 0 the whole of it at the lowest of the largest."""
    best = x.double().argmax(-1, keepdim=True)
    greedy = torch.zeros(x.shape, dtype=torch.float64, device=x.device).scatter_(-1, best, 1.0)
    y = x.double() / torch.where(temperature > 0, temperature, 1.0).double()
    e = torch.exp(y - y.amax(-1, keepdim=True))
    return torch.where(temperature > 0, e / e.sum(-1, keepdim=True), greedy)


def _run_verify(s):
    c = s["case"]
    if own:
        s["plan"].verify(s["logits"], s["agent_rows"], s["tokens"], s["accept_u"], s["sample_u"], s["accepted"], s["token"],
                         draft_logits=s["draft_logits"], temperature=s["temperature"], prob=s["prob"])
        return {"accepted": s["accepted"], "token": s["token"], "prob": s["prob"]}
    a, r, n = c["agents"], c["rows"], c["n"]
    seq = torch.arange(a, device="cuda")
    temp = s["temperature"].view(a, 1, 1)
    p = _softmax(s["logits"].view(a, r, n), temp)
    tokens = s["tokens"].long().view(a, r)[:, 1:, None]
    if s["draft_logits"] is None:
        q = torch.zeros_like(p)
        q[:, 1:].scatter_(-1, tokens, 1.0)
    else:
        q = _softmax(s["draft_logits"].view(a, r, n), temp)
        # (without a temperature the draft is right or wrong, whatever it was drawn from)
        q[:, 1:] = torch.where(temp > 0, q[:, 1:], torch.zeros_like(q[:, 1:]).scatter_(-1, tokens, 1.0))
    pt, qt = p[:, :-1].gather(-1, tokens)[..., 0], q[:, 1:].gather(-1, tokens)[..., 0]
    yes = s["accept_u"].double().view(a, r)[:, 1:] * qt < pt
    accepted = yes.long().cumprod(-1).sum(-1)
    prob = torch.zeros(a, r, dtype=torch.float64, device="cuda")
    prob[:, 1:] = (pt / qt).clamp(max=1.0)
    # what the next token is drawn from: the target, less the draft that was refused
    left = p[seq, accepted]
    refused = q[seq, (accepted + 1).clamp(max=r - 1)]
    left = torch.where((accepted < r - 1)[:, None], (left - refused).clamp(min=0.0), left)
    run_up = left.cumsum(-1)
    token = (run_up <= s["sample_u"].double()[:, None] * run_up[:, -1:]).sum(-1)
    return {"accepted": accepted.to(torch.int32), "token": token.to(torch.int32), "prob": prob.float().view(-1)}


# ------------------------------------------------------------------------------ what a pass cannot do without
def _size(kind):
    return 4 if kind == "f32" else 2


def work(case):
    c = case
    if c["op"] == "verify":
        judged = c["rows"] - 1 if c["drafter"] else 0
        bytes_ = c["agents"] * (c["rows"] + judged) * c["n"] * _size(c["kind"]) + c["agents"] * (c["rows"] * 12 + 16)
        return {"bytes": bytes_, "flops": 4 * c["agents"] * (c["rows"] + judged) * c["n"]}
    if c["op"] == "rotate":
        elements = c["rows"] * (c["heads"] + c["kvh"]) * c["dim"]
        return {"bytes": elements * (_size(c["src"]) + _size(c["dst"])) + c["rows"] * c["axes"] * 4, "flops": 7 * elements}
    tok = 272 if c["fmt"] == "q8_0" else 4 * c["dim"]
    r, w, sinks, kvh, heads, dim = c["rows"], c["window"], c["sinks"], c["kvh"], c["heads"], c["dim"]
    cached = seen = 0
    for n in lengths(c):
        first = max(0, n - r + 1 - w)
        cached += n - first + min(first, sinks)
        for j in range(r):
            m = max(0, n - j)
            seen += min(m, w) + min(sinks, max(0, m - w))
    return {"bytes": cached * kvh * tok + c["agents"] * r * heads * (4 * dim + 4), "flops": 4 * seen * heads * dim}


# ------------------------------------------------------------------------------ the definition in 64 bits
def _token(s, a, g, t):
    """K and V [n, dim] of the tokens in slots t of sequence a, KV head g, by each token's place."""
    c = s["case"]
    page, at = s["table"][a].long()[t // c["page"]], t % c["page"]
    p = s["pool"]
    if c["fmt"] != "q8_0":
        return p[page, g, 0, at].double(), p[page, g, 1, at].double()
    rec = p[page, g]  # [n, 17408]
    dim = torch.arange(128, device="cuda").expand(t.numel(), 128)
    tt = at[:, None]
    kb = tt * 128 + 16 * torch.bitwise_xor(dim // 16, 2 * (tt % 4) + (tt // 4) % 2) + dim % 16
    half = rec.view(torch.float16)
    k = rec.gather(1, kb).view(torch.int8).double() * half.gather(1, 4096 + tt * 4 + dim // 32).double()
    v = rec.gather(1, 8704 + dim * 64 + tt).view(torch.int8).double() * half.gather(1, 8448 + dim // 32 * 64 + tt).double()
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    return {"window": _exact_window, "rotate": _exact_rotate, "verify": _exact_verify}[case["op"]](s)


def _exact_window(s):
    c = s["case"]
    if 4 * work(c)["flops"] > 2.5e12:  # (64-bit products: some seconds at most)
        return None
    grp, r, w, sinks = c["heads"] // c["kvh"], c["rows"], c["window"], c["sinks"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for a, n in enumerate(s["lens"]):
        for j0 in range(0, r, 256):  # rows that see much the same tokens
            rows = range(j0, min(r, j0 + 256))
            seen = [max(0, n - (r - 1 - j)) for j in rows]
            if not seen[-1]:
                continue
            begin = max(0, min(seen) - w)
            t = torch.cat([torch.arange(min(sinks, begin), device="cuda"), torch.arange(begin, seen[-1], device="cuda")])
            end = torch.tensor(seen, device="cuda")[:, None, None]
            hidden = (t >= end) | ((t >= sinks) & (t < end - w))
            at = a * r + j0
            for g in range(c["kvh"]):
                k, v = _token(s, a, g, t)
                h = slice(g * grp, (g + 1) * grp)
                x = s["q"][at:at + len(rows), h].double() @ k.T / math.sqrt(c["dim"])
                x = torch.where(hidden, -math.inf, x)
                total = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(total > -math.inf, total, 0.0)[..., None])
                out[at:at + len(rows), h] = p @ v
                lse[at:at + len(rows), h] = total
    return {"out": out, "lse": lse}


def _exact_rotate(s):
    c = s["case"]
    res = {}
    pairs = c["rot"] // 2
    for name in ("q", "k"):
        x = s[name].double()
        if c["norm"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + 1e-6) * s[name + "_weight"].double()
        y = x.clone()
        for i in range(pairs):
            at = s["pos"] if c["axes"] == 1 else s["pos"][int(s["axis"][i])]
            turn = torch.polar(torch.ones(c["rows"], dtype=torch.float64, device="cuda"), at.double() * float(s["inv_freq"][i]))
            lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + pairs)
            z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn[:, None]
            y[..., lo], y[..., hi] = z.real, z.imag
        res[name] = y
    return res


def _exact_verify(s):
    c = s["case"]
    temps = s["temperature"].tolist()
    prob = torch.zeros(c["agents"] * c["rows"], dtype=torch.float64, device="cuda")
    for a, t in enumerate(temps):
        for j in range(1, c["rows"]):
            i = a * c["rows"] + j
            token = int(s["tokens"][i])
            x = s["logits"][i - 1].double()
            if t == 0:
                prob[i] = float(int(torch.nonzero(x == x.max())[0]) == token)
                continue
            log_p = x[token] / t - torch.logsumexp(x / t, -1)
            if s["draft_logits"] is not None:
                y = s["draft_logits"][i].double()
                log_p = log_p - (y[token] / t - torch.logsumexp(y / t, -1))
            prob[i] = torch.exp(torch.clamp(log_p, max=0.0))
    return {"accepted": None, "token": None, "prob": prob}
