"""Paged caches and plain 64-bit references for the tests of the serving operators (numpy and CPU
torch; nothing here calls the library)."""
import numpy as np
import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def q8_k_byte(slot, dim):
    """Byte of K quant `dim` of slot `slot` in a q8_0 record, as the header places it."""
    return slot * 128 + 16 * ((dim // 16) ^ (2 * (slot % 4) + (slot // 4) % 2)) + dim % 16


class Cache:
    """Sequences of `lens` tokens in a pool whose pages are dealt out in a random order.

    k, v: float64 [agents][kv_heads][cap][D], the values the pool stands for; slots past a
    sequence's pages are zero there.  `room`: slots that the sequences' pages must hold."""

    def __init__(self, fmt, lens, kvh, dim=128, page=64, seed=0, room=None, extra_pages=1, width=None, first_page=0):
        rng = np.random.default_rng(seed)
        self.fmt, self.lens, self.kvh, self.dim, self.page = fmt, list(lens), kvh, dim, page
        need = [-(-max(1, n) // page) for n in (room or lens)]
        self.agents, self.max_pages = len(need), width or max(need)
        self.cap = self.max_pages * page
        self.pages = sum(need) + extra_pages + first_page
        order = rng.permutation(sum(need)) + first_page
        self.table = np.full((self.agents, self.max_pages), -7, dtype=np.int32)  # unused entries: not a page
        at = 0
        for a, n in enumerate(need):
            self.table[a, :n] = order[at:at + n]
            at += n
        if fmt == "q8_0":
            self.pool = torch.from_numpy(rng.integers(0, 256, (self.pages, kvh, 17408), dtype=np.uint8))
            for off in (8192, 16896):
                d = (np.abs(rng.standard_normal((self.pages, kvh, 256))) / 64).astype(np.float16)
                self.pool[:, :, off:off + 512] = torch.from_numpy(d.view(np.uint8))
        else:
            g = torch.Generator().manual_seed(seed)
            self.pool = torch.randn(self.pages, kvh, 2, page, dim, generator=g).to(TYPES[fmt])

    def parts(self, pool=None):
        """The pool's K and V by page: float64 [pages][kv_heads][2][page][D]."""
        p = self.pool if pool is None else pool
        if self.fmt != "q8_0":
            return p.double().numpy()
        b = p.numpy()
        t, d = np.meshgrid(np.arange(64), np.arange(128), indexing="ij")
        kq = b[:, :, q8_k_byte(t, d)].view(np.int8).astype(np.float64)
        ks = np.ascontiguousarray(b[:, :, 8192:8704]).view(np.float16).astype(np.float64)[:, :, t * 4 + d // 32]
        vq = b[:, :, 8704 + d * 64 + t].view(np.int8).astype(np.float64)
        vs = np.ascontiguousarray(b[:, :, 16896:]).view(np.float16).astype(np.float64)[:, :, (d // 32) * 64 + t]
        with np.errstate(invalid="ignore"):
            return np.stack([kq * ks, vq * vs], axis=2)

    def values(self, pool=None):
        """K, V float64 [agents][kv_heads][cap][D]."""
        x = self.parts(pool)
        out = np.zeros((2, self.agents, self.kvh, self.cap, self.dim))
        for a in range(self.agents):
            for i, pg in enumerate(self.table[a]):
                if 0 <= pg < self.pages:
                    out[:, a, :, i * self.page:(i + 1) * self.page] = x[pg].transpose(1, 0, 2, 3)
        return out[0], out[1]

    def plan(self, heads, rows, agent_rows=None):
        from bit_weight_streaming_q4_gb300 import serve
        return serve.KvPlan(torch.from_numpy(self.table).cuda(), format=self.fmt, heads=heads, kv_heads=self.kvh,
                            head_dim=self.dim, page_tokens=self.page, pool_pages=self.pages, max_rows=rows,
                            max_agent_rows=agent_rows or rows)


def attend_ref(k, v, agent_rows, row_len, q, scale, weight_in=None):
    """Attention in 64 bits: q float64 [rows][heads][D].  Returns out, lse, weight, and per output
    the sums that the tolerances are made of: sum p |v| and the largest sum |q k| scale of a row."""
    rows, heads, dim = q.shape
    agents, kvh, cap = k.shape[:3]
    grp = heads // kvh
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((rows, heads), -np.inf)
    big = np.zeros((rows, heads))
    weight = np.zeros((agents, kvh, cap)) if weight_in is None else np.array(weight_in, dtype=np.float64)
    wtol = np.zeros((agents, kvh, cap))
    for a in range(agents):
        for r in range(agent_rows[a], agent_rows[a + 1]):
            n = row_len[r]
            if n == 0:
                continue
            for h in range(heads):
                g = h // grp
                x = k[a, g, :n] @ q[r, h] * scale
                big[r, h] = (np.abs(k[a, g, :n]) @ np.abs(q[r, h])).max() * abs(scale) + np.abs(x).max()
                m = x.max()
                e = np.exp(x - m)
                p = e / e.sum()
                out[r, h], mag[r, h] = p @ v[a, g, :n], p @ np.abs(v[a, g, :n])
                lse[r, h] = m + np.log(e.sum())
                weight[a, g, :n] += p
                wtol[a, g, :n] += p * 4 * score_error(big[r, h])
    return {"out": out, "lse": lse, "weight": weight, "mag": mag, "big": big, "wtol": wtol}


def score_error(big):
    """Bound on a base-e score's error: fp32 sums of exact products (each partial sum rounded, by
    at most 2^-22 of the sum of magnitudes, the tensor core's truncation included), the scaling's
    and the shift's roundings, and the exponential's own error (2^-21)."""
    return 2.0 ** -22 * big + 2.0 ** -20


def check_attend(ref, out, lse, weight, kind, split_bits):
    """out's tolerance: each probability is off by at most twice the score's error on either
    side of the division (4 in all), its two parts lose 2^-split_bits, and the result is
    rounded once to `kind`."""
    err = score_error(ref["big"])[..., None]
    ulp = {"f32": 2.0 ** -23, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    tol = ref["mag"] * (4 * err + 2.0 ** -split_bits) + ulp * np.abs(ref["out"]) + (2.0 ** -25 if kind == "f16" else 1e-30)
    bad = np.abs(out - ref["out"]) - tol
    assert np.isfinite(out).all()
    assert (bad <= 0).all(), f"out: worst {np.max(np.abs(out - ref['out']) / tol):.3f} of the tolerance"
    if lse is not None:
        seen = np.isfinite(ref["lse"])
        assert np.array_equal(np.isneginf(lse), ~seen)
        tol = 2 * score_error(ref["big"][seen]) + 2.0 ** -22 * np.abs(ref["lse"][seen])
        assert (np.abs(lse[seen] - ref["lse"][seen]) <= tol).all()
    if weight is not None:
        tol = ref["wtol"] + 2.0 ** -22 * np.abs(ref["weight"]) + 1e-30
        diff = np.abs(weight - ref["weight"])
        assert (diff <= tol).all(), f"weight: worst {np.max(diff / tol):.3f} of the tolerance"


def quantise_ref(x):
    """q8_0 of fp32 [..., D]: (scales fp16 [..., D / 32], quants int8 [..., D]), each step in fp32."""
    x = np.asarray(x, dtype=np.float32)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(all="ignore"):
        big = np.abs(b).max(-1)
        d = np.minimum(big / np.float32(127), np.float32(65504)).astype(np.float16)
        inv = np.where(d == 0, np.float32(0), np.float32(1) / np.where(d == 0, np.float16(1), d).astype(np.float32))
        q = np.clip(np.rint(b * inv[..., None]), -127, 127)
        odd = ~np.isfinite(b).all(-1)
        d = np.where(odd, np.float16(np.nan), d)
        q = np.where(odd[..., None], 0, q).astype(np.int8)
    return d, q.reshape(x.shape)


def evict_ref(weight, pos, n, keep, sink, protect_from):
    """Slots kept of 0 .. n - 1, by the definition: a list of (slot, where it ends up)."""
    budget = n if keep < 0 else min(n, keep)

    def rank(t):
        if pos[t] < sink or pos[t] >= protect_from:
            return (2, 0.0)
        w = float(weight[t])
        return (0, 0.0) if np.isnan(w) else (1, w + 0.0)
    order = sorted(range(n), key=lambda t: (tuple(-x for x in rank(t)), t))[:budget]
    kept = set(order)
    holes = [t for t in range(budget) if t not in kept]
    late = sorted(t for t in kept if t >= budget)
    return budget, list(zip(late, holes))
