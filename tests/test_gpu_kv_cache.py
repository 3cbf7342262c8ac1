"""Appending to the paged cache and evicting from it: what the pool holds afterwards, exactly."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from kv_util import TYPES, Cache, evict_ref, q8_k_byte, quantise_ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ append
def append(c, per, k, v, lens=None, plan=None, weight=True):
    t = torch_cuda()
    ar = np.concatenate([[0], np.cumsum(per)]).tolist()
    rows = ar[-1]
    w, pos = t.full((c.agents, c.kvh, c.cap), 2.5, device="cuda"), t.full((c.agents, c.kvh, c.cap), -9, dtype=t.int32, device="cuda")
    pool = c.pool.cuda()
    plan = plan or c.plan(c.kvh, max(1, rows))
    row_pos = i32([1000 + r for r in range(rows)])
    plan.append(pool, i32(ar), i32(lens or c.lens), k, v, **(dict(weight=w, pos=pos, row_pos=row_pos) if weight else {}))
    t.cuda.synchronize()
    return pool.cpu(), w.cpu().numpy(), pos.cpu().numpy(), plan.error()


def expected(c, per, k, v, skip=()):
    """The pool, weights and positions after appending k, v float32 [rows][kvh][D]."""
    pool = c.pool.clone()
    w, pos = np.full((c.agents, c.kvh, c.cap), 2.5, np.float32), np.full((c.agents, c.kvh, c.cap), -9, np.int32)
    r = 0
    for a, n in enumerate(per):
        for j in range(n):
            t = c.lens[a] + j
            if a not in skip:
                pg, s = int(c.table[a, t // c.page]), t % c.page
                w[a, :, t], pos[a, :, t] = 0, 1000 + r
                if c.fmt != "q8_0":
                    pool[pg, :, 0, s] = torch.from_numpy(k[r]).to(c.pool.dtype)
                    pool[pg, :, 1, s] = torch.from_numpy(v[r]).to(c.pool.dtype)
                else:
                    d = np.arange(128)
                    for i, x in enumerate((k[r], v[r])):
                        sc, q = quantise_ref(x)
                        b = pool[pg].numpy()
                        b[:, q8_k_byte(s, d) if i == 0 else 8704 + d * 64 + s] = q.view(np.uint8)
                        h = b[:, 8192:8704].view(np.float16) if i == 0 else b[:, 16896:].view(np.float16)
                        h[:, 4 * s + np.arange(4) if i == 0 else 64 * np.arange(4) + s] = sc
            r += 1
    return pool, w, pos


def same_pool(c, got, want):
    if c.fmt == "q8_0":
        a, b = got.numpy(), want.numpy()
        for lo, hi in ((8192, 8704), (16896, 17408)):  # scales: a NaN is a NaN
            x, y = a[:, :, lo:hi].view(np.float16), b[:, :, lo:hi].view(np.float16)
            assert np.array_equal(np.isnan(x), np.isnan(y)) and np.array_equal(x[~np.isnan(x)], y[~np.isnan(y)])
        for lo, hi in ((0, 8192), (8704, 16896)):
            assert np.array_equal(a[:, :, lo:hi], b[:, :, lo:hi])
    else:
        assert torch.equal(got.view(torch.int16)[~got.isnan()], want.view(torch.int16)[~got.isnan()])
        assert torch.equal(got.isnan(), want.isnan())


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64), ("f16", 64, 16), ("f16", 128, 64), ("bf16", 256, 32), ("bf16", 128, 256)])
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,per", [((0, 5, 63, 64), (1, 1, 1, 1)), ((70, 0, 31), (3, 0, 2)), ((9, 60), (200, 131)), ((0,), (64,))],
                         ids=["single", "drafts", "prompts", "page"])
def test_append_writes_what_the_format_says(fmt, dim, page, src, lens, per):
    c = Cache(fmt, lens, 2, dim, page, seed=dim + page, room=[n + p for n, p in zip(lens, per)])
    g = torch.Generator().manual_seed(3)
    rows = sum(per)
    y = (torch.randn(rows, 5 * dim, generator=g) * 3).to(TYPES[src])  # columns of a wider matrix
    k, v = (y[:, i * dim:(i + 2) * dim].unflatten(1, (2, dim)) for i in (1, 3))
    yd = y.cuda()
    kd, vd = (yd[:, i * dim:(i + 2) * dim].unflatten(1, (2, dim)) for i in (1, 3))
    pool, w, pos, err = append(c, per, kd, vd)
    assert err == 0
    want, ww, wp = expected(c, per, k.float().numpy(), v.float().numpy())
    same_pool(c, pool, want)
    assert np.array_equal(w, ww) and np.array_equal(pos, wp)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_append_rows_of_any_alignment(fmt, shift):
    """A row stride and a first element that are no multiple of 16 bytes."""
    t = torch_cuda()
    c = Cache(fmt, (40,), 2, seed=5, room=[80])
    g = torch.Generator().manual_seed(6)
    y = torch.randn(37, 2 * 256 + 5, generator=g)
    yd = y.cuda()
    pool, _, _, err = append(c, (37,), *(yd[:, o:o + 256].unflatten(1, (2, 128)) for o in (shift, 256 + shift)))
    want, _, _ = expected(c, (37,), *(y[:, o:o + 256].unflatten(1, (2, 128)).numpy() for o in (shift, 256 + shift)))
    assert err == 0
    same_pool(c, pool, want)


def test_append_q8_values_of_the_whole_range():
    """Blocks of zeros, of tiny and of huge values, ties of the rounding, NaN and infinities."""
    c = Cache("q8_0", (10,), 1, seed=7, room=[80])
    rng = np.random.default_rng(8)
    x = rng.standard_normal((2, 40, 1, 128)).astype(np.float32)
    x *= np.exp2(rng.integers(-40, 40, (2, 40, 1, 4, 1))).repeat(32, -1).reshape(2, 40, 1, 128).astype(np.float32)
    x[0, 0] = 0
    x[1, 1, 0, :32] = -0.0
    x[0, 2, 0, 40] = np.nan
    x[1, 3, 0, 100] = np.inf
    x[0, 4, 0, 127] = -np.inf
    x[0, 5, 0, :32] = np.arange(32) - 15.5  # with 127: halves that round to even
    x[0, 5, 0, 31] = 127
    x[1, 6, 0, :32] = 3e38
    pool, _, _, err = append(c, (40,), *(torch.from_numpy(a).cuda() for a in x))
    want, _, _ = expected(c, (40,), x[0], x[1])
    assert err == 0
    same_pool(c, pool, want)


def test_append_without_the_slots_arrays_and_past_4_gb():
    t = torch_cuda()
    c = Cache("bf16", (60,), 8, seed=9, room=[100])
    pages = (5 << 30) // (8 * 64 * 512)
    k, v = torch.randn(33, 8, 128), torch.randn(33, 8, 128)
    want, _, _ = expected(c, (33,), k.numpy(), v.numpy())
    big = t.empty(pages, 8, 2, 64, 128, dtype=t.bfloat16, device="cuda")
    big[pages - c.pages:] = c.pool.cuda()
    small, c.table = c.pages, np.where(c.table < 0, c.table, c.table + pages - c.pages).astype(np.int32)
    c.pages = pages
    plan = c.plan(8, 33)
    plan.append(big, i32([0, 33]), i32([60]), k.cuda(), v.cuda())
    assert plan.error() == 0
    same_pool(c, big[pages - small:].cpu(), want)


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
def test_append_refuses_on_the_device_what_does_not_fit(fmt):
    """A sequence whose rows pass its slots is left alone; a page outside the pool is not written."""
    c = Cache(fmt, (60, 10), 2, seed=10, room=[64, 30])
    k, v = torch.randn(9, 2, 128), torch.randn(9, 2, 128)
    pool, w, pos, err = append(c, (5, 4), k.cuda(), v.cuda())  # 60 + 5 > 64 slots
    assert err == 4
    want, ww, wp = expected(c, (5, 4), k.numpy(), v.numpy(), skip=(0,))
    same_pool(c, pool, want)
    assert np.array_equal(w, ww) and np.array_equal(pos, wp)
    for bad in (-1, c.pages):
        table, c.table = c.table, c.table.copy()
        c.table[0, 0] = bad
        pool, w, pos, err = append(c, (4, 4), k[:8].cuda(), v[:8].cuda())
        c.table = table
        assert err == 2
        want, ww, wp = expected(c, (4, 4), k.numpy(), v.numpy(), skip=(0,))
        same_pool(c, pool, want)
        assert np.array_equal(w, ww) and np.array_equal(pos, wp)


# ------------------------------------------------------------------------------ evict
def evict(c, weight, pos, keep, sink=0, protect=None, inplace=False, pool=None):
    t = torch_cuda()
    plan = c.plan(c.kvh, 1)
    pool = c.pool.cuda() if pool is None else pool
    w, p = t.from_numpy(weight).cuda(), t.from_numpy(pos).cuda()
    wo, po = (w, p) if inplace else (t.full_like(w, -3.0), t.full_like(p, -3))
    n = t.full((c.agents,), -1, dtype=t.int32, device="cuda")
    plan.evict(pool, i32(c.lens), i32(keep), w, p, weight_out=wo, pos_out=po, len_out=n, sink=sink,
               protect_from=None if protect is None else i32(protect))
    t.cuda.synchronize()
    return pool, wo.cpu().numpy(), po.cpu().numpy(), n.tolist(), plan.error()


def check_evict(c, weight, pos, keep, sink=0, protect=None, inplace=False):
    before = c.parts()
    k0, v0 = c.values()
    pool, w, p, n, err = evict(c, weight, pos, keep, sink, protect, inplace)
    assert err == 0
    old, c.pool = c.pool, pool.cpu()
    k1, v1 = c.values()
    c.pool = old
    for a in range(c.agents):
        for g in range(c.kvh):
            m = c.lens[a]
            from_ = 1 << 30 if protect is None else protect[a]
            budget, moves = evict_ref(weight[a, g], pos[a, g], m, keep[a], sink, from_)
            assert n[a] == budget
            ww, pp = weight[a, g].copy(), pos[a, g].copy()
            kk, vv = k0[a, g].copy(), v0[a, g].copy()
            for src, dst in moves:
                ww[dst], pp[dst], kk[dst], vv[dst] = weight[a, g, src], pos[a, g, src], k0[a, g, src], v0[a, g, src]
            assert np.array_equal(w[a, g, :budget], ww[:budget], equal_nan=True) and np.array_equal(p[a, g, :budget], pp[:budget])
            # the pool: everything but the holes is untouched, slots past the budget too
            assert np.array_equal(k1[a, g], kk) and np.array_equal(v1[a, g], vv)
            if not inplace:
                assert (w[a, g, budget:] == -3.0).all() and (p[a, g, budget:] == -3).all()
    assert before.shape == c.parts().shape


def slots(c, seed=1, kind="random"):
    rng = np.random.default_rng(seed)
    shape = (c.agents, c.kvh, c.cap)
    pos = np.stack([np.stack([rng.permutation(c.cap) for _ in range(c.kvh)]) for _ in range(c.agents)]).astype(np.int32)
    w = {"random": lambda: rng.random(shape) ** 4 * 30, "equal": lambda: np.full(shape, 0.5), "few": lambda: rng.integers(0, 3, shape) - 1.0,
         "rising": lambda: np.arange(c.cap) + np.zeros(shape), "falling": lambda: -np.arange(c.cap) + np.zeros(shape),
         "odd": lambda: rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, 1.0], shape)}[kind]().astype(np.float32)
    return w, pos


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64), ("f16", 64, 16), ("bf16", 128, 64), ("f16", 256, 32), ("f16", 128, 256)])
@pytest.mark.parametrize("kind", ["random", "equal", "few", "rising", "falling", "odd"])
def test_evict_keeps_and_moves_what_the_definition_says(fmt, dim, page, kind):
    c = Cache(fmt, (333, 64, 1, 130, 700), 2, dim, page, seed=dim)
    check_evict(c, *slots(c, kind=kind), keep=[100, 63, 1, 64, 513], sink=3, protect=[300, 60, 0, 120, 650])


@pytest.mark.parametrize("keep", [0, 1, 199, 200, 201, -1, 100])
@pytest.mark.parametrize("inplace", [False, True])
def test_evict_budgets(keep, inplace):
    c = Cache("f16", (200, 199), 2, 64, 16, seed=21)
    check_evict(c, *slots(c), keep=[keep, keep], sink=2, protect=[190, 190], inplace=inplace)


def test_evict_protection_beyond_the_budget_and_none():
    c = Cache("bf16", (200,), 2, 64, 16, seed=22)
    w, p = slots(c)
    check_evict(c, w, p, keep=[50], sink=0, protect=[0])       # all protected: the lowest slots stay
    check_evict(c, w, p, keep=[50], sink=150, protect=None)
    check_evict(c, w, p, keep=[50], sink=-5, protect=[1 << 30])


@pytest.mark.parametrize("fmt,dim,page,n", [("q8_0", 128, 64, 9001), ("f16", 64, 256, 20011)])
def test_evict_long(fmt, dim, page, n):
    c = Cache(fmt, (n, 17), 1, dim, page, seed=23)
    check_evict(c, *slots(c, seed=2), keep=[n // 2 + 1, 20], sink=4, protect=[n - 500, 0])
    check_evict(c, *slots(c, seed=3, kind="few"), keep=[n // 3, 3], sink=4, protect=[n - 500, 9])


@pytest.mark.parametrize("n", [33001, 140001, 270001])
def test_evict_longer_than_the_keys_that_a_block_holds(n):
    """Clusters of two and eight blocks, and keys formed again from memory where a block's share passes
    its shared memory."""
    t = torch_cuda()
    c = Cache("f16", (n,), 1, 64, 256, seed=24)
    w, pos = slots(c, seed=4)
    keep = n * 3 // 7
    pool, wo, po, m, err = evict(c, w, pos, [keep], 4, [n - 1000])
    assert err == 0 and m == [keep]
    budget, moves = evict_ref(w[0, 0], pos[0, 0], n, keep, 4, n - 1000)
    ww, pp = w[0, 0].copy(), pos[0, 0].copy()
    src, dst = np.array(moves).T
    ww[dst], pp[dst] = w[0, 0, src], pos[0, 0, src]
    assert np.array_equal(wo[0, 0, :budget], ww[:budget]) and np.array_equal(po[0, 0, :budget], pp[:budget])
    table = torch.from_numpy(c.table[0]).long()
    want = c.pool.clone()
    want[table[dst // 256], 0, :, dst % 256] = c.pool[table[src // 256], 0, :, src % 256]
    assert torch.equal(pool.cpu().view(torch.int16), want.view(torch.int16))


def test_evict_then_attend_sees_the_kept_tokens():
    """Attention over an evicted cache equals attention over its kept tokens, in any order."""
    from kv_util import attend_ref, check_attend
    t = torch_cuda()
    c = Cache("q8_0", (300, 90), 2, seed=25)
    w, pos = slots(c)
    pool, _, _, n, err = evict(c, w, pos, [100, 64], 4, [290, 80])
    assert err == 0
    q = torch.randn(2, 4, 128).half()
    k, v = c.values()
    out = t.zeros(2, 4, 128, device="cuda")
    plan = c.plan(4, 2, 1)
    plan.attend(pool, i32([0, 1, 2]), i32(n), q.cuda(), out)
    kk, vv = np.zeros_like(k), np.zeros_like(v)
    for a in range(2):
        for g in range(2):
            b, moves = evict_ref(w[a, g], pos[a, g], c.lens[a], [100, 64][a], 4, [290, 80][a])
            gone = {d for _, d in moves}
            kept = [x for x in range(b) if x not in gone] + [s for s, _ in moves]
            kk[a, g, :b], vv[a, g, :b] = k[a, g, kept], v[a, g, kept]
    ref = attend_ref(kk, vv, [0, 1, 2], n, q.double().numpy(), 128 ** -0.5)
    check_attend(ref, out.double().cpu().numpy(), None, None, "f32", 20)


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
def test_evict_reports_bad_pages_and_lengths(fmt):
    c = Cache(fmt, (128, 70), 2, seed=26)
    w, pos = slots(c, kind="rising")
    table, c.table = c.table, c.table.copy()
    c.table[0, 1] = c.pages  # the page that the survivors are in
    pool, wo, _, n, err = evict(c, w, pos, [64, 70])
    c.table = table
    assert err == 2 and n == [64, 70] and torch.equal(pool.cpu(), c.pool)
    for bad in (-1, c.cap + 1):
        lens, c.lens = c.lens, [bad, 70]
        pool, wo, _, n, err = evict(c, w, pos, [3, 70])
        c.lens = lens
        assert err == 4 and n == [bad, 70] and torch.equal(pool.cpu(), c.pool) and (wo[0] == -3.0).all()
