"""Attention with a sliding window over the paged cache (qmm_kv_attend_window) against a plain
implementation in 64 bits.  Tolerances, per output: a probability's relative error is at most twice the
score's on either side of the division (4 errors in all, kv_util.score_error); the product with V takes it
rounded to the pool's 16 bits, at most half a step off (fp16 2^-11, bf16 2^-8), and a q8_0 pool's V as two fp16
parts (together off by 2^-25, half a step of fp16's smallest numbers, at most); an fp16 probability below the normal range, kept times 2^9 relative to a
reference of the row, is off by 2^-25 * 2^-9 of the row's largest at most; the result is rounded once (half a step)."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from kv_util import TYPES, Cache, score_error

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
PRODUCT = {"q8_0": 2.0 ** -11, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def window_ref(k, v, agent_rows, row_len, q, scale, window, sinks, hidden=None):
    """Rows in 64 bits: out, lse, sum p |v|, score magnitudes, and max |v| times the tokens seen."""
    k, v, q = (torch.from_numpy(np.ascontiguousarray(x)) for x in (k, v, q))
    rows, heads, dim = q.shape
    agents, kvh = k.shape[:2]
    grp = heads // kvh
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((rows, heads), -torch.inf, dtype=torch.float64)
    big, small = torch.zeros(rows, heads, dtype=torch.float64), torch.zeros(rows, heads, 1, dtype=torch.float64)
    for a in range(agents):
        for r in range(agent_rows[a], agent_rows[a + 1]):
            n = row_len[r]
            t = [i for i in range(n) if (i >= n - window or i < sinks) and not (hidden and hidden(a, i))]
            if not t:
                continue
            for g in range(kvh):
                h = slice(g * grp, (g + 1) * grp)
                kk, vv = k[a, g, t], v[a, g, t]
                x = q[r, h] @ kk.T * scale
                p = torch.softmax(x, -1)
                out[r, h], mag[r, h], lse[r, h] = p @ vv, p @ vv.abs(), torch.logsumexp(x, -1)
                big[r, h] = (q[r, h].abs() @ kk.abs().T).amax(-1) * abs(scale) + x.abs().amax(-1)
                small[r, h] = float(vv.abs().max()) * len(t)
    return {n: x.numpy() for n, x in dict(out=out, mag=mag, lse=lse, big=big, small=small).items()}


def tolerance(ref, fmt, kind):
    err = score_error(ref["big"])[..., None]
    tiny = ref["small"] * (0 if fmt == "bf16" else 2.0 ** -34) + (2.0 ** -25 if fmt == "q8_0" else 0)
    return ref["mag"] * (4 * err + PRODUCT[fmt]) * 1.001 + tiny + HALF[kind] * np.abs(ref["out"]) * 1.001 + (2.0 ** -25 if kind == "f16" else 1e-30)


def check_window(ref, out, lse, fmt, kind):
    tol = tolerance(ref, fmt, kind)
    diff = np.abs(out - ref["out"])
    assert np.isfinite(out).all()
    assert (diff <= tol).all(), f"out: worst {np.max(diff / tol):.3f} of the tolerance"
    seen = np.isfinite(ref["lse"])
    assert np.array_equal(np.isneginf(lse), ~seen)
    lt = 2 * score_error(ref["big"][seen]) + 2.0 ** -22 * np.abs(ref["lse"][seen])
    assert (np.abs(lse[seen] - ref["lse"][seen]) <= lt).all()


def queries(c, rows, heads, seed=1, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, heads, c.dim, generator=g) * spread).to(torch.bfloat16 if c.fmt == "bf16" else torch.float16)


def run(c, heads, agent_rows, row_len, q, window, sinks, kind="f32", scale=None, plan=None, stride=0, pool=None):
    t = torch_cuda()
    rows = q.shape[0]
    plan = plan or c.plan(heads, max(1, rows), max([b - a for a, b in zip(agent_rows, agent_rows[1:])] + [1]))
    qd = q.cuda()
    if stride:
        wide = t.zeros(rows, heads * c.dim + stride, dtype=qd.dtype, device="cuda")
        wide[:, stride:] = qd.flatten(1)
        qd = wide[:, stride:].unflatten(1, (heads, c.dim))
    out = t.full((rows, heads, c.dim), 7.0, dtype=TYPES[kind], device="cuda")
    lse = t.full((rows, heads), 7.0, device="cuda")
    plan.attend_window(c.pool.cuda() if pool is None else pool, t.tensor(agent_rows, dtype=t.int32, device="cuda"),
                       t.tensor(row_len, dtype=t.int32, device="cuda"), qd, out, window=window, sinks=sinks, lse=lse, scale=scale)
    t.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), plan.error()


def rows_of(lens, per):
    per = [per] * len(lens) if isinstance(per, int) else per
    ar = np.concatenate([[0], np.cumsum(per)]).tolist()
    return ar, [max(0, n - (p - 1 - j)) for n, p in zip(lens, per) for j in range(p)]


def check(c, heads, per, window, sinks, kind="f32", seed=1, spread=1.0, scale=None, row_len=None, **kw):
    ar, rl = rows_of(c.lens, per)
    rl = row_len or rl
    q = queries(c, len(rl), heads, seed, spread)
    out, lse, err = run(c, heads, ar, rl, q, window, sinks, kind, scale, **kw)
    assert err == 0
    k, v = c.values()
    ref = window_ref(k, v, ar, rl, q.double().numpy(), c.dim ** -0.5 if scale is None else scale, window or 1 << 30, sinks)
    check_window(ref, out, lse, c.fmt, kind)
    return out, lse


GEOMETRY = [("q8_0", 128, 64), ("f16", 64, 16), ("f16", 128, 16), ("f16", 128, 256), ("f16", 256, 32), ("bf16", 64, 128), ("bf16", 128, 64),
            ("bf16", 256, 64)]


@pytest.mark.parametrize("fmt,dim,page", GEOMETRY)
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (100, 0), (128, 129), (None, 0)])
def test_decode_lengths(fmt, dim, page, window, sinks):
    c = Cache(fmt, [1, 0, 63, 64, 65, 127, 128, 129, 257, 500], 2, dim, page, seed=3)
    check(c, 6, 1, window, sinks)


@pytest.mark.parametrize("fmt,dim,page", GEOMETRY)
@pytest.mark.parametrize("window,sinks", [(64, 4), (None, 0)])
def test_drafts(fmt, dim, page, window, sinks):
    c = Cache(fmt, [2, 300, 129], 2, dim, page, seed=4)  # (the first sequence's first row sees nothing)
    check(c, 12, [3, 8, 5], window, sinks, kind="bf16" if fmt == "bf16" else "f16")


@pytest.mark.parametrize("fmt,dim,page", GEOMETRY)
@pytest.mark.parametrize("window,sinks", [(37, 5), (200, 0), (None, 0)])
def test_prompts(fmt, dim, page, window, sinks):
    c = Cache(fmt, [171, 90, 333], 2, dim, page, seed=5)
    check(c, 8, [171, 1, 100], window, sinks)


@pytest.mark.parametrize("heads,kvh", [(1, 1), (3, 3), (7, 1), (32, 2), (130, 1)])
@pytest.mark.parametrize("rows", [1, 50])
def test_groups(heads, kvh, rows):
    c = Cache("f16", [140, 61], kvh, 128, 32, seed=6)
    check(c, heads, [rows, min(rows, 3)], 33, 2)


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("bf16", 128), ("f16", 256)])
def test_long(fmt, dim):
    c = Cache(fmt, [20001, 9000], 1, dim, 64, seed=7)
    check(c, 4, 2, None, 0)
    check(c, 4, 2, 4097, 130)


@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
def test_rows_of_any_length(fmt):
    """Rows that see less than the ones before them, nothing, or everything, in no order."""
    rng = np.random.default_rng(8)
    c = Cache(fmt, [700, 400], 2, 128, 64, seed=8)
    rl = rng.integers(0, 700, 90).tolist() + rng.integers(0, 400, 40).tolist()
    rl[3], rl[77], rl[100] = 700, 0, 400
    check(c, 6, [90, 40], 50, 70, row_len=rl)


@pytest.mark.parametrize("spread,scale", [(30.0, None), (1.0, -0.3), (1.0, 0.0), (40.0, 3.0), (1000.0, 100.0)])
def test_scales(spread, scale):
    """Steep and flat distributions: references that move, a negative scale, scores past 2^22."""
    c = Cache("f16", [400, 300], 2, 128, 64, seed=9)
    check(c, 4, [40, 3], 333, 1, spread=spread, scale=scale)


def test_rising_scores():
    """Each tile's largest score is far above the one before: every tile moves the reference."""
    c = Cache("f16", [1000], 1, 128, 64, seed=10)
    p = c.pool.float()
    for i, pg in enumerate(c.table[0]):
        p[pg, :, 0] *= 1 + i
    c.pool = p.half()
    check(c, 4, 30, None, 0, spread=4.0)


@pytest.mark.parametrize("fmt,dim", [("f16", 64), ("f16", 128), ("bf16", 128), ("bf16", 256), ("q8_0", 128)])
@pytest.mark.parametrize("rows", [3, 60])
def test_unseen_slots_have_no_effect(fmt, dim, rows):
    """NaN and infinity in slots past the rows, before the window, and in between rows."""
    c = Cache(fmt, [350], 2, dim, 64, seed=11)
    ar, rl = rows_of(c.lens, rows)
    q = queries(c, rows, 4)
    k, v = c.values()
    ref = window_ref(k, v, ar, rl, q.double().numpy(), dim ** -0.5, 100, 5)
    rl_min = min(rl)
    pool = c.pool.clone()
    # slots that no row sees: all NaN or infinity
    unseen = list(range(5, max(0, rl_min - 100))) + list(range(350, c.cap))
    for t in unseen:
        pg, s = c.table[0][t // 64], t % 64
        if fmt == "q8_0":
            half = pool[pg].view(torch.float16)
            half[:, 4096 + s * 4:4096 + s * 4 + 4] = float("nan")
            half[:, 8448 + s:8704:64] = float("inf") if t % 2 else float("nan")
        else:
            pool[pg, :, :, s] = float("inf") if t % 2 else float("nan")
    out, lse, err = run(c, 4, ar, rl, q, 100, 5, pool=pool.cuda())
    assert err == 0
    check_window(ref, out, lse, fmt, "f32")
    # a slot that only the last row sees, and one that only the first row sees (of its window)
    for t, who in ((349, lambda r: rl[r] > 349), (rl[0] - 100, lambda r: rl[r] - 100 <= rl[0] - 100)):
        if t < 5:
            continue
        bad = pool.clone()
        pg, s = c.table[0][t // 64], t % 64
        if fmt == "q8_0":
            bad[pg].view(torch.float16)[:, 8448 + s] = float("inf")
        else:
            bad[pg, :, 1, s, 3] = float("inf")
        out, lse, err = run(c, 4, ar, rl, q, 100, 5, pool=bad.cuda())
        assert err == 0
        dims = slice(0, 32) if fmt == "q8_0" else slice(3, 4)
        tol = tolerance(ref, fmt, "f32")
        for r in range(rows):
            good = np.abs(out[r] - ref["out"][r]) <= tol[r]
            if who(r):
                assert not np.isfinite(out[r][:, dims]).any()
                good[:, dims] = True
            assert good.all(), (t, r)


def test_nan_scores():
    c = Cache("f16", [200], 1, 128, 64, seed=12)
    pg, s = c.table[0][150 // 64], 150 % 64
    c.pool[pg, 0, 0, s, 0] = float("nan")
    ar, rl = rows_of(c.lens, 100)  # rows of lengths 101 .. 200
    q = queries(c, 100, 2)
    out, lse, err = run(c, 2, ar, rl, q, 20, 0)
    sees = np.array([151 <= n <= 170 for n in rl])
    assert err == 0
    assert np.isnan(out[sees]).all() and np.isnan(lse[sees]).all()
    assert np.isfinite(out[~sees]).all() and np.isfinite(lse[~sees]).all()


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
@pytest.mark.parametrize("rows", [2, 150])
def test_pages_outside_the_pool(fmt, rows):
    c = Cache(fmt, [400], 2, 128, 64, seed=13)
    ar, rl = rows_of(c.lens, rows)
    q = queries(c, rows, 4)
    k, v = c.values()
    c.table[0][4] = c.pages if fmt == "q8_0" else -1
    out, lse, err = run(c, 4, ar, rl, q, 300, 0)
    assert err == 2
    ref = window_ref(k, v, ar, rl, q.double().numpy(), 128 ** -0.5, 300, 0, hidden=lambda a, t: t // 64 == 4)
    check_window(ref, out, lse, fmt, "f32")
    # entries of pages that no row sees hold anything
    c = Cache(fmt, [400], 2, 128, 64, seed=13)
    c.table[0][1] = -5
    _, rl = rows_of(c.lens, min(rows, 20))
    out, lse, err = run(c, 4, [0, len(rl)], rl, q[:len(rl)], 200, 40)
    assert err == 0


def test_bad_rows():
    """Lengths and sequences out of range: error word 4, rows that see nothing; the others as they are."""
    c = Cache("f16", [100, 120, 90], 2, 128, 64, seed=14)
    q = queries(c, 9, 4)
    good = [98, 99, 100, 118, 119, 120, 88, 89, 90]
    want, wlse, err = run(c, 4, [0, 3, 6, 9], good, q, 50, 2)
    assert err == 0
    for bad in (-1, c.cap + 1):
        rl = list(good)
        rl[4] = bad
        out, lse, err = run(c, 4, [0, 3, 6, 9], rl, q, 50, 2)
        keep = np.arange(9) != 4
        assert err == 4 and (out[4] == 0).all() and np.isneginf(lse[4]).all()
        assert np.array_equal(out[keep], want[keep]) and np.array_equal(lse[keep], wlse[keep])
    # rows of no sequence, before and behind
    plan = c.plan(4, 9, 3)
    out, lse, err = run(c, 4, [1, 3, 6, 8], good, q, 50, 2, plan=plan)
    none = np.isin(np.arange(9), [0, 8])
    assert err == 4 and (out[none] == 0).all() and np.isneginf(lse[none]).all()
    assert np.array_equal(out[~none], want[~none])
    # a sequence with too many rows
    plan = c.plan(4, 9, 3)
    out, lse, err = run(c, 4, [0, 3, 7, 9], good, q, 50, 2, plan=plan)
    assert err == 4 and (out[3:7] == 0).all() and np.array_equal(out[:3], want[:3]) and np.array_equal(out[7:], want[7:])
    # agent_rows that falls
    plan = c.plan(4, 9, 9)
    out, lse, err = run(c, 4, [0, 6, 3, 9], good, q, 50, 2, plan=plan)
    assert err == 4 and (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 128), ("bf16", 64), ("f16", 256)])
@pytest.mark.parametrize("most", [8, 200])
def test_bits_do_not_depend_on_company(fmt, dim, most):
    """A row alone and among others of its sequence, and of other sequences, under the same plan."""
    c = Cache(fmt, [900, 300, 77], 2, dim, 64, seed=15)
    plan = c.plan(12, 3 * most, most)
    per = [min(most, 8), min(most, 150), 5]
    ar, rl = rows_of(c.lens, per)
    q = queries(c, len(rl), 12)
    out, lse, err = run(c, 12, ar, rl, q, 130, 9, plan=plan)
    assert err == 0
    for r in (0, 3, per[0], per[0] + per[1] - 1, len(rl) - 1):
        a = next(i for i in range(3) if ar[i] <= r < ar[i + 1])
        one, l1, err = run(c, 12, [0] * (a + 1) + [1] * (3 - a), [rl[r]], q[r:r + 1], 130, 9, plan=plan)
        assert err == 0
        assert np.array_equal(one[0], out[r]) and np.array_equal(l1[0], lse[r]), r


def test_strides_and_types():
    c = Cache("bf16", [200, 133], 2, 128, 32, seed=16)
    for kind in ("f32", "f16", "bf16"):
        check(c, 4, [20, 2], 77, 3, kind=kind, stride=24)


def test_far_pages():
    """Pages whose bytes lie past 2^32."""
    t = torch_cuda()
    kvh, dim, page = 8, 128, 64
    pages = 34000  # 4.4 GB
    c = Cache("f16", [300], kvh, dim, page, seed=17)
    pool = t.zeros(pages, kvh, 2, page, dim, dtype=t.float16, device="cuda")
    far = [33999, 33001, 32999, 33500, 33333]
    for i, pg in enumerate(far):
        pool[pg] = c.pool[c.table[0][i]].cuda()
    ar, rl = rows_of(c.lens, 4)
    q = queries(c, 4, 16)
    k, v = c.values()
    c.table[0] = far
    c.pages = pages
    out, lse, err = run(c, 16, ar, rl, q, 200, 4, pool=pool)
    assert err == 0
    check_window(window_ref(k, v, ar, rl, q.double().numpy(), dim ** -0.5, 200, 4), out, lse, "f16", "f32")


def test_streams_and_graphs():
    """Two streams with plans of their own, and a captured call replayed with new rows in its buffers."""
    t = torch_cuda()
    c = Cache("q8_0", [3000, 2500], 2, 128, 64, seed=18)
    ar, rl = rows_of(c.lens, 3)
    q = [queries(c, 6, 12, seed=s) for s in (1, 2)]
    want = [run(c, 12, ar, rl, x, 1000, 4) for x in q]
    pool = c.pool.cuda()
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    plans, streams = [c.plan(12, 6, 3) for _ in q], [t.cuda.Stream() for _ in q]
    qd, outs = [x.cuda() for x in q], [t.empty(6, 12, 128, device="cuda") for _ in q]
    a, r = i32(ar), i32(rl)
    t.cuda.synchronize()
    for _ in range(20):
        for p, s, x, o in zip(plans, streams, qd, outs):
            p.attend_window(pool, a, r, x, o, window=1000, sinks=4, stream=s.cuda_stream)
    t.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.double().cpu().numpy(), w[0])
    plan, buf, o = plans[0], qd[0].clone(), outs[0]
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        plan.attend_window(pool, a, r, buf, o, window=1000, sinks=4)
    for x, w in zip(qd, want):
        buf.copy_(x)
        o.fill_(3)
        g.replay()
        t.cuda.synchronize()
        assert np.array_equal(o.double().cpu().numpy(), w[0])
    assert all(p.error() == 0 for p in plans)


def test_agrees_with_attend_where_the_window_takes_all():
    t = torch_cuda()
    c = Cache("q8_0", [1500, 40], 8, 128, 64, seed=19)
    ar, rl = rows_of(c.lens, 3)
    q = queries(c, 6, 48)
    out, lse, err = run(c, 48, ar, rl, q, None, 0)
    plan = c.plan(48, 6, 3)
    o, ls = t.empty(6, 48, 128, device="cuda"), t.empty(6, 48, device="cuda")
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    plan.attend(c.pool.cuda(), i32(ar), i32(rl), q.cuda(), o, lse=ls)
    # (both within their tolerances of the same numbers)
    k, v = c.values()
    ref = window_ref(k, v, ar, rl, q.double().numpy(), 128 ** -0.5, 1 << 30, 0)
    assert err == 0 and plan.error() == 0
    assert (np.abs(out - o.double().cpu().numpy()) <= 2 * tolerance(ref, "q8_0", "f32")).all()
    assert np.abs(lse - ls.double().cpu().numpy()).max() <= 4 * score_error(ref["big"].max()) + 1e-5


def test_no_rows():
    t = torch_cuda()
    c = Cache("f16", [10], 1, 64, 16, seed=20)
    q = t.empty(0, 2, 64, dtype=t.float16, device="cuda")
    c.plan(2, 4).attend_window(c.pool.cuda(), t.zeros(2, dtype=t.int32, device="cuda"), t.empty(0, dtype=t.int32, device="cuda"), q,
                               t.empty_like(q), window=4)
    t.cuda.synchronize()
