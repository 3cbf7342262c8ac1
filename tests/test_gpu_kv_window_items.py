"""Attention with a sliding window where blocks take many items in turn, of uneven lengths, and where sequences are cut into
chunks: rows picked from large calls, against 64-bit sums on the GPU.  Tolerances: test_gpu_kv_window."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from kv_util import Cache, score_error
from test_gpu_kv_window import HALF, PRODUCT, queries, rows_of

pytestmark = pytest.mark.gpu


def large(fmt, dim, page, lens, per, heads, kvh, window, sinks, seed, picks=200):
    t = torch_cuda()
    c = Cache(fmt, lens, kvh, dim, page, seed=seed)
    ar, rl = rows_of(c.lens, per)
    q = queries(c, len(rl), heads, seed)
    plan = c.plan(heads, len(rl), max(b - a for a, b in zip(ar, ar[1:])))
    out = t.full((len(rl), heads, dim), 7.0, device="cuda")
    lse = t.full((len(rl), heads), 7.0, device="cuda")
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    args = (c.pool.cuda(), i32(ar), i32(rl), q.cuda(), out)
    for _ in range(3):  # (the same bits each time)
        plan.attend_window(*args, window=window, sinks=sinks, lse=lse)
        now = out.clone()
        plan.attend_window(*args, window=window, sinks=sinks, lse=lse)
        assert t.equal(now, out)
    assert plan.error() == 0
    part = torch.from_numpy(c.parts()).cuda()  # [pages][kv_heads][2][page][D]
    rng = np.random.default_rng(seed)
    rows = sorted(set(rng.integers(0, len(rl), picks).tolist()) | {0, len(rl) - 1})
    worst = 0.0
    for r in rows:
        a = int(np.searchsorted(ar, r, side="right")) - 1
        n, h = rl[r], int(rng.integers(0, heads))
        if n == 0:
            assert bool((out[r] == 0).all())
            continue
        slot = torch.arange(n, device="cuda")
        if window:
            slot = slot[(slot >= n - window) | (slot < sinks)]
        pg = torch.from_numpy(c.table[a]).cuda().long()[slot // page]
        kk, vv = part[pg, h // (heads // kvh), 0, slot % page], part[pg, h // (heads // kvh), 1, slot % page]
        qq = q[r, h].double().cuda()
        x = kk @ qq * dim ** -0.5
        p = torch.softmax(x, 0)
        want, mag = p @ vv, p @ vv.abs()
        big = float((kk.abs() @ qq.abs()).max() * dim ** -0.5 + x.abs().max())
        tol = mag * (4 * score_error(big) + PRODUCT[fmt]) * 1.001 + float(vv.abs().max()) * len(slot) * 2.0 ** -34 + HALF["f32"] * want.abs() + 2.0 ** -25
        worst = max(worst, float(((out[r, h].double() - want).abs() / tol).max()))
        assert abs(float(lse[r, h]) - float(torch.logsumexp(x, 0))) <= 2 * score_error(big) + 2.0 ** -22 * abs(float(lse[r, h]))
    assert worst <= 1, worst


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64), ("f16", 64, 16), ("f16", 128, 64), ("bf16", 128, 128), ("bf16", 256, 32)])
@pytest.mark.parametrize("window,sinks", [(300, 4), (None, 0)])
def test_many_sequences(fmt, dim, page, window, sinks):
    """Decode steps of 150 sequences, lengths 0 to 900, one to four rows: several items a block."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 900, 150).tolist()
    large(fmt, dim, page, lens, rng.integers(0, 5, 150).tolist(), 12, 4, window, sinks, 31)


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64), ("f16", 64, 16), ("f16", 128, 64), ("bf16", 128, 16), ("f16", 256, 256)])
@pytest.mark.parametrize("window,sinks", [(257, 130), (None, 0)])
def test_many_prompts(fmt, dim, page, window, sinks):
    """Prompts of uneven lengths, tiles of queries that end inside a row's heads, one and two tiles an item."""
    rng = np.random.default_rng(2)
    per = [1, 700, 43, 22, 300, 0, 129, 513, 2, 600]
    lens = [p + int(rng.integers(0, 400)) for p in per]
    large(fmt, dim, page, lens, per, 30, 5, window, sinks, 32)


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("bf16", 128), ("f16", 256)])
@pytest.mark.parametrize("rows", [2, 40])
def test_chunks(fmt, dim, rows):
    """One long sequence and an unused one: tokens in chunks, joined; few KV heads, windows that begin inside a chunk."""
    for window, sinks in ((None, 0), (7001, 300), (12000, 1)):
        large(fmt, dim, 64, [30001, 0], [rows, 0], 6, 1, window, sinks, 33, picks=20)


def test_bad_lengths_where_tokens_are_cut_into_chunks():
    """A plan of chunks (one long sequence, few items): a sequence whose only row is out of range, rows of no sequence."""
    t = torch_cuda()
    c = Cache("f16", [20000, 300], 1, 128, 64, seed=34)
    plan = c.plan(4, 4, 2)
    assert plan._bytes("qmm_kv_window_workspace_bytes", 4, plan.cap, 0) > 0
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    q = queries(c, 4, 4).cuda()
    pool = c.pool.cuda()
    want = None
    for rows, lens, bad in (([0, 2, 4], [19999, 20000, 299, 300], []), ([0, 2, 3], [19999, 20000, -1, 300], [2, 3]),
                            ([0, 2, 3], [19999, 20000, c.cap + 1, 0], [2, 3]), ([0, 2, 1], [19999, 20000, 299, 300], [0, 1, 2, 3])):
        plan = c.plan(4, 4, 2)
        out, lse = t.full((4, 4, 128), 7.0, device="cuda"), t.full((4, 4), 7.0, device="cuda")
        plan.attend_window(pool, i32(rows), i32(lens), q, out, window=None, lse=lse)
        assert plan.error() == (4 if bad else 0)
        want = out.clone() if want is None else want
        for r in range(4):
            if r in bad:
                assert bool((out[r] == 0).all()) and bool((lse[r] == -float("inf")).all())
            else:
                assert t.equal(out[r], want[r])


@pytest.mark.parametrize("fmt,dim,page", [("f16", 64, 16), ("q8_0", 128, 64)])
def test_more_sequences_than_threads(fmt, dim, page):
    rng = np.random.default_rng(3)
    large(fmt, dim, page, rng.integers(0, 130, 950).tolist(), rng.integers(0, 3, 950).tolist(), 4, 2, 60, 2, 35)


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("bf16", 64), ("f16", 256)])
def test_order_of_sequences_changes_no_bits(fmt, dim):
    """320 items and more: rows of a sequence in any order of lengths, alone, among others, and beside a sequence with
    too many rows, one with a bad length and rows of none."""
    t = torch_cuda()
    rng = np.random.default_rng(4)
    lens = rng.integers(3, 700, 40).tolist()
    c = Cache(fmt, lens, 8, dim, 64, seed=36)
    pool = c.pool.cuda()
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    row_len = np.array([[int(x) for x in rng.integers(1, n + 1, 3)] for n in lens])  # three rows each
    q = queries(c, 123, 16).cuda()

    def call(agent_rows, lengths, rows):
        plan = c.plan(16, 123, 3)
        out, lse = t.full((rows, 16, dim), 7.0, device="cuda"), t.full((rows, 16), 7.0, device="cuda")
        plan.attend_window(pool, i32(agent_rows), i32(lengths), q[:rows], out, window=200, sinks=3, lse=lse)
        return out, lse, plan.error()

    every = [3 * a for a in range(41)]
    out, lse, err = call(every, row_len.reshape(-1).tolist(), 120)
    assert err == 0 and bool(t.isfinite(lse).all())
    for a in (0, 17, 39):  # alone, its rows where they were
        o, s, err = call([3 * a if b <= a else 3 * a + 3 for b in range(41)], row_len.reshape(-1).tolist(), 120)
        assert err == 4  # (the other rows are no sequence's)
        assert t.equal(o[3 * a:3 * a + 3], out[3 * a:3 * a + 3]) and t.equal(s[3 * a:3 * a + 3], lse[3 * a:3 * a + 3])
        assert bool((o[:3 * a] == 0).all()) and bool((o[3 * a + 3:] == 0).all())
    # sequence 5 loses its rows to sequence 4, which then has six; a row of sequence 9 is longer than the table; three rows are no sequence's
    bad = every.copy()
    bad[5] = 18
    lengths = row_len.reshape(-1).tolist() + [5, 5, 5]
    lengths[28] = c.cap + 1
    o, s, err = call(bad, lengths, 123)
    assert err == 4
    for r in range(123):
        if 12 <= r < 18 or r == 28 or r >= 120:
            assert bool((o[r] == 0).all()) and bool((s[r] == -float("inf")).all())
        else:
            assert t.equal(o[r], out[r]) and t.equal(s[r], lse[r]), r


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("f16", 128), ("bf16", 256)])
@pytest.mark.parametrize("agents,rows", [(80, 2), (950, 1), (12, 400)])
def test_items_without_tokens(fmt, dim, agents, rows):
    """Blocks whose items have no token in turn, between others: rows of length 0 (whole sequences, or runs of rows)."""
    t = torch_cuda()
    rng = np.random.default_rng(5)
    kvh, heads, cap = 4, 8, 128
    c = Cache(fmt, [cap] * agents, kvh, dim, 64, seed=37)
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    n = agents * rows
    ar = [rows * a for a in range(agents + 1)]
    lens = rng.integers(1, cap + 1, (agents, rows))
    q = queries(c, n, heads).cuda()
    pool = c.pool.cuda()

    def call(lengths):
        plan = c.plan(heads, n, rows)
        out, lse = t.full((n, heads, dim), 7.0, device="cuda"), t.full((n, heads), 7.0, device="cuda")
        plan.attend_window(pool, i32(ar), i32(lengths.reshape(-1).tolist()), q, out, window=100, sinks=3, lse=lse)
        assert plan.error() == 0
        return out, lse

    out, lse = call(lens)
    for empty in (rng.random(agents) < 0.5, rng.random(agents) < 0.95, np.arange(agents) % 2 == 0, np.arange(agents) >= agents // 2):
        some = lens.copy()
        if rows > 2:  # runs of rows
            for a in range(agents):
                at = int(rng.integers(0, rows))
                some[a, :at] = 0 if empty[a] else some[a, :at]
                some[a, at:] = some[a, at:] if empty[a] else 0
        else:
            some[empty] = 0
        o, s = call(some)
        none = torch.from_numpy(some.reshape(-1) == 0).cuda()
        assert bool((o[none] == 0).all()) and bool((s[none] == -float("inf")).all())
        assert t.equal(o[~none], out[~none]) and t.equal(s[~none], lse[~none])
