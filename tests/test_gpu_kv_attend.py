"""Attention of new tokens over the paged cache (qmm_kv_attend) against a plain implementation in
64 bits.  The tolerances follow from the arithmetic (kv_util.check_attend)."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from kv_util import TYPES, Cache, attend_ref, check_attend

pytestmark = pytest.mark.gpu

SPLIT = {"q8_0": 20, "f16": 20, "bf16": 15}  # bits that the probabilities' two parts keep (2 * 11, 2 * 8; one or two for sums)


def run(c, heads, agent_rows, row_len, q, kind="f32", weight_in=None, weights=True, scale=None, plan=None, stride=0, alias=False,
        pool=None):
    """One call; returns out, lse, weight as float64 numpy and the error word."""
    t = torch_cuda()
    rows = q.shape[0]
    most = max([b - a for a, b in zip(agent_rows, agent_rows[1:])] + [1])
    plan = plan or c.plan(heads, max(1, rows), most)
    pool = c.pool.cuda() if pool is None else pool
    qd = q.cuda()
    if stride:
        wide = t.zeros(rows, heads * c.dim + stride, dtype=qd.dtype, device="cuda")
        wide[:, stride:] = qd.flatten(1)
        qd = wide[:, stride:].unflatten(1, (heads, c.dim))
    out = t.full((rows, heads, c.dim), 7.0, dtype=TYPES[kind], device="cuda")
    lse = t.full((rows, heads), 7.0, device="cuda")
    ar = t.tensor(agent_rows, dtype=t.int32, device="cuda")
    rl = t.tensor(row_len, dtype=t.int32, device="cuda")
    win = None if weight_in is None else t.from_numpy(weight_in).float().cuda()
    wout = None
    if weights:
        wout = win if alias else t.full((c.agents, c.kvh, c.cap), 0.0 if weight_in is None else -3.0, device="cuda")
    plan.attend(pool, ar, rl, qd, out, lse=lse, weight_in=win, weight_out=wout, scale=scale)
    t.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), None if wout is None else wout.double().cpu().numpy(), plan.error()


def queries(c, rows, heads, seed=1, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, heads, c.dim, generator=g) * spread).to(torch.bfloat16 if c.fmt == "bf16" else torch.float16)


def rows_of(lens, per):
    """agent_rows and row_len of a token and its drafts per sequence."""
    per = [per] * len(lens) if isinstance(per, int) else per
    ar = np.concatenate([[0], np.cumsum(per)]).tolist()
    return ar, [max(0, n - (p - 1 - j)) for n, p in zip(lens, per) for j in range(p)]


def check(c, heads, per, kind="f32", seed=1, spread=1.0, scale=None, row_len=None, **kw):
    ar, rl = rows_of(c.lens, per)
    rl = row_len or rl
    q = queries(c, len(rl), heads, seed, spread)
    win = np.random.default_rng(seed).random((c.agents, c.kvh, c.cap)).astype(np.float32)
    out, lse, w, err = run(c, heads, ar, rl, q, kind, weight_in=win, scale=scale, **kw)
    assert err == 0
    k, v = c.values()
    ref = attend_ref(k, v, ar, rl, q.double().numpy(), c.dim ** -0.5 if scale is None else scale, win)
    longest = [max([rl[r] for r in range(ar[a], ar[a + 1])] + [0]) for a in range(c.agents)]
    if not kw.get("alias"):
        for a, n in enumerate(longest):  # slots from the longest row on are not written
            assert (w[a, :, n:] == -3.0).all()
            w[a, :, n:] = ref["weight"][a, :, n:]
    check_attend(ref, out, lse, w, kind, SPLIT[c.fmt])


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64)] + [(f, d, p) for f in ("f16", "bf16") for d, p in
                         [(64, 16), (64, 32), (64, 256), (128, 16), (128, 64), (128, 256), (256, 16), (256, 128)]])
@pytest.mark.parametrize("lens,per,heads,kvh", [((1, 70, 5, 129), 1, 8, 8), ((64, 63, 65, 333), 3, 12, 2), ((700, 2), 5, 6, 1)],
                         ids=["mha", "gqa6-r3", "mqa6-r5"])
def test_attend_matches_plain(fmt, dim, page, lens, per, heads, kvh):
    check(Cache(fmt, lens, kvh, dim, page, seed=dim + page), heads, per)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
def test_attend_output_types(fmt, kind):
    check(Cache(fmt, (200, 31), 2, seed=3), 12, 2, kind)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
def test_attend_long(fmt):
    check(Cache(fmt, (9001, 3), 2, seed=4), 12, 2)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("per,heads,kvh", [(11, 12, 2), (40, 2, 2), (8, 48, 8)], ids=["66q", "40q", "48q"])
def test_attend_many_queries(fmt, per, heads, kvh):
    check(Cache(fmt, (333, 90), kvh, seed=5), heads, per)


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("f16", 128), ("bf16", 256)])
def test_attend_rows_of_any_length_and_sequences_without_rows(fmt, dim):
    """Rows of one sequence in any order of lengths, rows that see nothing, sequences without rows."""
    c = Cache(fmt, (500, 64, 10, 128), 2, dim, seed=6)
    check(c, 4, [4, 0, 2, 3], row_len=[500, 0, 17, 64, 0, 0, 65, 128, 1])


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
def test_attend_scale_stride_and_weights_in_place(fmt):
    c = Cache(fmt, (77, 130), 2, seed=7)
    check(c, 4, 2, scale=0.31)
    check(c, 4, 2, scale=-0.05)
    check(c, 4, 2, stride=24)
    check(c, 4, 2, alias=True)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
def test_attend_without_weights_has_the_same_bits(fmt):
    c = Cache(fmt, (300, 41), 2, seed=8)
    ar, rl = rows_of(c.lens, 2)
    q = queries(c, 4, 8)
    a = run(c, 8, ar, rl, q, weights=False)
    b = run(c, 8, ar, rl, q, weights=True)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1]) and a[2] is None
    ref = attend_ref(*c.values(), ar, rl, q.double().numpy(), c.dim ** -0.5)
    check_attend(ref, b[0], b[1], b[2], "f32", SPLIT[fmt])  # weight_in None counts as zeros


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("f16", 256), ("bf16", 128)])
def test_attend_peaked_scores(fmt, dim):
    """One token takes nearly everything: the others' probabilities lie far below fp16's range."""
    c = Cache(fmt, (400,), 1, dim, seed=9)
    check(c, 4, 1, spread=12.0)
    check(c, 4, 1, spread=60.0)


def test_attend_small_probabilities_add_up():
    """A sink with all but a thousandth of the softmax, and 4,000 tokens that share the rest."""
    c = Cache("f16", (4001,), 1, seed=10)
    q = torch.zeros(1, 1, 128, dtype=torch.float16)
    q[..., 0] = 8.0
    for t in range(4001):
        c.pool[c.table[0, t // 64], 0, 0, t % 64] = 0
        c.pool[c.table[0, t // 64], 0, 1, t % 64] = 1.0
    c.pool[c.table[0, 0], 0, 0, 0, 0] = 15.25 * 128 ** 0.5 / 8.0
    c.pool[c.table[0, 0], 0, 1, 0] = 0.0
    out, lse, w, err = run(c, 1, [0, 1], [4001], q)
    ref = attend_ref(*c.values(), [0, 1], [4001], q.double().numpy(), 128 ** -0.5)
    assert err == 0 and 5e-4 < ref["out"][0, 0, 0] < 2e-3
    check_attend(ref, out, lse, w, "f32", SPLIT["f16"])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_attend_what_a_row_does_not_see_has_no_effect(fmt, dim):
    """NaN and infinities in slots past the cache, in tokens that only later drafts see, and in pages
    of no sequence."""
    lens, per = (70, 33, 128), 3
    c = Cache(fmt, lens, 2, dim, 32, seed=11)
    clean = c.pool.clone()
    ar, rl = rows_of(lens, per)
    q = queries(c, len(rl), 6)
    odd = torch.tensor([float("nan"), float("inf"), float("-inf")]).to(c.pool.dtype)
    used = {int(p) for p in c.table.ravel() if p >= 0}
    for p in set(range(c.pages)) - used:
        c.pool[p] = odd[0]
    for a, n in enumerate(lens):
        for t in range(n - 2, -(-n // 32) * 32):  # from the first draft's token on
            c.pool[c.table[a, t // 32], :, :, t % 32] = odd[t % 3]
    out, lse, w, err = run(c, 6, ar, rl, q)
    assert err == 0
    first = [r for r in range(len(rl)) if r % per == 0]
    kept, c.pool = c.pool, clean
    k, v = c.values()
    ref = attend_ref(k, v, ar, rl, q.double().numpy(), dim ** -0.5)
    sub = {n: ref[n][first] for n in ("out", "lse", "mag", "big")}
    check_attend(sub, out[first], lse[first], None, "f32", SPLIT[fmt])
    # the rows that see them are not numbers
    assert not np.isfinite(out[[r for r in range(len(rl)) if r % per == 2]]).any()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_attend_infinite_value_of_a_draft(fmt):
    """One infinite element of V: infinite in that dim for the rows that see it, no effect elsewhere."""
    c = Cache(fmt, (50,), 1, 64, 64, seed=12)
    ar, rl = rows_of(c.lens, 2)
    q = queries(c, 2, 3)
    k, v = c.values()
    ref = attend_ref(k, v, ar, rl, q.double().numpy(), 64 ** -0.5)
    c.pool[c.table[0, 0], 0, 1, 49, 5] = float("inf")
    out, lse, _, err = run(c, 3, ar, rl, q)
    assert err == 0 and np.isposinf(out[1, :, 5]).all()
    out[1, :, 5] = ref["out"][1, :, 5]
    check_attend(ref, out, lse, None, "f32", SPLIT[fmt])


def test_attend_q8_scales_of_the_whole_range():
    """Scales from fp16's smallest subnormal to its largest value, zeros among them, in one block of
    a token or in all; NaN and infinite scales where a row does not look."""
    c = Cache("q8_0", (190,), 1, seed=13)
    rng = np.random.default_rng(14)
    pool = c.pool.numpy()
    vs = pool[:, :, 16896:].view(np.float16)
    vs[:] = np.exp2(rng.uniform(-24, 15.9, vs.shape)).astype(np.float16)
    vs[..., rng.integers(0, 256, 40)] = 0
    vs[:, :, :] = np.where(rng.random(vs.shape) < 0.2, np.float16(0.01), vs)
    ks = pool[:, :, 8192:8704].view(np.float16)
    ks[..., ::7] = 0
    ar, rl = rows_of(c.lens, 3)
    q = queries(c, 3, 4)
    ref = attend_ref(*c.values(), ar, rl, q.double().numpy(), 128 ** -0.5)
    out, lse, w, err = run(c, 4, ar, rl, q)
    assert err == 0
    check_attend(ref, out, lse, w, "f32", SPLIT["q8_0"])
    # (small values beside large ones: each 32-dim block of a token keeps its own accuracy, so
    # the bound above, sum p |v| per dim, holds for the small dims too)
    for t in (188, 189, 190, 191):
        pool[c.table[0, t // 64], 0, 8192:8704].view(np.float16)[4 * (t % 64):4 * (t % 64) + 4] = np.nan
        pool[c.table[0, t // 64], 0, 16896:].view(np.float16)[t % 64::64] = np.inf if t % 2 else np.nan
    out, lse, _, err = run(c, 4, ar, rl, q)
    assert err == 0
    check_attend({n: ref[n][:1] for n in ("out", "lse", "mag", "big")}, out[:1], lse[:1], None, "f32", SPLIT["q8_0"])


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64), ("f16", 128, 16), ("bf16", 64, 32), ("f16", 256, 64)])
def test_attend_rows_do_not_depend_on_the_call(fmt, dim, page):
    """A row's bits are the same alone, with fewer rows of its sequence, and in the full call."""
    c = Cache(fmt, (300, 1500, 40), 2, dim, page, seed=15)
    ar, rl = rows_of(c.lens, 3)
    q = queries(c, 9, 12)
    full = run(c, 12, ar, rl, q)
    one = run(c, 12, [0, 0, 1, 1], rl[3:4], q[3:4])  # sequence 1's first row alone
    assert np.array_equal(one[0][0], full[0][3]) and np.array_equal(one[1][0], full[1][3])
    two = run(c, 12, [0, 1, 1, 3], [rl[2]] + rl[6:8], q[[2, 6, 7]])
    assert np.array_equal(two[0], full[0][[2, 6, 7]]) and np.array_equal(two[1], full[1][[2, 6, 7]])


def test_attend_matches_the_q8_decode_attention():
    """The same pool through qmm_attn_decode, within the sum of the two tolerances."""
    from bit_weight_streaming_q4_gb300.qmm import attn_decode
    t = torch_cuda()
    c = Cache("q8_0", (700, 90), 2, seed=16)
    ar, rl = rows_of(c.lens, 3)
    q = queries(c, 6, 12)
    out, _, _, err = run(c, 12, ar, rl, q)
    old = t.empty(6, 12, 128, device="cuda")
    table = np.where(c.table < 0, 0, c.table)
    attn_decode(c.pool.cuda(), t.from_numpy(table).cuda(), t.tensor(ar, dtype=t.int32).cuda(), t.tensor(rl, dtype=t.int32).cuda(),
                q.cuda(), old, 2)
    ref = attend_ref(*c.values(), ar, rl, q.double().numpy(), 128 ** -0.5)
    assert err == 0 and (np.abs(old.double().cpu().numpy() - out) <= 3e-3 * ref["mag"] + 1e-6).all()


def test_attend_offsets_past_32_bits():
    """Pages whose bytes lie beyond 4 GB of the pool."""
    t = torch_cuda()
    c = Cache("f16", (333,), 8, seed=17, first_page=0)
    pages = (5 << 30) // (8 * 64 * 512)
    big = t.empty(pages, 8, 2, 64, 128, dtype=t.float16, device="cuda")
    big[pages - c.pages:] = c.pool.cuda()
    ar, rl = rows_of(c.lens, 1)
    q = queries(c, 1, 48)
    ref = attend_ref(*c.values(), ar, rl, q.double().numpy(), 128 ** -0.5)
    c.table = np.where(c.table < 0, c.table, c.table + pages - c.pages).astype(np.int32)
    c.pages = pages
    out, lse, w, err = run(c, 48, ar, rl, q, pool=big)
    assert err == 0
    check_attend(ref, out, lse, w, "f32", SPLIT["f16"])


def test_attend_on_another_stream_and_in_a_graph():
    t = torch_cuda()
    c = Cache("f16", (300, 60), 2, seed=18)
    ar, rl = rows_of(c.lens, 1)
    q = queries(c, 2, 8)
    want = run(c, 8, ar, rl, q)
    plan, pool, qd = c.plan(8, 2, 1), c.pool.cuda(), q.cuda()
    out, lse = t.zeros(2, 8, 128, device="cuda"), t.zeros(2, 8, device="cuda")
    w = t.zeros(2, 2, c.cap, device="cuda")
    ard, rld = t.tensor(ar, dtype=t.int32, device="cuda"), t.tensor(rl, dtype=t.int32, device="cuda")
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        plan.attend(pool, ard, rld, qd, out, lse=lse, weight_out=w)
    s.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(w.double().cpu().numpy(), want[2])
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        plan.attend(pool, ard, rld, qd, out, lse=lse, weight_in=w, weight_out=w)
    out.zero_()
    w.zero_()
    for _ in range(3):
        graph.replay()
    t.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0]) and plan.error() == 0
    assert np.allclose(w.double().cpu().numpy(), 3 * want[2], rtol=3e-7, atol=0)  # three roundings of 2^-24


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
def test_attend_reports_bad_pages_rows_and_lengths(fmt):
    c = Cache(fmt, (200, 50), 2, seed=19)
    ar, rl = rows_of(c.lens, 1)
    q = queries(c, 2, 4)
    good = run(c, 4, ar, rl, q)
    for bad_page in (-1, c.pages, 1 << 30):
        table = c.table.copy()
        c.table = c.table.copy()
        c.table[0, 1] = bad_page
        out, lse, _, err = run(c, 4, ar, rl, q)
        c.table = table
        # the page's tokens are left out; the other sequence is untouched
        assert err == 2 and np.isfinite(out).all() and np.array_equal(out[1], good[0][1])
    for bad in ([-1, 50], [c.cap + 1, 50]):
        out, lse, _, err = run(c, 4, ar, bad, q)
        assert err == 4 and (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.array_equal(out[1], good[0][1])
    # a row of no sequence; more rows than the plan allows
    out, lse, _, err = run(c, 4, [1, 1, 2], rl, q)
    assert err == 4 and (out[0] == 0).all() and np.array_equal(out[1], good[0][1])
    out, lse, _, err = run(c, 4, [0, 2, 2], [200, 200], q, plan=c.plan(4, 2, 1))
    assert err == 4 and (out == 0).all()


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("bf16", 64), ("f16", 128), ("bf16", 128), ("f16", 256), ("bf16", 256)])
@pytest.mark.parametrize("heads", [8, 9, 16, 17, 24, 25, 32, 33, 48, 49, 65, 73])
def test_attend_numbers_of_queries_around_the_tiles(fmt, dim, heads):
    check(Cache(fmt, (333, 66), 1, dim, 32 if fmt != "q8_0" else 64, seed=heads), heads, 1)


@pytest.mark.parametrize("fmt,dim,page,n", [("q8_0", 128, 64, 5003), ("f16", 64, 16, 5003), ("bf16", 256, 32, 5003), ("f16", 128, 64, 40001)])
def test_attend_more_chunks_than_a_warp_has_lanes(fmt, dim, page, n):
    check(Cache(fmt, (n, 70), 1, dim, page, seed=13), 3, 2)


@pytest.mark.parametrize("fmt,dim,page", [("f16", 64, 16), ("q8_0", 128, 64), ("bf16", 256, 32)])
def test_attend_bits_of_a_row_in_a_small_and_a_large_call(fmt, dim, page):
    """A row alone, and beside the 39 rows of another sequence: how the join is split differs."""
    c = Cache(fmt, (5003, 300), 1, dim, page, seed=14)
    q = queries(c, 40, 16)
    plan = c.plan(16, 40, 39)
    few = run(c, 16, [0, 1, 1], [5003], q[:1], plan=plan)
    many = run(c, 16, [0, 1, 40], [5003] + [300 - i for i in range(39)], q, plan=plan)
    assert few[3] == 0 and many[3] == 0
    assert np.array_equal(few[0][0], many[0][0]) and np.array_equal(few[1][0], many[1][0])
    assert np.array_equal(few[2][0], many[2][0])
