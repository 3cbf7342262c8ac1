"""Windowed attention of rows whose windows lie apart: what is between them belongs to no row, so it has no effect, and
its page table entries may hold anything.  Tolerances: test_gpu_kv_window."""
import numpy as np
import pytest
import torch

from kv_util import Cache
from test_gpu_kv_window import GEOMETRY, check_window, queries, run, window_ref

pytestmark = pytest.mark.gpu
ANYTHING = [-1, -(1 << 31), (1 << 31) - 1, "end", "nan"]  # the pool's number of pages; a page of NaN that no sequence has


def unseen_pages(c, agent_rows, row_len, window, sinks):
    """(sequence, page) of the pages that no row sees."""
    for a in range(c.agents):
        seen = np.zeros(c.cap, dtype=bool)
        for n in row_len[agent_rows[a]:agent_rows[a + 1]]:
            seen[max(0, n - window):n] = True
            seen[:min(n, sinks)] = True
        for i, s in enumerate(seen.reshape(-1, c.page)):
            if not s.any():
                yield a, i


def check_gaps(c, heads, agent_rows, row_len, window, sinks):
    q = queries(c, len(row_len), heads)
    k, v = c.values()
    ref = window_ref(k, v, agent_rows, row_len, q.double().numpy(), c.dim ** -0.5, window, sinks)
    if c.fmt == "q8_0":
        c.pool[-1, :, 8192:8704] = c.pool[-1, :, 16896:] = 0x7F
    else:
        c.pool[-1] = float("nan")
    changed = 0
    for j, (a, i) in enumerate(unseen_pages(c, agent_rows, row_len, window, sinks)):
        other = ANYTHING[j % len(ANYTHING)]
        c.table[a, i] = {"end": c.pages, "nan": c.pages - 1}.get(other, other)
        changed += 1
    out, lse, err = run(c, heads, agent_rows, row_len, q, window, sinks)
    assert err == 0 and changed > 0
    check_window(ref, out, lse, c.fmt, "f32")


@pytest.mark.parametrize("fmt,dim,page", GEOMETRY)
@pytest.mark.parametrize("sinks", [0, 5, 100])
def test_two_rows_apart(fmt, dim, page, sinks):
    c = Cache(fmt, [2000, 900], 2, dim, page, seed=50)
    check_gaps(c, 6, [0, 2, 5], [100, 2000, 900, 70, 450], 64, sinks)
    c = Cache(fmt, [2000, 900], 2, dim, page, seed=50)
    check_gaps(c, 6, [0, 2, 5], [1990, 0, 20, 900, 300], 9, sinks)


@pytest.mark.parametrize("fmt,dim,page", GEOMETRY)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (150, 0)])
def test_many_rows_apart(fmt, dim, page, window, sinks):
    """Items of a prompt's size whose rows lie anywhere, in no order."""
    rng = np.random.default_rng(51)
    c = Cache(fmt, [9000, 5000], 1, dim, page, seed=51)
    rl = rng.choice(9001, 30).tolist() + rng.choice(5001, 25).tolist()
    rl[4], rl[9] = 9000, 0
    check_gaps(c, 12, [0, 30, 55], rl, window, sinks)


@pytest.mark.parametrize("fmt,dim,page", GEOMETRY)
def test_rows_apart_in_chunks(fmt, dim, page):
    c = Cache(fmt, [30001], 1, dim, page, seed=52)
    plan = c.plan(4, 3, 3)
    assert plan._bytes("qmm_kv_window_workspace_bytes", 3, 5000, 40) > 0
    check_gaps(c, 4, [0, 3], [6000, 30001, 14000], 5000, 40)


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64), ("f16", 64, 16), ("f16", 128, 64), ("bf16", 256, 32)])
@pytest.mark.parametrize("rows", [3, 40])
def test_gaps_after_values_that_are_not_finite(fmt, dim, page, rows):
    """Sequences with V all NaN, among those with gaps: what a block has held of the one does not reach the other."""
    agents, heads = 160, 4
    c = Cache(fmt, [700] * agents, 1, dim, page, seed=53)
    for a in range(0, agents, 2):
        for pg in c.table[a]:
            if fmt == "q8_0":
                c.pool[pg].view(torch.float16)[:, 8448:] = float("nan")
            else:
                c.pool[pg, :, 1] = float("nan")
    ar = [rows * a for a in range(agents + 1)]
    rl = [n for _ in range(agents) for n in ([50, 700] + [360 + j for j in range(rows - 2)])]
    q = queries(c, len(rl), heads)
    k, v = c.values()
    odd = [r for r in range(len(rl)) if (r // rows) % 2]
    ref = window_ref(k, np.nan_to_num(v), ar, rl, q.double().numpy(), dim ** -0.5, 30, 2)
    for a, i in unseen_pages(c, ar, rl, 30, 2):
        c.table[a, i] = c.pages
    out, lse, err = run(c, heads, ar, rl, q, 30, 2)
    assert err == 0
    check_window({n: x[odd] for n, x in ref.items()}, out[odd], lse[odd], fmt, "f32")
    assert np.isnan(np.delete(out, odd, 0)).all()
