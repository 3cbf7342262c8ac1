"""Attention calls whose agent_rows falls somewhere: refused as a whole, whatever row_len holds, and
nothing of an earlier call's workspace shows."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from kv_util import Cache
from test_gpu_kv_attend import queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("f16", 128), ("bf16", 256)])
@pytest.mark.parametrize("agent_rows", [[0, 100, 2, 4], [0, 3, 1, 4], [4, 0, 2, 4], [0, 4, 0, 4], [0, 2, 4, -1], [-3, -5, 2, 4], [0, 4, 2, 2]])
@pytest.mark.parametrize("row_len", [[200, 199, 50, 60], [1 << 30, 200, 1 << 30, 1 << 30], [-1, -(1 << 31), 7, (1 << 31) - 1]])
def test_rows_that_fall(fmt, dim, agent_rows, row_len):
    torch_cuda()
    c = Cache(fmt, (200, 50, 60), 2, dim, seed=80)
    q = queries(c, 4, 4)
    plan = c.plan(4, 4, 4)
    pool = c.pool.cuda()
    good = run(c, 4, [0, 2, 3, 4], [199, 200, 50, 60], q, plan=plan, pool=pool)
    assert good[3] == 0 and (good[0] != 0).all()
    win = np.ones((c.agents, c.kvh, c.cap), np.float32)
    out, lse, w, err = run(c, 4, agent_rows, row_len, q, plan=plan, pool=pool, weight_in=win)
    assert err == 4 and (out == 0).all() and np.isneginf(lse).all() and (w == -3.0).all()
    plan.error_word.zero_()
    again = run(c, 4, [0, 2, 3, 4], [199, 200, 50, 60], q, plan=plan, pool=pool)
    assert again[3] == 0 and all(np.array_equal(a, b) for a, b in zip(again[:3], good[:3]))


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("bf16", 128)])
def test_ranges_outside_the_call_leave_the_others(fmt, dim):
    """Non-decreasing, but beginning below 0 or ending past the call's rows: that sequence alone is refused."""
    c = Cache(fmt, (200, 50), 2, dim, seed=81)
    q = queries(c, 4, 4)
    good = run(c, 4, [0, 2, 4], [199, 200, 49, 50], q)
    low = run(c, 4, [-2, 2, 4], [1 << 30, 200, 49, 50], q, plan=c.plan(4, 4, 4))
    high = run(c, 4, [0, 2, 9], [199, 200, 49, 1 << 30], q, plan=c.plan(4, 4, 9))
    for got, kept in ((low, slice(2, 4)), (high, slice(0, 2))):
        gone = slice(2 - kept.start, 4 - kept.start)
        assert got[3] == 4 and (got[0][gone] == 0).all() and np.isneginf(got[1][gone]).all()
        assert np.array_equal(got[0][kept], good[0][kept]) and np.array_equal(got[1][kept], good[1][kept])
