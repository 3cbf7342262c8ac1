"""Append calls whose agent_rows falls somewhere: refused as a whole; a range outside the call's rows costs its
own sequence only."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from kv_util import Cache
from test_gpu_kv_cache import expected, i32, same_pool

pytestmark = pytest.mark.gpu


def append(c, agent_rows, k, v):
    t = torch_cuda()
    w, pos = t.full((c.agents, c.kvh, c.cap), 2.5, device="cuda"), t.full((c.agents, c.kvh, c.cap), -9, dtype=t.int32, device="cuda")
    pool, plan = c.pool.cuda(), c.plan(c.kvh, len(k))
    plan.append(pool, i32(agent_rows), i32(c.lens), k, v, weight=w, pos=pos, row_pos=i32([1000 + r for r in range(len(k))]))
    t.cuda.synchronize()
    return pool.cpu(), w.cpu().numpy(), pos.cpu().numpy(), plan.error()


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
@pytest.mark.parametrize("agent_rows", [[0, 600, 0, 600], [0, 600, 400, 500], [0, 200, 100, 100], [600, 0, 300, 600], [0, 300, 600, -1]])
def test_rows_that_fall(fmt, agent_rows):
    c = Cache(fmt, (0, 5, 9), 2, seed=90, room=[640, 640, 640])
    k, v = torch.randn(600, 2, 128), torch.randn(600, 2, 128)
    pool, w, pos, err = append(c, agent_rows, k.cuda(), v.cuda())
    assert err == 4 and torch.equal(pool.view(torch.uint8), c.pool.view(torch.uint8)) and (w == 2.5).all() and (pos == -9).all()


@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
def test_ranges_outside_the_call_leave_the_others(fmt):
    c = Cache(fmt, (0, 5), 2, seed=91, room=[640, 640])
    k, v = torch.randn(40, 2, 128), torch.randn(40, 2, 128)
    for agent_rows, skip in (([0, 30, 41], 1), ([0, 30, (1 << 31) - 1], 1), ([-(1 << 31), 0, 40], 0), ([-1, 0, 40], 0)):
        pool, w, pos, err = append(c, agent_rows, k.cuda(), v.cuda())
        want, ww, wp = expected(c, (30, 10) if skip else (0, 40), k.numpy(), v.numpy(), skip=(skip,))
        assert err == 4 and np.array_equal(w, ww) and np.array_equal(pos, wp)
        same_pool(c, pool, want)
