"""The workspaces of a plan whose calls have windows of their own: bounded, whatever their number, and what a captured call was
given stays."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from kv_util import Cache
from test_gpu_kv_window import queries, run

pytestmark = pytest.mark.gpu


def setup(seed):
    t = torch_cuda()
    c = Cache("f16", [20000], 1, 128, 64, seed=seed)
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    q = queries(c, 2, 4)
    return t, c, c.plan(4, 2, 2), (c.pool.cuda(), i32([0, 2]), i32([19999, 20000])), q, t.empty(2, 4, 128, device="cuda")


def test_windows_that_grow():
    """A window of its own for each step: hundreds under one plan."""
    t, c, plan, args, q, out = setup(60)
    windows = list(range(300, 20000, 61))
    need = max(plan._bytes("qmm_kv_window_workspace_bytes", 2, w, s) for w in windows for s in (0, 3))
    qd = q.cuda()
    t.cuda.synchronize()
    before = t.cuda.memory_allocated()
    for w in windows + windows[::-1]:
        for s in (0, 3):
            plan.attend_window(*args, qd, out, window=w, sinks=s)
    t.cuda.synchronize()
    # (each is at least twice the one before it, none more than twice what a call needs; the allocator's blocks are of 512 bytes)
    assert t.cuda.memory_allocated() - before <= 4 * need + 64 * 512
    assert plan.error() == 0
    for w in (300, 5180, windows[-1]):
        plan.attend_window(*args, qd, out, window=w, sinks=3)
        want, _, _ = run(c, 4, [0, 2], [19999, 20000], q, w, 3)
        assert np.array_equal(out.double().cpu().numpy(), want)


def test_a_captured_call_keeps_its_workspace():
    t, c, plan, args, q, out = setup(61)
    qd = q.cuda()
    want, _, _ = run(c, 4, [0, 2], [19999, 20000], q, 1500, 0)
    plan.attend_window(*args, qd, out, window=1500)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        plan.attend_window(*args, qd, out, window=1500)
    other = t.empty_like(out)
    for w in (3000, 9000, None, 400):
        plan.attend_window(*args, qd, other, window=w, sinks=7)
        out.fill_(3)
        g.replay()
        t.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want)
    assert plan.error() == 0
