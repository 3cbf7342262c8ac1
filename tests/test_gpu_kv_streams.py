"""Calls on a stream that is not the current one (the binding's `stream=`), by a plan that nothing has
used before."""
import pytest
import torch

from gpu_util import torch_cuda
from kv_util import Cache
from test_gpu_kv_attend import queries, rows_of, run
from test_gpu_kv_cache import evict, i32, slots

pytestmark = pytest.mark.gpu
SLEEP = 400_000_000  # clocks: some 0.2 s


def freed_block_in_use(t, n):
    """A block of n bytes that the current stream still has to read, given back to the allocator; returns
    the copy that the pending read makes, and what it has to hold."""
    t.cuda.synchronize()
    t.cuda.empty_cache()
    old, copy = t.full((n,), 5, dtype=t.uint8, device="cuda"), t.zeros(n, dtype=t.uint8, device="cuda")
    t.cuda.synchronize()
    t.cuda._sleep(SLEEP)
    copy.copy_(old)
    return copy


@pytest.mark.parametrize("kind", ["attend", "weights", "evict"])
def test_the_workspace_is_no_memory_that_the_current_stream_still_reads(kind):
    t = torch_cuda()
    c = Cache("f16", (300, 60), 2, seed=70)
    ar, rl = rows_of(c.lens, 1)
    q = queries(c, 2, 8)
    want = run(c, 8, ar, rl, q)
    evict(c, *slots(c), [100, 20])  # (a kernel's first launch loads it, which waits for the GPU)
    plan, pool, qd = c.plan(8, 2, 1), c.pool.cuda(), q.cuda()
    out, w = t.zeros(2, 8, 128, device="cuda"), t.zeros(2, 2, c.cap, device="cuda")
    ard, rld, lens, keep, left = i32(ar), i32(rl), i32(c.lens), i32([100, 20]), i32([0, 0])
    weight, pos = (t.from_numpy(x).cuda() for x in slots(c))
    n = plan._bytes("qmm_kv_evict_workspace_bytes") if kind == "evict" else \
        plan._bytes("qmm_kv_attend_workspace_bytes", int(kind == "weights"))
    s = t.cuda.Stream()
    copy = freed_block_in_use(t, n)
    if kind == "evict":
        plan.evict(pool, lens, keep, weight, pos, weight_out=weight, pos_out=pos, len_out=left, stream=s.cuda_stream)
    else:
        plan.attend(pool, ard, rld, qd, out, weight_out=w if kind == "weights" else None, stream=s.cuda_stream)
    s.synchronize()
    busy = not t.cuda.current_stream().query()
    t.cuda.synchronize()
    assert busy and bool((copy == 5).all()) and plan.error() == 0  # (the call did run beside the pending read)
    if kind != "evict":
        assert (out.double().cpu().numpy() == want[0]).all()
    else:
        assert left.tolist() == [100, 20]


def test_the_error_word_is_zero_before_the_first_call_on_any_stream():
    t = torch_cuda()
    c = Cache("f16", (300, 60), 2, seed=71)
    c.table[0, 1] = c.pages  # a page outside the pool
    ar, rl = rows_of(c.lens, 1)
    pool, qd, ard, rld = c.pool.cuda(), queries(c, 2, 8).cuda(), i32(ar), i32(rl)
    out = t.zeros(2, 8, 128, device="cuda")
    s = t.cuda.Stream()
    table = t.from_numpy(c.table).cuda()
    from bit_weight_streaming_q4_gb300 import serve
    t.cuda.synchronize()
    t.cuda._sleep(SLEEP)
    plan = serve.KvPlan(table, format="f16", heads=8, kv_heads=2, head_dim=128, page_tokens=64, pool_pages=c.pages, max_rows=2)
    plan.attend(pool, ard, rld, qd, out, stream=s.cuda_stream)
    t.cuda.synchronize()
    assert plan.error() == 2


def test_a_plan_dropped_while_its_call_runs():
    """The workspace goes back to the allocator only for work behind the call's: here a call on a stream that sleeps
    first, while the current stream takes and fills blocks of the workspace's size."""
    t = torch_cuda()
    c = Cache("f16", (3000, 60), 2, seed=72)
    ar, rl = rows_of(c.lens, 1)
    q = queries(c, 2, 8)
    want = run(c, 8, ar, rl, q)
    pool, qd, ard, rld = c.pool.cuda(), q.cuda(), i32(ar), i32(rl)
    out, w = t.zeros(2, 8, 128, device="cuda"), t.zeros(2, 2, c.cap, device="cuda")
    plan = c.plan(8, 2, 1)
    n = plan._bytes("qmm_kv_attend_workspace_bytes", 1)
    s, other = t.cuda.Stream(), t.cuda.Stream()
    t.cuda.synchronize()
    plan.attend(pool, ard, rld, qd, out, weight_out=w, stream=other.cuda_stream)  # allocates, on one stream
    other.synchronize()
    with t.cuda.stream(s):
        t.cuda._sleep(SLEEP)
    plan.attend(pool, ard, rld, qd, out, weight_out=w, stream=s.cuda_stream)      # and runs on another
    address = plan._workspace["weights"][0]
    err = plan.error_word
    del plan
    for stream in (t.cuda.current_stream(), other):
        with t.cuda.stream(stream):
            taken = [t.empty(n, dtype=t.uint8, device="cuda") for _ in range(4)]
            assert all(not (x.data_ptr() <= address < x.data_ptr() + n) for x in taken)
    t.cuda.synchronize()
    assert (out.double().cpu().numpy() == want[0]).all() and int(err.item()) == 0
