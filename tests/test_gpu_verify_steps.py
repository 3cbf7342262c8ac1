"""Verification: what a step waits for."""
import ctypes

import pytest

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


class EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte), ("reserved", ctypes.c_ubyte * 5)]


def captured_edges(stream, work):
    """Types of the edges of the graph that `work` is on a stream (0: full, 1: programmatic); nothing of it runs."""
    rt = ctypes.CDLL("libcudart.so.13")
    s, graph, n = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()
    assert rt.cudaStreamBeginCapture(s, 2) == 0
    try:
        work()
    finally:
        assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) == 0
    assert rt.cudaGraphGetEdges(graph, None, None, None, ctypes.byref(n)) == 0
    a, b, d = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (EdgeData * n.value)()
    assert rt.cudaGraphGetEdges(graph, a, b, d, ctypes.byref(n)) == 0
    kinds = {(a[i], b[i]): d[i].type for i in range(n.value)}
    assert rt.cudaGraphDestroy(graph) == 0
    return sorted(kinds.values())


@pytest.mark.parametrize("rows", [0, 4])
def test_the_kernel_before_has_finished(rows):
    """The kernel that reads agent_rows starts behind the one that wrote it: it may start early behind verification's own first
    kernel only, which a step without rows does not have."""
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    plan = serve.VerifyPlan(agents=2, max_rows=4, columns=100)
    x, ar, tok = t.zeros(rows, 100, device="cuda"), i32([0, rows // 2, rows]), i32([1] * rows)
    au, su, acc, out = t.zeros(rows, device="cuda"), t.zeros(2, device="cuda"), i32([9, 9]), i32([9, 9])
    step = lambda: plan.verify(x, ar, tok, au, su, acc, out)  # noqa: E731
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        step()
        s.synchronize()
        assert plan.error() == 0
        if rows == 0:
            assert acc.tolist() == [0, 0] and out.tolist() == [-1, -1]
        edges = captured_edges(s, lambda: (ar.mul_(1), step()))
    assert edges == ([0, 1] if rows else [0])
