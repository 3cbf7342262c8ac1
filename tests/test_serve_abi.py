"""The serving operators' C ABI without a GPU: exports, and refusals before the device is touched."""
import ctypes
import subprocess

import pytest

from bit_weight_streaming_q4_gb300 import build as qbuild
from bit_weight_streaming_q4_gb300 import qmm as Q
from bit_weight_streaming_q4_gb300 import serve as S

INVALID, SHAPE, MISALIGNED, SCRATCH = 1, 2, 3, 9


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return S.load()


def dims(**kw):
    d = dict(format=1, heads=8, kv_heads=2, head_dim=128, page_tokens=64, agents=3, max_pages=10, max_agent_rows=4, pool_pages=40)
    d.update(kw)
    return S.KvDims(*[d[n] for n, _ in S.KvDims._fields_])


P = 0x10000  # an aligned address that no refused call may touch


def attend(lib, d, **kw):
    a = dict(pool=P, table=P, agent_rows=P, row_len=P, q=P, q_stride=1024, rows=4, scale=1.0, out=P, out_type=0, lse=P, w_in=None,
             w_out=None, ws=P, ws_bytes=1 << 40, err=P, stream=None)
    a.update(kw)
    return lib.qmm_kv_attend(ctypes.byref(d) if d else None, *a.values())


def append(lib, d, **kw):
    a = dict(pool=P, table=P, agent_rows=P, cache_len=P, k=P, ks=256, v=P, vs=256, type=0, rows=4, weight=P, pos=P, row_pos=P, err=P,
             stream=None)
    a.update(kw)
    return lib.qmm_kv_append(ctypes.byref(d) if d else None, *a.values())


def evict(lib, d, **kw):
    a = dict(pool=P, table=P, cache_len=P, keep=P, sink=0, protect=None, weight=P, pos=P, weight_out=P, pos_out=P, len_out=2 * P, ws=P,
             ws_bytes=1 << 40, err=P, stream=None)
    a.update(kw)
    return lib.qmm_kv_evict(ctypes.byref(d) if d else None, *a.values())


def logprobs(lib, **kw):
    a = dict(logits=P, type=0, m=2, n=100, stride=100, tokens=P, given=1, top=5, lse=P, entropy=P, logprob=P, top_index=P, top_logprob=P,
             stream=None)
    a.update(kw)
    return lib.qmm_logprobs(*a.values())


def test_header_and_exports(lib):
    names = S.header_functions()
    assert names == ["qmm_kv_append", "qmm_kv_attend", "qmm_kv_attend_workspace_bytes", "qmm_kv_evict",
                     "qmm_kv_evict_workspace_bytes", "qmm_logprobs"]
    out = subprocess.run(["nm", "-D", "--defined-only", Q.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(names) <= exported


@pytest.mark.parametrize("call", [attend, append, evict])
@pytest.mark.parametrize("kw,status", [
    (dict(format=3), INVALID), (dict(format=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=7), INVALID),
    (dict(kv_heads=0), INVALID), (dict(agents=0), INVALID), (dict(max_pages=0), INVALID), (dict(pool_pages=0), INVALID),
    (dict(pool_pages=1 << 31), INVALID), (dict(max_agent_rows=0), INVALID), (dict(head_dim=96), SHAPE), (dict(page_tokens=48), SHAPE),
    (dict(page_tokens=512), SHAPE), (dict(format=0, head_dim=64), SHAPE), (dict(format=0, page_tokens=32), SHAPE),
    (dict(agents=961), SHAPE), (dict(max_pages=1 << 30), SHAPE)])
def test_dims_are_checked(lib, call, kw, status):
    assert call(lib, dims(**kw)) == status
    assert call(lib, None) == INVALID


def test_attend_arguments(lib):
    d = dims()
    for name in ("pool", "table", "agent_rows", "row_len", "q", "out", "ws", "err"):
        assert attend(lib, d, **{name: None}) == INVALID
    for name, by in (("pool", 8), ("q", 2), ("out", 4), ("ws", 8), ("table", 2), ("row_len", 1), ("lse", 2), ("err", 2)):
        assert attend(lib, d, **{name: P + by}) == MISALIGNED
    assert attend(lib, d, rows=-1) == INVALID
    assert attend(lib, d, q_stride=1023) == INVALID
    assert attend(lib, d, q_stride=1028) == MISALIGNED
    assert attend(lib, d, out_type=3) == INVALID
    assert attend(lib, d, w_in=P) == INVALID  # weights in, but not out
    assert attend(lib, d, ws_bytes=0) == SCRATCH
    assert attend(lib, dims(max_agent_rows=1025)) == SHAPE  # 4,100 queries of one sequence and KV head
    assert attend(lib, d, rows=1 << 24) == SHAPE
    assert attend(lib, d, rows=0, pool=None) == 0
    n = ctypes.c_int64()
    assert lib.qmm_kv_attend_workspace_bytes(ctypes.byref(d), 0, None) == INVALID
    assert lib.qmm_kv_attend_workspace_bytes(ctypes.byref(d), 0, ctypes.byref(n)) == 0 and n.value > 0
    plain = n.value
    assert lib.qmm_kv_attend_workspace_bytes(ctypes.byref(d), 1, ctypes.byref(n)) == 0 and n.value > plain
    assert attend(lib, d, ws_bytes=n.value - 1, w_out=P) == SCRATCH


def test_append_arguments(lib):
    d = dims()
    for name in ("pool", "table", "agent_rows", "cache_len", "k", "v", "err"):
        assert append(lib, d, **{name: None}) == INVALID
    for name, by in (("pool", 8), ("k", 2), ("v", 1), ("cache_len", 2), ("weight", 2), ("row_pos", 1)):
        assert append(lib, d, **{name: P + by}) == MISALIGNED
    assert append(lib, d, rows=-1) == INVALID and append(lib, d, type=3) == INVALID and append(lib, d, ks=255) == INVALID
    assert append(lib, d, rows=(1 << 24) + 1) == SHAPE
    assert append(lib, d, rows=0, k=None) == 0


def test_evict_arguments(lib):
    d = dims()
    for name in ("pool", "table", "cache_len", "keep", "weight", "pos", "weight_out", "pos_out", "len_out", "ws", "err"):
        assert evict(lib, d, **{name: None}) == INVALID
    for name, by in (("pool", 8), ("ws", 4), ("keep", 2), ("protect", P + 2), ("weight_out", 1)):
        assert evict(lib, d, **{name: P + by}) == MISALIGNED
    assert evict(lib, d, len_out=P) == INVALID  # the lengths before
    n = ctypes.c_int64()
    assert lib.qmm_kv_evict_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    assert evict(lib, d, ws_bytes=n.value - 1) == SCRATCH
    assert lib.qmm_kv_evict_workspace_bytes(ctypes.byref(d), None) == INVALID


def test_logprobs_arguments(lib):
    for kw in (dict(type=3), dict(type=-1), dict(m=-1), dict(n=0), dict(n=1 << 31, stride=1 << 31), dict(stride=99), dict(given=-1),
               dict(top=-1), dict(top=33), dict(top=5, n=4), dict(tokens=None), dict(logprob=None), dict(top_index=None),
               dict(top_logprob=None), dict(logits=None)):
        assert logprobs(lib, **kw) == INVALID, kw
    for name, by in (("logits", 2), ("tokens", 1), ("lse", 2), ("entropy", 2), ("logprob", 2), ("top_index", 2), ("top_logprob", 2)):
        assert logprobs(lib, **{name: P + by}) == MISALIGNED
    assert logprobs(lib, m=0, logits=None) == 0
