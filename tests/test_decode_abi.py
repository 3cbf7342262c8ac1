"""The C ABI of rotation, windowed attention and draft verification without a GPU: exports, and refusals before
the device is touched."""
import ctypes
import subprocess

import pytest

from bit_weight_streaming_q4_gb300 import build as qbuild
from bit_weight_streaming_q4_gb300 import qmm as Q
from bit_weight_streaming_q4_gb300 import serve as S

INVALID, SHAPE, MISALIGNED, SCRATCH = 1, 2, 3, 9
P = 0x10000  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return S.load()


def kv_dims(**kw):
    d = dict(format=1, heads=8, kv_heads=2, head_dim=128, page_tokens=64, agents=3, max_pages=10, max_agent_rows=4, pool_pages=40)
    d.update(kw)
    return S.KvDims(*[d[n] for n, _ in S.KvDims._fields_])


def rot_dims(**kw):
    d = dict(heads=8, kv_heads=2, head_dim=128, rot_dim=128, axes=1, interleaved=0, in_type=0, q_type=1, k_type=0, eps=1e-6)
    d.update(kw)
    return S.RotateDims(*[d[n] for n, _ in S.RotateDims._fields_])


def rotate(lib, d, **kw):
    a = dict(q=P, qs=1024, k=P, ks=256, rows=4, qw=P, kw=P, pos=P, inv=P, axis=None, qo=2 * P, qos=1024, ko=3 * P, kos=256, stream=None)
    a.update(kw)
    return lib.qmm_rotate(ctypes.byref(d) if d else None, *a.values())


def window(lib, d, **kw):
    a = dict(pool=P, table=P, agent_rows=P, row_len=P, q=P, q_stride=1024, rows=4, max_rows=12, scale=1.0, window=64, sinks=4, out=P,
             out_type=0, lse=P, ws=P, ws_bytes=1 << 40, err=P, stream=None)
    a.update(kw)
    return lib.qmm_kv_attend_window(ctypes.byref(d) if d else None, *a.values())


def verify(lib, **kw):
    a = dict(logits=P, type=0, stride=100, n=100, draft=P, ds=100, agent_rows=P, agents=2, rows=6, tokens=P, temp=None, au=P, su=P,
             accepted=P, token=P, prob=None, ws=P, ws_bytes=1 << 40, err=P, stream=None)
    a.update(kw)
    return lib.qmm_verify(*a.values())


def test_header_and_exports(lib):
    names = S.header_functions(S.DECODE_HEADER)
    assert names == ["qmm_kv_attend_window", "qmm_kv_window_workspace_bytes", "qmm_rotate", "qmm_verify", "qmm_verify_workspace_bytes"]
    out = subprocess.run(["nm", "-D", "--defined-only", qbuild.LIB], capture_output=True, text=True).stdout
    for n in names:
        assert f" T {n}\n" in out


@pytest.mark.parametrize("change", [dict(heads=-1), dict(heads=0, kv_heads=0), dict(in_type=3), dict(q_type=-1), dict(k_type=7), dict(eps=-1.0),
                                    dict(eps=float("nan"))])
def test_rotate_dims_invalid(lib, change):
    assert rotate(lib, rot_dims(**change)) == INVALID
    assert rotate(lib, None) == INVALID


@pytest.mark.parametrize("change", [dict(head_dim=80), dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=-16), dict(axes=0), dict(axes=5),
                                    dict(heads=70000)])
def test_rotate_dims_unsupported(lib, change):
    assert rotate(lib, rot_dims(**change)) == SHAPE


@pytest.mark.parametrize("change", [dict(rows=-1), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(qs=1023), dict(ks=255),
                                    dict(qos=1000), dict(kos=1), dict(pos=None), dict(inv=None), dict(qo=P)])
def test_rotate_arguments(lib, change):
    assert rotate(lib, rot_dims(), **change) == INVALID


def test_rotate_in_place_needs_the_same_layout(lib):
    assert rotate(lib, rot_dims(q_type=0), qo=P, qos=1032) == INVALID
    assert rotate(lib, rot_dims(k_type=1), ko=P) == INVALID


@pytest.mark.parametrize("change", [dict(q=P + 2), dict(k=P + 1), dict(qo=P + 1), dict(ko=P + 2), dict(qw=P + 2), dict(kw=P + 1), dict(pos=P + 2),
                                    dict(inv=P + 2), dict(axis=P + 2)])
def test_rotate_misaligned(lib, change):
    assert rotate(lib, rot_dims(), **change) == MISALIGNED


def test_no_rows_is_no_work(lib):
    assert rotate(lib, rot_dims(), rows=0, q=None, k=None, pos=None) == 0
    assert window(lib, kv_dims(), rows=0, pool=None, q=None) == 0


@pytest.mark.parametrize("change", [dict(heads=0), dict(heads=9), dict(agents=0), dict(max_pages=0), dict(pool_pages=0), dict(format=3),
                                    dict(max_agent_rows=0)])
def test_window_dims_invalid(lib, change):
    assert window(lib, kv_dims(**change)) == INVALID
    assert window(lib, None) == INVALID
    n = ctypes.c_int64()
    assert lib.qmm_kv_window_workspace_bytes(ctypes.byref(kv_dims(**change)), 12, 64, 4, ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("change", [dict(head_dim=96), dict(page_tokens=24), dict(agents=961), dict(format=0, page_tokens=32),
                                    dict(max_agent_rows=1 << 23), dict(max_pages=1 << 25)])
def test_window_dims_unsupported(lib, change):
    assert window(lib, kv_dims(**change)) == SHAPE


@pytest.mark.parametrize("change", [dict(rows=-1), dict(rows=13), dict(window=0), dict(window=-4), dict(sinks=-1), dict(out_type=3), dict(pool=None),
                                    dict(table=None), dict(agent_rows=None), dict(row_len=None), dict(q=None), dict(out=None), dict(err=None),
                                    dict(q_stride=1000), dict(max_rows=-1)])
def test_window_arguments(lib, change):
    assert window(lib, kv_dims(), **change) == INVALID


@pytest.mark.parametrize("change", [dict(pool=P + 8), dict(q=P + 8), dict(q_stride=1028), dict(out=P + 4), dict(table=P + 1), dict(agent_rows=P + 2),
                                    dict(row_len=P + 2), dict(lse=P + 2), dict(err=P + 1), dict(ws=P + 8)])
def test_window_misaligned(lib, change):
    assert window(lib, kv_dims(), **change) == MISALIGNED


def test_window_workspace(lib):
    n = ctypes.c_int64(-1)
    assert lib.qmm_kv_window_workspace_bytes(ctypes.byref(kv_dims()), 12, 64, 4, None) == INVALID
    for d in (kv_dims(), kv_dims(max_pages=4000, pool_pages=4000, agents=1)):
        for w in (1, 64, 4096, 1 << 30):
            assert lib.qmm_kv_window_workspace_bytes(ctypes.byref(d), 12, w, 4, ctypes.byref(n)) == 0 and n.value >= 0
            if n.value:
                assert window(lib, d, window=w, ws_bytes=n.value - 1) == SCRATCH
                assert window(lib, d, window=w, ws=None) == INVALID


@pytest.mark.parametrize("change", [dict(type=3), dict(agents=0), dict(rows=-1), dict(n=0), dict(stride=99), dict(ds=99), dict(logits=None),
                                    dict(agent_rows=None), dict(tokens=None), dict(au=None), dict(su=None), dict(accepted=None), dict(token=None),
                                    dict(err=None), dict(ws=None)])
def test_verify_arguments(lib, change):
    assert verify(lib, **change) == INVALID


@pytest.mark.parametrize("change", [dict(n=(1 << 19) + 1, stride=1 << 20, ds=1 << 20), dict(rows=65536), dict(agents=65536)])
def test_verify_unsupported(lib, change):
    assert verify(lib, **change) == SHAPE


@pytest.mark.parametrize("change", [dict(logits=P + 2), dict(draft=P + 1), dict(agent_rows=P + 2), dict(tokens=P + 2), dict(temp=P + 2), dict(au=P + 1),
                                    dict(su=P + 2), dict(accepted=P + 2), dict(token=P + 2), dict(prob=P + 2), dict(ws=P + 8), dict(err=P + 2)])
def test_verify_misaligned(lib, change):
    assert verify(lib, **change) == MISALIGNED


def test_verify_workspace(lib):
    n = ctypes.c_int64()
    assert lib.qmm_verify_workspace_bytes(6, 100, None) == INVALID
    assert lib.qmm_verify_workspace_bytes(6, 100, ctypes.byref(n)) == 0 and n.value > 0
    assert verify(lib, ws_bytes=n.value - 1) == SCRATCH


def test_no_device(lib):
    """Calls that pass every check say that there is no GPU (where there is none)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")
    for st in (rotate(lib, rot_dims()), window(lib, kv_dims()), verify(lib)):
        with pytest.raises(Q.QmmError):
            Q._check(st, "call")
