"""Page tables far wider than what the sequences hold: chunks, workspaces, clusters and the joins' work follow the
table, the results follow the sequences."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from kv_util import Cache
from test_gpu_kv_attend import check
from test_gpu_kv_cache import append, check_evict, evict, expected, same_pool, slots

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim,page", [("q8_0", 128, 64), ("f16", 64, 16), ("f16", 128, 16), ("bf16", 128, 256), ("bf16", 256, 32)])
@pytest.mark.parametrize("slots_wide", [2048, 16384])
@pytest.mark.parametrize("heads,per", [(4, 1), (12, 2)])
def test_attend(fmt, dim, page, slots_wide, heads, per):
    check(Cache(fmt, (300, 1, 70), 2, dim, page, seed=100, width=slots_wide // page), heads, per)


@pytest.mark.parametrize("fmt,page", [("q8_0", 64), ("f16", 16), ("bf16", 256)])
@pytest.mark.parametrize("slots_wide", [16384, 65536, 262144])  # one block a KV head, and clusters
def test_evict(fmt, page, slots_wide):
    c = Cache(fmt, (333, 64, 1), 1, 128 if fmt == "q8_0" else 64, page, seed=101, width=slots_wide // page)
    if slots_wide <= 16384:
        check_evict(c, *slots(c), keep=[100, 63, 1], sink=3, protect=[300, 60, 0])
        return
    # (the same sequences under a narrow table keep the same tokens)
    narrow = Cache(fmt, (333, 64, 1), 1, 128 if fmt == "q8_0" else 64, page, seed=101)
    w, pos = slots(narrow, kind="few")
    shape = (3, 1, c.cap)
    ww, pp = np.zeros(shape, np.float32), np.zeros(shape, np.int32)
    ww[:, :, :narrow.cap], pp[:, :, :narrow.cap] = w, pos
    a = evict(narrow, w, pos, [100, 63, 1], 3, [300, 60, 0])
    b = evict(c, ww, pp, [100, 63, 1], 3, [300, 60, 0])
    assert a[4] == b[4] == 0 and a[3] == b[3] and torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))
    for x, y in ((a[1], b[1]), (a[2], b[2])):
        for s, n in enumerate(a[3]):
            assert np.array_equal(x[s, :, :n], y[s, :, :n])


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
def test_append(fmt):
    torch_cuda()
    c = Cache(fmt, (60, 0, 5), 2, seed=102, room=[100, 70, 70], width=1000)
    k, v = torch.randn(43, 2, 128), torch.randn(43, 2, 128)
    pool, w, pos, err = append(c, (3, 33, 7), k.cuda(), v.cuda())
    want, ww, wp = expected(c, (3, 33, 7), k.numpy(), v.numpy())
    assert err == 0 and np.array_equal(w, ww) and np.array_equal(pos, wp)
    same_pool(c, pool, want)
