"""Attention rows whose scores are not numbers: out and lse are NaN, never those of an empty row, and
what another row or head gets is unchanged bit for bit."""
import numpy as np
import pytest
import torch

from kv_util import Cache
from test_gpu_kv_attend import queries, run

pytestmark = pytest.mark.gpu

POOLS = [("q8_0", 128), ("f16", 64), ("f16", 128), ("f16", 256), ("bf16", 64), ("bf16", 128), ("bf16", 256)]
HEADS = 4  # over two KV heads


def keys_nan(c, a, lo, hi, heads=slice(None)):
    """Every K of sequence a's slots lo .. hi - 1 becomes NaN (q8_0: its scales do)."""
    for t in range(lo, hi):
        pg, s = c.table[a, t // c.page], t % c.page
        if c.fmt == "q8_0":
            c.pool.numpy()[pg, heads, 8192 + 8 * s:8200 + 8 * s] = np.full(4, np.nan, np.float16).view(np.uint8)
        else:
            c.pool[pg, heads, 0, s] = torch.nan


# (33 chunks and more of up to 1,024 slots are joined another way than fewer)
@pytest.mark.parametrize("fmt,dim", POOLS)
@pytest.mark.parametrize("n", [1, 70, 1500, 34000])
def test_a_query_that_is_nan_gives_nan(fmt, dim, n):
    c = Cache(fmt, (n, 40), 2, dim, seed=31)
    ar, rl = [0, 3, 4], [n, 0, max(1, n - 1), 40]
    q = queries(c, 4, HEADS)
    want = run(c, HEADS, ar, rl, q)
    q[0, 1, 5] = torch.nan  # one element of one head
    q[1] = torch.nan        # a row that sees nothing
    out, lse, _, err = run(c, HEADS, ar, rl, q)
    assert err == 0
    assert np.isnan(out[0, 1]).all() and np.isnan(lse[0, 1])
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    rest = np.ones((4, HEADS), bool)
    rest[0, 1] = False
    assert np.array_equal(out[rest], want[0][rest]) and np.array_equal(lse[rest], want[1][rest])


@pytest.mark.parametrize("fmt,dim", POOLS)
@pytest.mark.parametrize("n,lo,hi", [(70, 0, 70), (3000, 0, 3000), (3000, 1024, 2048), (3000, 2999, 3000)],
                         ids=["all", "all long", "whole chunks", "last"])
def test_keys_that_are_nan_give_nan(fmt, dim, n, lo, hi):
    c = Cache(fmt, (n, 40), 2, dim, seed=32)
    ar, rl = [0, 2, 3], [lo, n, 40]
    q = queries(c, 3, HEADS)
    want = run(c, HEADS, ar, rl, q)
    keys_nan(c, 0, lo, hi)
    out, lse, _, err = run(c, HEADS, ar, rl, q)
    assert err == 0 and np.isnan(out[1]).all() and np.isnan(lse[1]).all()
    for r in (0, 2):  # the row that ends before them (or sees nothing), and the other sequence
        assert np.array_equal(out[r], want[0][r]) and np.array_equal(lse[r], want[1][r])
