"""Accumulated weights around scores that are not numbers: NaN for every token that such a row
sees, and nothing added to the others."""
import numpy as np
import pytest
import torch

from kv_util import Cache, attend_ref
from test_gpu_kv_attend import queries, run
from test_gpu_kv_attend_nan import HEADS, POOLS, keys_nan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", POOLS)
@pytest.mark.parametrize("short,n", [(40, 64), (200, 500), (1500, 3000)])
def test_a_nan_row_leaves_the_tokens_that_it_does_not_see(fmt, dim, short, n):
    c = Cache(fmt, (n,), 2, dim, seed=33)
    q = queries(c, 2, HEADS)
    q[0, 0, 3] = torch.nan  # KV head 0
    win = np.random.default_rng(1).random((1, 2, c.cap)).astype(np.float32)
    _, _, w, err = run(c, HEADS, [0, 2], [short, n], q, weight_in=win)
    assert err == 0 and np.isnan(w[0, 0, :short]).all()
    # the rest is what the row that sees it adds: row 1 in KV head 0, both in KV head 1
    k, v = c.values()
    one = attend_ref(k, v, [0, 1], [n], q[1:].double().numpy(), dim ** -0.5, win)
    q[0, 0, 3] = 0
    two = attend_ref(k, v, [0, 2], [short, n], q.double().numpy(), dim ** -0.5, win)
    for got, ref, s in ((w[0, 0, short:n], one, (0, 0, slice(short, n))), (w[0, 1, :n], two, (0, 1, slice(0, n)))):
        tol = ref["wtol"][s] + 2.0 ** -22 * np.abs(ref["weight"][s])  # as check_attend derives it
        assert (np.abs(got - ref["weight"][s]) <= tol).all()


@pytest.mark.parametrize("fmt,dim", POOLS)
@pytest.mark.parametrize("lo,hi", [(0, 1024), (1024, 2048), (0, 3000), (17, 18)])
@pytest.mark.parametrize("rows", [1, 9, 40])
def test_nan_keys_make_every_seen_weight_nan(fmt, dim, lo, hi, rows):
    """The softmax of a row that sees a NaN score has no entry that is a number, also in the parts of the
    sequence without one."""
    c = Cache(fmt, (3000,), 2, dim, seed=34)
    keys_nan(c, 0, lo, hi, slice(0, 1))  # KV head 0 only
    q = queries(c, rows, HEADS)
    _, _, w, err = run(c, HEADS, [0, rows], [3000 - i for i in range(rows)], q)
    assert err == 0 and np.isnan(w[0, 0, :3000]).all() and np.isfinite(w[0, 1]).all()
