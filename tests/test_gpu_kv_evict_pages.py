"""Eviction where the page table points outside the pool: the tokens concerned stay where they are, with
their weight and position."""
import numpy as np
import pytest
import torch

from kv_util import Cache, evict_ref
from test_gpu_kv_cache import evict, slots

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,page", [("q8_0", 64), ("f16", 64), ("bf16", 16)])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_a_page_outside_the_pool_moves_nothing_of_a_token(fmt, page, inplace, at):
    """at: which of the sequence's 64-slot ranges has a bad page; 0 holds destinations, 2 sources, 1 both."""
    c = Cache(fmt, (190, 70), 2, 128, page, seed=60)
    w, pos = slots(c, kind="random")
    keep = [100, 50]
    bad = 64 * at // page  # the bad page's column
    good, c.table = c.table, c.table.copy()
    c.table[0, bad] = c.pages
    pool, wo, po, n, err = evict(c, w, pos, keep, inplace=inplace)
    assert err == 2 and n == keep
    c.table = good
    k0, v0 = c.values()
    c.pool = pool.cpu()
    k1, v1 = c.values()
    skipped = 0
    for a in range(2):
        for g in range(2):
            budget, moves = evict_ref(w[a, g], pos[a, g], c.lens[a], keep[a], 0, 1 << 30)
            ww, pp, kk, vv = w[a, g].copy(), pos[a, g].copy(), k0[a, g].copy(), v0[a, g].copy()
            for src, dst in moves:
                if a == 0 and bad in (src // page, dst // page):
                    skipped += 1
                    continue
                ww[dst], pp[dst], kk[dst], vv[dst] = w[a, g, src], pos[a, g, src], k0[a, g, src], v0[a, g, src]
            assert np.array_equal(k1[a, g], kk) and np.array_equal(v1[a, g], vv)
            assert np.array_equal(wo[a, g, :budget], ww[:budget]) and np.array_equal(po[a, g, :budget], pp[:budget])
    assert skipped > 0
