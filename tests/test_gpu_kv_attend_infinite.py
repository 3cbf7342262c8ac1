"""Infinities in V that a row sees: out is infinite in that dim whatever the token's probability and whichever rows
see it; opposite ones, or one beside a NaN, are NaN; the other dims are numbers as ever."""
import numpy as np
import pytest

from kv_util import Cache, attend_ref, check_attend
from test_gpu_kv_attend import SPLIT, queries, run

pytestmark = pytest.mark.gpu


def put(c, a, g, t, dim, value):
    """V of one element (q8_0: the scale of its 32-dim block, quants 1, or -1 for a negative value)."""
    pg, s = c.table[a, t // c.page], t % c.page
    if c.fmt != "q8_0":
        c.pool[pg, g, 1, s, dim] = value
        return [dim]
    b, blk = c.pool.numpy()[pg, g], dim // 32
    b[16896:].view(np.float16)[blk * 64 + s] = abs(value)
    dims = np.arange(32 * blk, 32 * blk + 32)
    b[8704 + dims * 64 + s] = np.int8(-1 if value < 0 else 1).view(np.uint8)
    return list(dims)


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("f16", 128), ("f16", 256), ("bf16", 64), ("bf16", 128), ("bf16", 256)])
@pytest.mark.parametrize("heads", [2, 12, 40])
@pytest.mark.parametrize("n,at", [(1, 0), (200, 5), (3000, 2100)])
@pytest.mark.parametrize("spread", [1.0, 40.0])
def test_an_infinity_that_rows_see(fmt, dim, heads, n, at, spread):
    c = Cache(fmt, (n, 70), 2, dim, seed=110)
    q = queries(c, 3, heads, spread=spread)
    k, v = c.values()
    ar, rl = [0, 2, 3], [n, min(n, at), 70]
    ref = attend_ref(k, v, ar, rl, q.double().numpy(), dim ** -0.5)
    up = put(c, 0, 0, at, 7, np.inf)
    down = put(c, 0, 0, at, 50, -np.inf)
    both = []
    if n > 1:
        both = put(c, 0, 0, at, 39 if fmt != "q8_0" else 100, np.inf)
        put(c, 0, 0, at - 1 if at < n - 1 else at + 1, 39 if fmt != "q8_0" else 100, -np.inf)
    mine = slice(0, heads // 2)  # the heads of KV head 0
    for rows in (1, 3):  # alone, so that every row sees it, and beside a row that does not
        # (no row but the first sees the tokens changed: row 1 ends before `at`, whose neighbour is past it or left out)
        lens = [rl[0], max(0, min(rl[1], at - 1)), rl[2]]
        out, lse, _, err = run(c, heads, [0, 1, 1] if rows == 1 else ar, lens[:rows], q[:rows])
        assert err == 0 and np.isfinite(lse[0]).all()
        assert np.isposinf(out[0, mine][:, up]).all() and np.isneginf(out[0, mine][:, down]).all()
        assert not both or np.isnan(out[0, mine][:, both]).all()
        keep = np.ones(dim, bool)
        keep[up + down + both] = False
        assert np.isfinite(out[0, mine][:, keep]).all() and np.isfinite(out[0, heads // 2:]).all()
        # (a bound by sum p |v| alone holds of ordinary scores: with peaked ones a q8_0 row can have a dim whose largest
        # tokens have quant 0, and what is left there lies below the 2^-38 of the largest probability that are kept)
        for h in range(heads if spread == 1.0 else 0):
            sel = keep if h < heads // 2 else np.ones(dim, bool)
            sub = {x: ref[x][:1, h:h + 1] for x in ("lse", "big")}
            sub.update(out=ref["out"][:1, h:h + 1, sel], mag=ref["mag"][:1, h:h + 1, sel])
            check_attend(sub, out[:1, h:h + 1, sel], lse[:1, h:h + 1], None, "f32", SPLIT[fmt])
        if rows == 3:
            assert np.isfinite(out[1:]).all()
