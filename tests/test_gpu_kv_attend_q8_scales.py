"""q8_0 values whose 32-dim blocks differ widely in scale: each output's error is bounded by that
dim's own sum p |v| (kv_util.check_attend), so a block keeps its accuracy beside a larger one."""
import numpy as np
import pytest

from kv_util import Cache, attend_ref, check_attend
from test_gpu_kv_attend import SPLIT, queries, rows_of, run

pytestmark = pytest.mark.gpu


def scales(c):
    """V's scales of the whole pool, fp16 [pages][kv_heads][4][64]."""
    return c.pool.numpy()[:, :, 16896:].view(np.float16).reshape(c.pages, c.kvh, 4, 64)


@pytest.mark.parametrize("blocks", [(14, -12, 0, -3), (15.9, -6, -14, 3), (8, -14, -24, 2), (0, -22, -24, -20), (-10, -24, -24, -14),
                                    (15.9, -24, -20, -9), (15.5, 15.9, -24, -23)], ids=str)
@pytest.mark.parametrize("heads,per", [(4, 1), (20, 1), (12, 3), (48, 1)])
def test_blocks_of_large_and_of_small_values(blocks, heads, per):
    c = Cache("q8_0", (333, 70), 1, seed=50)
    # (a quarter of a binade's spread, so that significands differ; what fp16 cannot hold rounds here)
    wide = np.array(blocks)[:, None] + np.random.default_rng(51).uniform(-0.25, 0, (c.pages, 1, 4, 64))
    scales(c)[:] = np.exp2(wide).astype(np.float16)
    ar, rl = rows_of(c.lens, per)
    q = queries(c, len(rl), heads)
    ref = attend_ref(*c.values(), ar, rl, q.double().numpy(), 128 ** -0.5)
    out, lse, w, err = run(c, heads, ar, rl, q)
    assert err == 0
    check_attend(ref, out, lse, w, "f32", SPLIT["q8_0"])


def test_a_few_tokens_of_extreme_blocks_among_ordinary_ones():
    """Also where only the later rows of a sequence see them, and where one of them is not finite."""
    c = Cache("q8_0", (300, 130), 2, seed=52)
    s = scales(c)
    for a, t in ((0, 7), (0, 128), (0, 298), (0, 299), (1, 0), (1, 129)):
        s[c.table[a, t // 64], :, :, t % 64] = np.float16([60000.0, 6e-8, 1e-7, 0.0])[[0, 1, 2, 3]]
    ar, rl = rows_of(c.lens, 3)
    q = queries(c, 6, 8)
    ref = attend_ref(*c.values(), ar, rl, q.double().numpy(), 128 ** -0.5)
    out, lse, w, err = run(c, 8, ar, rl, q)
    assert err == 0
    check_attend(ref, out, lse, w, "f32", SPLIT["q8_0"])
    s[c.table[0, 299 // 64], :, 2, 299 % 64] = np.nan  # the last draft's token
    again, _, _, err = run(c, 8, ar, rl, q)
    assert err == 0 and np.isnan(again[2, :, 64:96]).all()
    rest = [0, 1, 3, 4, 5]
    assert np.array_equal(again[rest], out[rest])
