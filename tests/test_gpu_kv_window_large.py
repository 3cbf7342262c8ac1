"""Windowed attention over scores of large magnitude, where neighbouring fp32 values lie further apart than a softmax's
exponents can be off (qmm_kv_attend_window).

A softmax over such scores is decided by exact ties, or by one token that is far above the others.  The tied tokens have
the same key, so the same score, and all others lie thousands below it in the exponent: out is the mean of the tied tokens'
V, whatever the roundings of the scores.  A probability is rounded once to the pool's 16 bits (half a step: test_gpu_kv_window's
PRODUCT), all ties alike, and the sums and the division take a few roundings of fp32, 2^-20.  lse is off by a few roundings of
the score, 2^-21 of it.  Queries have several bits, so that a score times the scale is not a number of fp32."""
import numpy as np
import pytest
import torch

from kv_util import Cache
from test_gpu_kv_attend_large import set_key
from test_gpu_kv_window import PRODUCT, run

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634
POWERS = [19.6, 21.9, 22.3, 24.7, 26.2, 27.3, 28.6, 29.5, 30.2, 31.0, 33.7, 45.1, 60.0, 100.0]


def many_bits(fmt, rows, heads, dim):
    """Queries in dim 0: 1 to 2 in steps of the type's (fp16 2^-10, bf16 2^-7), no two neighbours alike."""
    step = 128 if fmt == "bf16" else 1024
    q = torch.zeros(rows, heads, dim, dtype=torch.bfloat16 if fmt == "bf16" else torch.float16)
    i = torch.arange(rows * heads).reshape(rows, heads)
    q[..., 0] = 1 + (37 * i + 3) % step / step
    return q


def check_ties(fmt, dim, sign, rows, heads, n, at, power, window=None, sinks=0, chunks=None):
    c = Cache(fmt, (n,), 1, dim, seed=40)
    for t in range(n):
        set_key(c, t, {1: 384.0 if t > 1 else 448.0, -1: -4096.0 if t > 1 else -2560.0}[sign])
    for t in at:
        set_key(c, t, sign * 1024.0)
    k, v = c.values()
    q = many_bits(fmt, rows, heads, dim)
    top = float(np.abs(k[0, 0, at[0], 0]))
    scale = 2.0 ** power / LOG2E / top  # base-2 scores of +-2^power to twice that
    plan = c.plan(heads, rows, rows)
    if chunks is not None:
        assert (plan._bytes("qmm_kv_window_workspace_bytes", rows, window or plan.cap, sinks) > 0) == chunks
    out, lse, err = run(c, heads, [0, rows], [n] * rows, q, window, sinks, scale=scale, plan=plan)
    assert err == 0
    want, mag = v[0, 0, at].mean(0), np.abs(v[0, 0, at]).mean(0)
    assert np.isfinite(out).all()
    assert (np.abs(out - want) <= mag * (PRODUCT[fmt] * 1.001 + 2.0 ** -20)).all()
    x = sign * top * float(np.float32(scale)) * q[..., 0].double().numpy()
    assert (np.abs(lse - (x + np.log(len(at)))) <= 2.0 ** -21 * np.abs(x)).all()


KINDS = [("q8_0", 128), ("f16", 64), ("f16", 128), ("f16", 256), ("bf16", 64), ("bf16", 128), ("bf16", 256)]


@pytest.mark.parametrize("fmt,dim", KINDS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("rows", [1, 8])  # 40 queries, and 320: decode steps and prompts
@pytest.mark.parametrize("power", POWERS)
def test_ties(fmt, dim, sign, rows, power):
    check_ties(fmt, dim, sign, rows, 40, 900, [3, 130, 131, 500, 899], power)
    check_ties(fmt, dim, sign, rows, 40, 250, [3, 64, 130, 131, 249], power, chunks=False)


@pytest.mark.parametrize("fmt,dim", KINDS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", POWERS)
def test_one_token(fmt, dim, sign, power):
    """A row that sees one token has its V."""
    check_ties(fmt, dim, sign, 3, 40, 1, [0], power)


@pytest.mark.parametrize("fmt,dim", KINDS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("window,sinks", [(None, 0), (7001, 300)])
@pytest.mark.parametrize("power", [21.9, 28.6, 31.0, 60.0])
def test_ties_in_chunks(fmt, dim, sign, window, sinks, power):
    """Tokens cut into chunks, whose references are joined."""
    check_ties(fmt, dim, sign, 1, 20, 12000, [200, 5100, 5101, 9000, 11999], power, window, sinks, chunks=True)


@pytest.mark.parametrize("fmt,dim", KINDS)
@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("spread", [0.25, 4.0, 64.0])
def test_random_scores(fmt, dim, rows, spread):
    """Scores of 2^26 to 2^36 of random signs.  Where the largest is above the next by more than what their roundings can
    be off (2^-18 of the magnitudes) and 64 more, all of the weight is its token's."""
    heads, n = 8, 300
    c = Cache(fmt, (n, 40), 1, dim, seed=41)
    ar, rl = [0, rows, rows + 1], [n - 7 * j for j in range(rows)] + [1]
    g = torch.Generator().manual_seed(42)
    q = (torch.randn(rows + 1, heads, dim, generator=g) * 500).to(torch.bfloat16 if fmt == "bf16" else torch.float16)
    if fmt == "q8_0":
        scale = spread * 2.0 ** 15
    else:
        c.pool[:, :, 0] *= 500
        scale = spread * 2.0 ** 6
    k, v = c.values()
    out, lse, err = run(c, heads, ar, rl, q, None, 0, scale=scale)
    assert err == 0
    compared = 0
    for r in range(rows + 1):
        a = int(r == rows)
        for h in range(heads):
            kk, qq = k[a, 0, :rl[r]], q[r, h].double().numpy()
            x = kk @ qq * float(np.float32(scale))
            big = (np.abs(kk) @ np.abs(qq)).max() * scale
            first = int(x.argmax())
            if rl[r] > 1 and np.sort(x)[-2] > x[first] - 2.0 ** -18 * big - 64:
                continue
            compared += 1
            want = v[a, 0, first]
            assert (np.abs(out[r, h] - want) <= np.abs(want) * (PRODUCT[fmt] * 1.001 + 2.0 ** -20)).all(), (r, h)
            assert abs(lse[r, h] - x[first]) <= 2.0 ** -20 * big
    assert compared >= 0.9 * (rows + 1) * heads
