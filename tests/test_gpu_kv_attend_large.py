"""Scores of large magnitude, where neighbouring fp32 values lie further apart than the shifts that
keep the probabilities in 16 bits.

A softmax over such scores is decided by exact ties: some tokens share the largest score bit for bit
(their keys are the same), all others lie thousands below it in the exponent.  So out is the mean of
the tied tokens' V and their weight 1 / ties, whatever the roundings of the scores themselves:
2^-20 (2^-15 with bf16's parts) of the sum of |v| / ties for out, 2^-20 for a weight, and a few
roundings of the score, 2^-21 of it, for lse."""
import numpy as np
import pytest
import torch

from kv_util import Cache
from test_gpu_kv_attend import SPLIT, run

pytestmark = pytest.mark.gpu


def set_key(c, t, value):
    """K of slot t: `value` in dim 0, else 0 (q8_0: quant 127 or -127 times a scale)."""
    pg, s = c.table[0, t // c.page], t % c.page
    if c.fmt == "q8_0":
        b = c.pool.numpy()
        d = np.arange(128)
        b[pg, :, s * 128 + 16 * ((d // 16) ^ (2 * (s % 4) + (s // 4) % 2)) + d % 16] = 0
        b[pg, :, s * 128 + 16 * (2 * (s % 4) + (s // 4) % 2)] = np.int8(127 * np.sign(value)).view(np.uint8)
        b[pg, :, 8192 + 8 * s:8200 + 8 * s] = np.full(4, abs(value) / 127, np.float16).view(np.uint8)
    else:
        c.pool[pg, :, 0, s] = 0
        c.pool[pg, :, 0, s, 0] = value


@pytest.mark.parametrize("fmt,dim", [("q8_0", 128), ("f16", 64), ("f16", 128), ("f16", 256), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("heads", [1, 20, 40])  # tiles of 16, 24 and 48 queries at head dimension 128
@pytest.mark.parametrize("power", [19.6, 21.9, 22.3, 23.4, 24.7, 26.2, 27.3, 27.9, 28.6, 31.0, 60.0])
def test_ties_of_large_scores(fmt, dim, sign, heads, power):
    n, at = 2500, [130, 131, 1500, 2499]
    if heads == 1:
        at = [3] + at  # (else the first tile's largest score is a smaller one, and the reference moves)
    c = Cache(fmt, (n,), 1, dim, seed=40)
    for t in range(n):
        set_key(c, t, {1: 768.0 if t > 1 else 896.0, -1: -1536.0 if t > 1 else -1152.0}[sign])
    for t in at:
        set_key(c, t, sign * 1024.0)
    k, v = c.values()
    q = torch.zeros(1, heads, dim, dtype=torch.bfloat16 if fmt == "bf16" else torch.float16)
    q[..., 0] = 1.0
    top = float(np.abs(k[0, 0, at[0], 0]))
    scale = 2.0 ** power / 1.4426950408889634 / top  # base-2 scores of +-2^power
    out, lse, w, err = run(c, heads, [0, 1], [n], q, scale=scale)
    assert err == 0
    want, mag = v[0, 0, at].mean(0), np.abs(v[0, 0, at]).mean(0)
    assert (np.abs(out[0] - want) <= mag * (2.0 ** -SPLIT[fmt] + 2.0 ** -22)).all()
    x = sign * top * float(np.float32(scale))
    assert (np.abs(lse[0] - (x + np.log(len(at)))) <= 2.0 ** -21 * abs(x)).all()
    ww = np.zeros(n)
    ww[at] = heads / len(at)
    assert (np.abs(w[0, 0, :n] - ww) <= heads * 2.0 ** -20).all()
