"""Windowed attention with a scale of 0, or next to it, over scores near fp32's end: every token that a row sees weighs the same.

Scores reach 2^127; times a scale of 2^-149 (fp32's smallest) they are 2^-21 at most, which moves a weight by 2^-21, and the
probabilities are rounded once to bf16 (2^-8), all of a row's next to the same number; sums take 2^-20."""
import numpy as np
import pytest
import torch

from kv_util import Cache
from test_gpu_kv_window import PRODUCT, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_all_weigh_the_same(dim, rows, scale):
    heads, n, window = 4, 300, 200
    c = Cache("bf16", (n,), 1, dim, 64, seed=43)
    c.pool[:, :, 0] = 0
    c.pool[:, :, 0, :, 0] = torch.where(torch.arange(64) % 3 == 0, 2.0 ** 63, -2.0 ** 62).to(torch.bfloat16)
    q = torch.zeros(rows, heads, dim, dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** 63
    _, v = c.values()
    rl = [n - j for j in range(rows)]
    out, lse, err = run(c, heads, [0, rows], rl, q, window, 0, scale=scale)
    assert err == 0
    for r in range(rows):
        seen = v[0, 0, rl[r] - window:rl[r]]
        tol = np.abs(seen).mean(0) * (PRODUCT["bf16"] * 1.001 + 2.0 ** -18)
        assert (np.abs(out[r] - seen.mean(0)) <= tol).all()
        assert (np.abs(lse[r] - np.log(window)) <= 2.0 ** -18).all()
