"""Verification where probabilities are next to nothing: what the header says of 2^-1000 and of 2^-45 of a row's largest."""
import math

import pytest
import torch

from test_gpu_verify import call

pytestmark = pytest.mark.gpu


def decide(p, q, draft, u=0.5, sample=0.25):
    """Two rows, of which the second's draft is judged by p and q."""
    x, d = torch.tensor([p, p]), torch.tensor([q, q])
    acc, tok, prob, err = call(x, d, [0, 2], torch.tensor([0, draft]), None, torch.tensor([0.0, u]), torch.tensor([sample]))
    assert err == 0
    return acc[0], tok[0], float(prob[1])


def test_drafts_are_judged_down_to_2_to_the_minus_1000():
    assert decide([0.0, -690.0, -1.0], [0.0, -690.0, -1.0], 1) == (1, 0, 1.0)  # 2^-995: p = q, taken
    assert decide([0.0, -694.0, -1.0], [0.0, -694.0, -1.0], 1) == (0, 0, 0.0)  # 2^-1001: counts as 0, refused, and drawn from p
    acc, _, prob = decide([0.0, -600.0], [0.0, -599.0], 1, u=0.3)
    assert acc == 1 and abs(prob - math.exp(-1)) <= 2.0 ** -23.9 * prob  # (0.3 < p / q)
    assert decide([0.0, -600.0], [0.0, -599.0], 1, u=0.4)[0] == 0


def test_an_empty_rest_is_drawn_from_p():
    # max(p - q, 0) is 2^-51 at the first column alone: nothing is left of it, so the next token is p's, a number of 0.6 the last's
    p, q = [0.0, -40.0, 0.0], [0.0, -35.0, 0.0]
    assert decide(p, q, 1, sample=0.25)[:2] == (0, 0)
    assert decide(p, q, 1, sample=0.6)[:2] == (0, 2)


@pytest.mark.parametrize("row", [[-math.inf, -math.inf], [0.0, math.nan], [0.0, 1.0]])
def test_a_draft_row_without_a_distribution_refuses_whatever_judges_it(row):
    acc, tok, prob = decide(row, [0.0, math.inf], 0)
    assert acc == 0 and math.isnan(prob)
    assert tok == (0 if row[1] == 1.0 else -1)
