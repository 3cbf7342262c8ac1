"""The shapes that the binding of the log probabilities takes (no GPU: stand-in tensors)."""
import pytest

from test_serve_devices import F32, I32, Tensor, here  # noqa: F401  (a fixture)
from bit_weight_streaming_q4_gb300 import serve as S


@pytest.mark.parametrize("names,dtypes", [(("tokens", "logprob"), (I32, F32)), (("top_index", "top_logprob"), (I32, F32))])
@pytest.mark.parametrize("a,b", [((6,), (6,)), ((3,), (3,)), ((2, 3), (2, 3)), ((3, 2), (2, 3)), ((3, 2), (6,)), ((3, 2, 1), (3, 2, 1)), ((1, 6), (1, 6))])
def test_pairs_of_other_shapes_are_refused(here, names, dtypes, a, b):  # noqa: F811
    _, calls, _ = here
    kw = {n: Tensor(t, *s) for n, t, s in zip(names, dtypes, (a, b))}
    with pytest.raises(ValueError, match=f"^{names[0]} and {names[1]}:"):
        S.logprobs(Tensor(F32, 3, 50), **kw)
    assert not calls


def test_pairs_that_fit_are_taken(here):  # noqa: F811
    _, calls, _ = here
    S.logprobs(Tensor(F32, 3, 50), Tensor(I32, 3, 0), logprob=Tensor(F32, 3, 0), top_index=Tensor(I32, 3, 32), top_logprob=Tensor(F32, 3, 32))
    S.logprobs(Tensor(F32, 0, 50), Tensor(I32, 0, 2), logprob=Tensor(F32, 0, 2))
    assert [c[6:8] for c in calls] == [(0, 32), (2, 0)]
