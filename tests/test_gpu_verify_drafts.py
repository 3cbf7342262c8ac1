"""Verification: draft rows that do not count."""
import pytest
import torch

from gpu_util import torch_cuda
from test_gpu_verify import call, make, verify_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [100, 9001])
def test_first_draft_rows_lie_in_front_of_the_memory(kind, n):
    """A sequence's first draft row is not read, so draft_logits may begin one row before what the caller has."""
    x, d, ar, tok, au, su = make(1, 5, n, kind, seed=3)
    d[0] = float("nan")
    acc, token, prob, err = call(x, d, ar, tok, None, au, su)
    wa, wt, _, near = verify_ref(x, d, ar, tok, [1.0], au, su)
    assert err == 0 and near[0] > 2.0 ** -32 and (acc, token) == (wa, wt)
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    kept = d[1:].cuda()  # (rows 1 .. 4 alone; the base handed over lies a row in front)
    plan = serve.VerifyPlan(agents=1, max_rows=5, columns=n)
    xd, a, b, p = x.cuda(), i32([9]), i32([9]), t.zeros(5, device="cuda")
    args = (i32(ar), 1, 5, tok.int().cuda(), None, au.cuda(), su.cuda(), a, b, p)
    stream = plan._on(None)
    status = plan._verify(xd.data_ptr(), serve._types[xd.dtype], n, n, kept.data_ptr() - n * kept.element_size(), n,
                          *[v.data_ptr() if torch.is_tensor(v) else v for v in args], plan._workspace.data_ptr(), plan._bytes,
                          plan.error_word.data_ptr(), stream)
    t.cuda.synchronize()
    assert status == 0 and plan.error() == 0
    assert (a.tolist(), b.tolist()) == (acc, token) and torch.equal(p.double().cpu(), prob)


def test_draft_rows_of_greedy_sequences_do_not_count():
    x, d, ar, tok, au, su = make(6, 4, 3001, seed=4)
    tok[1:] = x[:-1].argmax(-1)
    tok[ar[3] + 2] = 5
    temperature = [0.0, 1.0, 0.0, 0.0, 0.7, float("nan")]
    want = call(x, d, ar, tok, temperature, au, su)
    for a in (0, 2, 3, 5):
        d[ar[a]:ar[a + 1]] = float("nan")
    got = call(x, d, ar, tok, temperature, au, su)
    assert got[0] == want[0] and got[1] == want[1] and got[3] == 0 and torch.equal(got[2], want[2])
    assert got[0][0] == 3 and got[0][3] == 1
