"""Log probabilities, entropy and top alternatives (qmm_logprobs) against numpy in 64 bits.

Tolerances: the terms of the sums are off by the exponential's error and the rounding of its
argument, at most 2^-21 of the sums in all; a sum passes fewer than 80 additions per thread
and merge (32 a round, then 5 + 15 + 7 merges), so 2^-17 bounds its relative error and
that of ln Z absolutely; the entropy's second sum has terms p d, its error is as large times
(1 + entropy); every result is then rounded once."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
SUM = 2.0 ** -17


def run(x, tokens=None, top=0):
    from bit_weight_streaming_q4_gb300 import serve
    t = torch_cuda()
    m, n = x.shape
    o = {k: t.full((m,), 7.0, device="cuda") for k in ("lse", "entropy")}
    given = None if tokens is None else t.tensor(tokens, dtype=t.int32, device="cuda")
    lp = None if tokens is None else t.full(given.shape, 7.0, device="cuda")
    ti = t.full((m, top), -5, dtype=t.int32, device="cuda") if top else None
    tl = t.full((m, top), 7.0, device="cuda") if top else None
    serve.logprobs(x, given, o["lse"], lp, o["entropy"], ti, tl)
    t.cuda.synchronize()
    o.update(logprob=lp, top_index=ti, top_logprob=tl)
    return {k: None if v is None else v.cpu().numpy().astype(np.int64 if k == "top_index" else np.float64) for k, v in o.items()}


def check(x, tokens=None, top=0, dev=None):
    """x: CPU tensor [m, n]; rows of finite values and -infinity, not all -infinity."""
    got = run(x.cuda() if dev is None else dev, tokens, top)
    a = x.double().numpy()
    m = a.max(-1, keepdims=True)
    e = np.exp(a - m)
    z = e.sum(-1, keepdims=True)
    lse = (m + np.log(z))[:, 0]
    with np.errstate(invalid="ignore"):
        h = np.log(z[:, 0]) - np.where(e > 0, e * (a - m), 0).sum(-1) / z[:, 0]
    assert (np.abs(got["lse"] - lse) <= SUM + 2.0 ** -23 * np.abs(lse)).all()
    assert (np.abs(got["entropy"] - h) <= SUM * (1 + h) + 2.0 ** -23 * h).all() and (got["entropy"] >= 0).all()
    lp = a - lse[:, None]

    def near(y, want):
        inf = np.isneginf(want)
        assert np.array_equal(np.isneginf(y), inf)
        assert (np.abs(y[~inf] - want[~inf]) <= SUM + 2.0 ** -22 * np.abs(want[~inf])).all()
    if tokens is not None:
        near(got["logprob"], np.take_along_axis(lp, np.asarray(tokens), 1))
    if top:
        order = np.argsort(-a, axis=-1, kind="stable")[:, :top]
        assert np.array_equal(got["top_index"], order)
        near(got["top_logprob"], np.take_along_axis(lp, order, 1))
    return got


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 511, 4096, 4097, 16385, 50257, 151936, 300001])
@pytest.mark.parametrize("kind", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])
def test_logprobs_matches_plain(n, kind):
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(3, n, generator=g) * 2.5).to(kind)
    check(x, torch.randint(0, n, (3, 2), generator=g).tolist(), min(n, 20))


@pytest.mark.parametrize("top", [1, 2, 5, 31, 32])
def test_logprobs_top(top):
    g = torch.Generator().manual_seed(top)
    check(torch.randn(5, 20011, generator=g) * 3, None, top)


def data(kind, n, seed=0):
    rng = np.random.default_rng(seed)
    x = {"equal": lambda: np.zeros(n), "rising": lambda: np.arange(n) * 1e-3, "falling": lambda: -np.arange(n) * 1e-3,
         "two": lambda: rng.integers(0, 2, n) * 1.0, "zeros": lambda: rng.choice([0.0, -0.0], n),
         "peak": lambda: np.where(np.arange(n) == n // 3, 80.0, rng.standard_normal(n)),
         "huge": lambda: rng.standard_normal(n) * 1e30, "tiny": lambda: rng.standard_normal(n) * 1e-30,
         "masked": lambda: np.where(rng.random(n) < 0.97, -np.inf, rng.standard_normal(n)),
         "lowest": lambda: np.where(rng.random(n) < 0.6, np.finfo(np.float32).min, rng.standard_normal(n)),
         # every large value in the same thread's share, and in a handful of threads'
         "one thread": lambda: np.where(np.arange(n) // 4 % 512 == 77, 5.0, 0.0) + rng.random(n),
         "few threads": lambda: np.where(np.arange(n) // 4 % 512 < 70, 5.0, 0.0) + rng.random(n)}[kind]()
    return torch.from_numpy(x[None].astype(np.float32))


@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two", "zeros", "peak", "huge", "tiny", "masked", "lowest", "one thread",
                                  "few threads"])
@pytest.mark.parametrize("n", [700, 151936, 200003])
def test_logprobs_hard_rows(kind, n):
    check(data(kind, n), [[0, n // 3, n - 1]], 32)


def test_logprobs_only_one_column_left():
    x = torch.full((2, 40000), -torch.inf)
    x[0, 39999] = -3.0
    x[1, 5] = 1e38
    got = check(x, [[39999, 0], [5, 6]], 3)
    assert (got["logprob"][:, 0] == 0).all() and (got["entropy"] == 0).all()


def test_logprobs_rows_without_a_distribution():
    """Nothing but -infinity; NaN; +infinity: each as documented, and no effect on other rows."""
    x = torch.randn(5, 30000)
    x[1] = -torch.inf
    x[2, 29999] = torch.nan
    x[3, 17] = torch.inf
    got = run(x.cuda(), [[1, 29999]] * 5, 7)
    fine = run(x[[0, 4]].cuda(), [[1, 29999]] * 2, 7)
    for k, v in fine.items():
        assert np.array_equal(got[k][[0, 4]], v)
    assert np.isneginf(got["lse"][1]) and got["entropy"][1] == 0 and np.isneginf(got["logprob"][1]).all()
    assert np.isneginf(got["top_logprob"][1]).all() and got["top_index"][1].tolist() == list(range(7))
    for r in (2, 3):
        assert all(np.isnan(got[k][r]).all() for k in ("lse", "entropy", "logprob", "top_logprob")) and (got["top_index"][r] == -1).all()


def test_logprobs_tokens_out_of_range():
    got = run(torch.randn(1, 1000).cuda(), [[-1, 0, 1000, 999, -(1 << 31), (1 << 31) - 1]])
    assert np.isnan(got["logprob"][0]).tolist() == [True, False, True, False, True, True]


@pytest.mark.parametrize("kind", [torch.float32, torch.float16], ids=["f32", "f16"])
def test_logprobs_strides_and_alignment(kind):
    t = torch_cuda()
    wide = (torch.randn(7, 5003) * 2).to(kind)
    for lo, hi in ((0, 5000), (1, 4099), (3, 5003)):
        check(wide[:, lo:hi], [[0]] * 7, 4, dev=wide.cuda()[:, lo:hi])


def test_logprobs_rows_do_not_depend_on_the_call():
    x = torch.randn(40, 151936).cuda() * 2
    full, one = run(x, [[5]] * 40, 10), run(x[17:18], [[5]], 10)
    for k, v in one.items():
        assert np.array_equal(full[k][17:18], v)


def test_logprobs_of_the_argmax_match_the_lm_head():
    """The first alternative of a matmul's output is qmm_run_argmax's column."""
    import synth
    from gpu_util import make
    t = torch_cuda()
    n, k, m = 3001, 512, 6
    q = make(synth.q4k_matrix(n, k, seed=3, tensor_id=9), m_max=m)
    x = t.from_numpy(synth.x_f16(m, k, seed=3, tensor_id=10).view(np.int16)).cuda().view(t.float16)
    y, idx, val = t.empty(m, n, device="cuda"), t.empty(m, dtype=t.int32, device="cuda"), t.empty(m, device="cuda")
    q.run(x, y, m)
    q.run_argmax(x, idx, val, m)
    got = run(y, None, 1)
    assert np.array_equal(got["top_index"][:, 0], idx.cpu().numpy())
    q.close()


def test_logprobs_none_of_the_outputs_and_no_rows():
    from bit_weight_streaming_q4_gb300 import serve
    t = torch_cuda()
    x = t.randn(3, 999, device="cuda")
    serve.logprobs(x)
    serve.logprobs(x[:0])
    lse = t.empty(3, device="cuda")
    serve.logprobs(x, lse=lse)
    t.cuda.synchronize()
    assert np.allclose(lse.cpu().numpy(), t.logsumexp(x.double(), -1).cpu().numpy(), atol=2.0 ** -16)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_logprobs_many_candidates_per_block(kind):
    """Hundreds of rows: a block has many segments, and 32 alternatives let some 80 elements of each pass."""
    t = torch_cuda()
    g = t.Generator(device="cuda").manual_seed(2)
    x = (t.randn(320, 151936, generator=g, device="cuda") * 2.5).to(kind)
    got = run(x, top=32)
    order = t.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :32].cpu().numpy()
    assert np.array_equal(got["top_index"], order)
