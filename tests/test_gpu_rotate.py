"""Norm and rotation of query and key heads (qmm_rotate) against a plain implementation in 64 bits.
Tolerance: the normalised value carries the sum of squares' roundings (a tree of 7 additions and E
products, 2^-24 each, halved by the root), rsqrtf's two steps and two products: below 2^-20 relative.  A rotated
one is a sum of two such products, with cosine and sine of an angle that is off by at most 2^-24 of half a turn (3 steps of
fp32 in all): below 2^-20 (|a| + |b|).  Then the output's rounding, half a step."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def rotate_ref(x, weight, pos, inv_freq, axis, interleaved, eps):
    """float64 [rows, heads, dim]; also the magnitudes that the tolerance is made of."""
    y = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    out, mag = y.copy(), np.abs(y)
    n = len(inv_freq)
    for i in range(n):
        t = pos[axis[i]].astype(np.float64) * inv_freq[i]
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
        mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, mag


def case(rows, heads, kvh, dim, rot, src="f32", dst="f16", axes=1, interleaved=False, norm=True, start=0, seed=0, pad=0, eps=1e-6, theta=1e6):
    t = torch_cuda()
    g = torch.Generator().manual_seed(seed)
    y = (torch.randn(rows, (heads + 2 * kvh) * dim + pad, generator=g) * 3).to(TYPES[src])
    w = [1 + 0.3 * torch.randn(dim, generator=g) if norm else None for _ in range(2)]
    n = rot // 2
    inv = (theta ** (-torch.arange(n).double() / max(1, n))).float()
    pos = (start + torch.randint(0, 5000, (axes, rows), generator=g)).to(torch.int32)
    axis = torch.randint(0, axes, (n,), generator=g).to(torch.int32)
    yd = y.cuda()
    q = yd[:, pad:pad + heads * dim].unflatten(1, (heads, dim))
    k = yd[:, pad + heads * dim:pad + (heads + kvh) * dim].unflatten(1, (kvh, dim))
    qo = t.full((rows, heads, dim), 7.0, dtype=TYPES[dst], device="cuda")
    ko = t.full((rows, kvh, dim), 7.0, dtype=TYPES[dst], device="cuda")
    from bit_weight_streaming_q4_gb300 import serve
    serve.rotate(q, k, pos.cuda() if axes > 1 else pos[0].cuda(), inv.cuda(), qo, ko, q_weight=None if w[0] is None else w[0].cuda(),
                 k_weight=None if w[1] is None else w[1].cuda(), axis=axis.cuda() if axes > 1 else None, interleaved=interleaved, eps=eps)
    t.cuda.synchronize()
    ax = axis.numpy() if axes > 1 else np.zeros(n, dtype=np.int64)
    for x, o, wt in ((q, qo, w[0]), (k, ko, w[1])):
        ref, mag = rotate_ref(x.double().cpu().numpy(), None if wt is None else wt.double().numpy(), pos.numpy(), inv.double().numpy(), ax,
                              interleaved, eps)
        got = o.double().cpu().numpy()
        tol = 2.0 ** -20 * mag + HALF[dst] * np.abs(ref) * 1.001 + (2.0 ** -25 if dst == "f16" else 1e-38)
        assert (np.abs(got - ref) <= tol).all(), f"worst {np.max(np.abs(got - ref) / tol):.3f}"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("src,dst", [("f32", "f16"), ("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types(dim, src, dst, interleaved):
    case(5, 6, 2, dim, dim, src, dst, interleaved=interleaved)


@pytest.mark.parametrize("dim,rot", [(64, 0), (64, 16), (64, 48), (128, 32), (128, 96), (256, 64), (256, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_a_head(dim, rot, interleaved):
    case(9, 4, 1, dim, rot, interleaved=interleaved, dst="f32")


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(axes, interleaved):
    case(33, 4, 2, 128, 128, "bf16", "f32", axes=axes, interleaved=interleaved)


@pytest.mark.parametrize("rows", [1, 2, 7, 151, 400, 1000])
@pytest.mark.parametrize("heads,kvh", [(1, 1), (48, 8), (7, 7)])
def test_rows(rows, heads, kvh):
    case(rows, heads, kvh, 128, 128, seed=rows)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("pad", [1, 2, 4])
@pytest.mark.parametrize("src", ["f32", "f16"])
def test_unaligned_rows(norm, pad, src):
    case(11, 6, 2, 64, 64, src, norm=norm, pad=pad)


@pytest.mark.parametrize("start", [-5000, 130_000, 20_000_000, 2 ** 31 - 5001, -(2 ** 31)])
def test_far_positions(start):
    case(6, 4, 2, 128, 128, dst="f32", start=start)


def test_frequencies():
    """Fast, slow and zero ones, and one of many turns a position."""
    for theta in (1.0, 1e-3, 1e9):
        case(6, 2, 1, 64, 64, dst="f32", start=1000, theta=theta)


def test_in_place_one_side_and_zero_heads():
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    g = torch.Generator().manual_seed(2)
    y = torch.randn(40, 10 * 128, generator=g).cuda()
    y[3, :128] = 0  # (a head of zeros stays one)
    inv, pos, w = (1e4 ** (-torch.arange(64) / 64.0)).cuda(), torch.arange(40, dtype=torch.int32).cuda(), torch.rand(128, generator=g).cuda()
    q, k = y[:, :6 * 128].unflatten(1, (6, 128)), y[:, 6 * 128:8 * 128].unflatten(1, (2, 128))
    qo, ko = t.empty(40, 6, 128, device="cuda"), t.empty(40, 2, 128, device="cuda")
    serve.rotate(q, k, pos, inv, qo, ko, q_weight=w)  # (k is not normalised)
    q1, k1 = t.empty_like(qo), t.empty_like(ko)
    serve.rotate(q, None, pos, inv, q1, None, q_weight=w)
    serve.rotate(None, k, pos, inv, None, k1)
    assert t.equal(q1, qo) and t.equal(k1, ko) and bool((qo[3, 0] == 0).all())
    rest = y[:, 8 * 128:].clone()
    serve.rotate(q, k, pos, inv, q, k, q_weight=w)
    assert t.equal(q, qo) and t.equal(k, ko) and t.equal(y[:, 8 * 128:], rest)
    with pytest.raises(ValueError):
        serve.rotate(q, k, pos[:39], inv, qo, ko)
    with pytest.raises(ValueError):
        serve.rotate(q, None, pos, inv, qo, ko)
    with pytest.raises(ValueError):
        serve.rotate(q, k.half(), pos, inv, qo, ko)


def test_rows_do_not_depend_on_company_and_graphs():
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    g = torch.Generator().manual_seed(3)
    x = torch.randn(900, 8, 128, generator=g).cuda()
    inv, w = (1e6 ** (-torch.arange(64) / 64.0)).cuda(), torch.rand(128, generator=g).cuda()
    pos = torch.arange(900, dtype=torch.int32).cuda()
    out, one = t.empty(900, 8, 128, dtype=t.float16, device="cuda"), t.empty(1, 8, 128, dtype=t.float16, device="cuda")
    serve.rotate(x, None, pos, inv, out, None, q_weight=w)
    for r in (0, 501, 899):
        serve.rotate(x[r:r + 1], None, pos[r:r + 1], inv, one, None, q_weight=w)
        assert t.equal(one[0], out[r])
    graph, dst = t.cuda.CUDAGraph(), t.empty_like(out)
    with t.cuda.graph(graph):
        serve.rotate(x, None, pos, inv, dst, None, q_weight=w)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    dst.zero_()
    t.cuda.synchronize()
    graph.replay()
    other = t.empty_like(out)
    serve.rotate(x, None, pos, inv, other, None, q_weight=w, stream=s.cuda_stream)
    t.cuda.synchronize()
    assert t.equal(dst, out) and t.equal(other, out)


def test_no_rows_and_numbers_that_are_none():
    t = torch_cuda()
    from bit_weight_streaming_q4_gb300 import serve
    inv = torch.ones(32).cuda()
    e = t.empty(0, 2, 64, device="cuda")
    serve.rotate(e, None, t.empty(0, dtype=t.int32, device="cuda"), inv, e, None)
    x = torch.ones(2, 2, 64).cuda()
    x[0, 1, 5] = float("nan")
    out = t.empty_like(x)
    serve.rotate(x, None, t.zeros(2, dtype=t.int32, device="cuda"), inv, out, None, q_weight=torch.ones(64).cuda())
    assert bool(out[0, 1].isnan().all()) and bool(out[0, 0].isfinite().all()) and bool(out[1].isfinite().all())
