"""The binding keeps calls of rotation, windowed attention and verification on one device, the current one (no GPU: the
tensors are stand-ins, and the library's entries must not be reached)."""
import pytest
import torch

from bit_weight_streaming_q4_gb300 import build as qbuild
from bit_weight_streaming_q4_gb300 import serve as S
from test_serve_devices import Tensor

I32, F32, F16 = torch.int32, torch.float32, torch.float16


@pytest.fixture
def here(monkeypatch):
    qbuild.build()
    S._setup()
    calls, now = [], [0]
    monkeypatch.setattr(S, "_here", lambda: now[0])
    monkeypatch.setattr(S, "_raw", lambda d: 0x99)
    reached = staticmethod(lambda *a: calls.append(a) or 0)
    plan = S.KvPlan(Tensor(I32, 2, 3), format="f16", heads=4, kv_heads=2, head_dim=64, page_tokens=16, pool_pages=6, max_rows=3)
    plan._on = lambda stream: 0x99
    plan._space = lambda kind, stream: (0x10000, 1 << 40, None)
    plan._attend_window = reached.__func__
    judge = S.VerifyPlan(agents=2, max_rows=4, columns=50, device="cpu")
    judge.device = 0
    judge._on = lambda stream: 0x99
    judge._workspace = torch.empty(16)
    judge._verify = reached.__func__
    monkeypatch.setattr(S, "load", lambda: type("Lib", (), {"qmm_rotate": reached}))
    return now, calls, plan, judge


def arguments(kind):
    if kind == "rotate":
        return dict(q=(F32, 3, 4, 64), k=(F32, 3, 2, 64), pos=(I32, 3), inv_freq=(F32, 32), q_out=(F16, 3, 4, 64), k_out=(F32, 3, 2, 64),
                    q_weight=(F32, 64), k_weight=(F32, 64), axis=(I32, 32))
    if kind == "attend_window":
        return dict(pool=(F16, 6, 2, 2, 16, 64), agent_rows=(I32, 3), row_len=(I32, 3), q=(F16, 3, 4, 64), out=(F32, 3, 4, 64), lse=(F32, 3, 4))
    return dict(logits=(F32, 4, 50), agent_rows=(I32, 3), tokens=(I32, 4), accept_u=(F32, 4), sample_u=(F32, 2), accepted=(I32, 2), token=(I32, 2),
                draft_logits=(F32, 4, 50), temperature=(F32, 2), prob=(F32, 4))


@pytest.mark.parametrize("kind", ["rotate", "attend_window", "verify"])
def test_every_tensor_is_on_one_device(here, kind):
    now, calls, plan, judge = here
    call = S.rotate if kind == "rotate" else judge.verify if kind == "verify" else plan.attend_window
    more = {"window": 9} if kind == "attend_window" else {}
    args = arguments(kind)
    call(**{n: Tensor(*v) for n, v in args.items()}, **more)
    assert len(calls) == 1
    for name in args:
        for device in (1, -1):
            if kind == "rotate" and name == "q":
                continue  # (its device is the call's)
            with pytest.raises(ValueError, match=f"^{name}"):
                call(**{n: Tensor(*v, device=device if n == name else 0) for n, v in args.items()}, **more)
    now[0] = 1  # all on device 0, but the library would launch on 1
    with pytest.raises(ValueError, match="^device:"):
        call(**{n: Tensor(*v) for n, v in args.items()}, **more)
    assert len(calls) == 1


def test_shapes_and_types(here):
    _, calls, plan, judge = here
    for kind, call, bad in (
            ("rotate", S.rotate, dict(k=(F16, 3, 2, 64), q_out=(F16, 3, 3, 64), k_out=(F32, 2, 2, 64), pos=(I32, 2, 2, 3), q_weight=(F32, 63),
                                      axis=(I32, 31))),
            ("attend_window", lambda **a: plan.attend_window(window=4, **a),
             dict(pool=(F32, 6, 2, 2, 16, 64), agent_rows=(I32, 2), row_len=(I32, 4), q=(F32, 3, 4, 64), out=(F32, 3, 4, 63), lse=(F32, 3, 3))),
            ("verify", judge.verify, dict(logits=(F32, 4, 49), tokens=(I32, 3), accept_u=(F16, 4), sample_u=(F32, 4), accepted=(F32, 2),
                                          token=(I32, 1), draft_logits=(F16, 4, 50), temperature=(F32, 4), prob=(F32, 2)))):
        args = arguments(kind)
        for name, value in bad.items():
            with pytest.raises(ValueError):
                call(**{n: Tensor(*v) for n, v in {**args, name: value}.items()})
    with pytest.raises(ValueError, match="max_rows"):
        plan.attend_window(Tensor(F16, 6, 2, 2, 16, 64), Tensor(I32, 3), Tensor(I32, 4), Tensor(F16, 4, 4, 64), Tensor(F32, 4, 4, 64), window=4)
    assert not calls
