"""The serving binding keeps a call on one device, the current one (no GPU: the tensors are stand-ins, and the
library's entries must not be reached)."""
import pytest
import torch

from bit_weight_streaming_q4_gb300 import build as qbuild
from bit_weight_streaming_q4_gb300 import serve as S


class Tensor:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.at = dtype, shape, device
        self.device, self.is_cuda = torch.device("cpu"), device >= 0

    def get_device(self):
        return self.at

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self):
        st, n = [], 1
        for s in reversed(self.shape):
            st.insert(0, n)
            n *= s
        return tuple(st)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def here(monkeypatch):
    """The current device, and the library's entries recorded."""
    qbuild.build()
    S._setup()
    calls, now = [], [0]
    monkeypatch.setattr(S, "_here", lambda: now[0])
    monkeypatch.setattr(S, "_raw", lambda d: 0x99)
    plan = S.KvPlan(Tensor(torch.int32, 2, 3), format="f16", heads=4, kv_heads=2, head_dim=64, page_tokens=16, pool_pages=6, max_rows=3)
    plan._on = lambda stream: 0x99
    plan._space = lambda kind, stream: (0x10000, 1 << 40, None)
    plan._append = plan._attend = plan._evict = lambda *a: calls.append(a) or 0
    monkeypatch.setattr(S, "load", lambda: type("Lib", (), {"qmm_logprobs": staticmethod(plan._append)}))
    return now, calls, plan


I32, F32, F16 = torch.int32, torch.float32, torch.float16
SLOTS = (2, 2, 48)


def arguments(kind):
    a = {"pool": (F16, 6, 2, 2, 16, 64)}
    if kind == "attend":
        a.update(agent_rows=(I32, 3), row_len=(I32, 3), q=(F16, 3, 4, 64), out=(F32, 3, 4, 64), lse=(F32, 3, 4), weight_in=(F32, *SLOTS),
                 weight_out=(F32, *SLOTS))
    elif kind == "append":
        a.update(agent_rows=(I32, 3), cache_len=(I32, 2), k=(F32, 3, 2, 64), v=(F32, 3, 2, 64), weight=(F32, *SLOTS), pos=(I32, *SLOTS),
                 row_pos=(I32, 3))
    elif kind == "evict":
        a.update(cache_len=(I32, 2), keep=(I32, 2), weight=(F32, *SLOTS), pos=(I32, *SLOTS), weight_out=(F32, *SLOTS), pos_out=(I32, *SLOTS),
                 len_out=(I32, 2), protect_from=(I32, 2))
    else:
        a = dict(logits=(F32, 3, 50), tokens=(I32, 3, 2), logprob=(F32, 3, 2), lse=(F32, 3), entropy=(F32, 3), top_index=(I32, 3, 4),
                 top_logprob=(F32, 3, 4))
    return a


@pytest.mark.parametrize("kind", ["attend", "append", "evict", "logprobs"])
def test_every_tensor_is_on_the_plans_device(here, kind):
    now, calls, plan = here
    call = S.logprobs if kind == "logprobs" else getattr(plan, kind)
    args = arguments(kind)
    call(**{n: Tensor(*v) for n, v in args.items()})
    assert len(calls) == 1
    for name in args:
        if name == "logits":
            continue  # (its device is the call's)
        for device in (1, -1):
            with pytest.raises(ValueError, match=f"^{name}:"):
                call(**{n: Tensor(*v, device=device if n == name else 0) for n, v in args.items()})
    now[0] = 1  # all on device 0, but the library would launch on 1
    with pytest.raises(ValueError, match="^device:"):
        call(**{n: Tensor(*v) for n, v in args.items()})
    assert len(calls) == 1
