"""ctypes binding of the serving operators (include/qmm_serve.h): argument checks and marshalling.

``KvPlan`` holds what a serving program sets up once for a paged KV cache -- its dims, the page
table, the workspace and the error word -- and appends to the cache, attends over it and evicts
from it; ``logprobs`` reads the lm_head's output.  As in ``qmm``, every step runs in the library's
CUDA kernels, there is no fallback, and PyTorch supplies only device memory and streams.  Calls go
to the current stream unless ``stream`` is given; a tensor last written on another stream has to be
ordered before them by the caller.  All tensors of a call are on one device, the current one.

A small call takes about as long here as on the GPU, so the checks below are plain comparisons and
form their messages only to raise them."""
from __future__ import annotations

import ctypes
import os
import re

from . import qmm as _q

HEADER = os.path.join(os.path.dirname(_q.HEADER), "qmm_serve.h")

FORMATS = {"q8_0": 0, "f16": 1, "bf16": 2}
TYPE_F32, TYPE_F16, TYPE_BF16 = 0, 1, 2


class KvDims(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("agents", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("max_agent_rows", ctypes.c_int32), ("pool_pages", ctypes.c_int64)]


def header_functions() -> list[str]:
    """Names of the functions declared in include/qmm_serve.h."""
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*qmm_status\s+(qmm_\w+)\s*\(", text, flags=re.M)))


_lib = None


def load():
    """libqmm.so with the serving operators' signatures set."""
    global _lib
    if _lib is None:
        lib = _q.load()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        dims = ctypes.POINTER(KvDims)
        for name, args in {
                "qmm_kv_append": [dims, vp, vp, vp, vp, vp, i64, vp, i64, i32, i64, vp, vp, vp, vp, vp],
                "qmm_kv_attend_workspace_bytes": [dims, i32, ctypes.POINTER(i64)],
                "qmm_kv_attend": [dims, vp, vp, vp, vp, vp, i64, i64, f32, vp, i32, vp, vp, vp, vp, i64, vp, vp],
                "qmm_kv_evict_workspace_bytes": [dims, ctypes.POINTER(i64)],
                "qmm_kv_evict": [dims, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp],
                "qmm_logprobs": [vp, i32, i64, i64, i64, vp, i32, i32, vp, vp, vp, vp, vp, vp]}.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = ctypes.c_int, args
        _lib = lib
    return _lib


_torch = _f32 = _i32 = _types = _raw = _here = None


def _setup():
    """torch and its types, looked up at the first use (the module imports without torch)."""
    global _torch, _f32, _i32, _types, _raw, _here
    import torch
    # (the handle alone, without the Stream object around it: 0.1 us instead of 3)
    _raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
    _here = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _f32, _i32 = torch.float32, torch.int32
    _types = {torch.float32: TYPE_F32, torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16}
    _torch = torch


def _refuse(name, what):
    raise ValueError(f"{name}: {what}")


def _vector(name, t, dtype, n, device):
    """Address of a contiguous CUDA tensor of n elements on a device."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != device:
        _refuse(name, f"a contiguous {dtype} CUDA tensor of {n} elements on device {device}")
    return t.data_ptr()


def _current(device):
    """The library launches on the current device: it has to be the tensors'."""
    if _here() != device:
        _refuse("device", f"the tensors are on {device}, the current device is {_here()}")


class KvPlan:
    """A paged KV cache of one layer: the dims, the page table, the workspace and the error word.

    page_table: int32 CUDA tensor [agents, max_pages], contiguous; its entries may be rewritten
    between calls.  format: "q8_0" (the pool of qmm_attn_decode: head_dim 128, page_tokens 64),
    "f16" or "bf16" (head_dim 64, 128 or 256, page_tokens 16 .. 256).  The pool is passed to each
    call, so that layers can share a plan: a uint8 tensor of pool_pages * kv_heads * 17,408 bytes,
    or a 16-bit one of pool_pages * kv_heads * 2 * page_tokens * head_dim elements.
    max_rows / max_agent_rows bound the rows of an attend call, and those of one sequence.
    Calls of one plan share its workspace: those on different streams have to be ordered by the caller.
    A workspace is allocated at the first call that needs it, as memory of that call's stream, and
    goes back to the allocator behind the work of every stream that calls went to; a stream that is
    handed to a call has to outlive the plan."""

    def __init__(self, page_table, *, format: str, heads: int, kv_heads: int, head_dim: int, page_tokens: int,
                 pool_pages: int, max_rows: int, max_agent_rows: int | None = None):
        if _torch is None:
            _setup()
        if page_table.dtype is not _i32 or page_table.dim() != 2 or not page_table.is_contiguous() or not page_table.is_cuda:
            _refuse("page_table", "a contiguous int32 CUDA tensor [agents, max_pages]")
        if format not in FORMATS:
            _refuse("format", f"one of {', '.join(FORMATS)}")
        agents, max_pages = page_table.shape
        self.page_table, self.format, self.max_rows = page_table, format, int(max_rows)
        self.dims = KvDims(FORMATS[format], heads, kv_heads, head_dim, page_tokens, agents, max_pages,
                           int(max_agent_rows or max_rows), pool_pages)
        self.agents, self.heads, self.kv_heads, self.head_dim = agents, heads, kv_heads, head_dim
        self.device = page_table.get_device()
        self.cap = max_pages * page_tokens
        self._slots = agents * kv_heads * self.cap
        self._ref = ctypes.byref(self.dims)
        self._pool_dtype = {"q8_0": _torch.uint8, "f16": _torch.float16, "bf16": _torch.bfloat16}[format]
        self._q_dtype = _torch.bfloat16 if format == "bf16" else _torch.float16
        self._pool_size = pool_pages * kv_heads * (17408 if format == "q8_0" else 2 * page_tokens * head_dim)
        self._scale = head_dim ** -0.5
        # (a copy from the host: it is there, on any stream, when the constructor returns)
        self.error_word = _torch.tensor([0], dtype=_i32, device=page_table.device)
        self._err, self._table = self.error_word.data_ptr(), page_table.data_ptr()
        self._workspace = {}
        self._streams = {}  # handles of the calls' streams, and the streams as torch knows them
        lib = load()
        self._append, self._attend, self._evict = lib.qmm_kv_append, lib.qmm_kv_attend, lib.qmm_kv_evict
        self._bytes("qmm_kv_evict_workspace_bytes")  # refuses dims that no call takes

    def _bytes(self, name, *args) -> int:
        n = ctypes.c_int64()
        _q._check(getattr(load(), name)(self._ref, *args, ctypes.byref(n)), name)
        return n.value

    def _on(self, stream: int | None) -> int:
        """The call's stream, of which the allocator is told at its first call."""
        if stream is None:
            stream = _raw(self.device)
        if stream not in self._streams:
            device = self.page_table.device
            s = _torch.cuda.ExternalStream(stream, device) if stream else _torch.cuda.default_stream(device)
            for t in [self.error_word] + [w[2] for w in self._workspace.values()]:
                t.record_stream(s)
            self._streams[stream] = s
        return stream

    def _space(self, kind: str, stream: int):
        """Address and bytes of a kind of call's workspace, allocated for the stream of its first use and kept."""
        w = self._workspace.get(kind)
        if w is None:
            n = self._bytes("qmm_kv_evict_workspace_bytes") if kind == "evict" else \
                self._bytes("qmm_kv_attend_workspace_bytes", int(kind == "weights"))
            # (not for torch's current stream, whose pending work may still use the block that it gets)
            with _torch.cuda.stream(self._streams[stream]):
                t = _torch.empty(n, dtype=_torch.uint8, device=self.page_table.device)
            for s in self._streams.values():
                t.record_stream(s)
            w = self._workspace[kind] = (t.data_ptr(), n, t)
        return w

    def _pool(self, pool) -> int:
        _current(self.device)
        if pool.dtype is not self._pool_dtype or pool.numel() != self._pool_size or not pool.is_contiguous() or \
                pool.get_device() != self.device:
            _refuse("pool", f"a contiguous {self._pool_dtype} CUDA tensor of {self._pool_size} elements on device {self.device}")
        return pool.data_ptr()

    def _vector(self, name, t, dtype, n) -> int:
        return _vector(name, t, dtype, n, self.device)

    def _rows_of(self, name, t, dtype, heads):
        """Address and row stride of [rows, heads, head_dim] with any row stride."""
        s = t.shape
        if len(s) != 3 or s[1] != heads or s[2] != self.head_dim or t.dtype is not dtype or t.get_device() != self.device:
            _refuse(name, f"a {dtype} CUDA tensor [rows, {heads}, {self.head_dim}] on device {self.device}")
        st = t.stride()
        if s[0] > 0 and (st[2] != 1 or (heads > 1 and st[1] != self.head_dim)):
            _refuse(name, "contiguous but for the row stride")
        # (a single row's stride says nothing)
        return t.data_ptr(), st[0] if s[0] > 1 else heads * self.head_dim

    def append(self, pool, agent_rows, cache_len, k, v, *, weight=None, pos=None, row_pos=None, stream: int | None = None) -> None:
        """Write K and V of new rows behind the sequences' cached tokens (qmm_kv_append).

        k, v: fp32, fp16 or bf16 [rows, kv_heads, head_dim], any row stride (columns of the qkv
        projection's output are taken in place).  cache_len: int32 [agents], tokens cached
        before the call (not changed).  weight / pos: the slots' arrays, whose new entries become
        0 and row_pos.  No other sequence may share the pages that are written to."""
        at = self._pool(pool)
        kind = _types.get(k.dtype)
        if kind is None:
            _refuse("k", "fp32, fp16 or bf16")
        kp, ks = self._rows_of("k", k, k.dtype, self.kv_heads)
        vp, vs = self._rows_of("v", v, k.dtype, self.kv_heads)
        rows = k.shape[0]
        if v.shape[0] != rows:
            _refuse("v", f"{rows} rows, as k")
        st = self._append(
            self._ref, at, self._table, self._vector("agent_rows", agent_rows, _i32, self.agents + 1),
            self._vector("cache_len", cache_len, _i32, self.agents), kp, ks, vp, vs, kind, rows,
            0 if weight is None else self._vector("weight", weight, _f32, self._slots),
            0 if pos is None else self._vector("pos", pos, _i32, self._slots),
            0 if row_pos is None else self._vector("row_pos", row_pos, _i32, rows), self._err, self._on(stream))
        if st:
            raise _q.QmmError(st, "qmm_kv_append")

    def attend(self, pool, agent_rows, row_len, q, out, *, lse=None, weight_in=None, weight_out=None,
               scale: float | None = None, stream: int | None = None) -> None:
        """Attention of new tokens over the cache (qmm_kv_attend).

        q: fp16 (bf16 for a bf16 cache) [rows, heads, head_dim], any row stride that is a multiple of
        8; out: contiguous fp16, bf16 or fp32 of the same shape; row_len: int32 [rows], slots
        that the row sees; lse: fp32 [rows, heads]; weight_in / weight_out: the slots' accumulated
        weights before and after (weight_in may be weight_out, or None for zeros); scale: None
        for 1 / sqrt(head_dim)."""
        at = self._pool(pool)
        qp, qs = self._rows_of("q", q, self._q_dtype, self.heads)
        rows = q.shape[0]
        if rows > self.max_rows:
            _refuse("q", f"at most {self.max_rows} rows (the plan's max_rows)")
        kind = _types.get(out.dtype)
        if kind is None or out.shape != q.shape or not out.is_contiguous() or out.get_device() != self.device:
            _refuse("out", f"a contiguous fp32, fp16 or bf16 CUDA tensor [{rows}, {self.heads}, {self.head_dim}] on device {self.device}")
        stream = self._on(stream)
        ws, ws_bytes, _ = self._space("attend" if weight_out is None else "weights", stream)
        st = self._attend(
            self._ref, at, self._table, self._vector("agent_rows", agent_rows, _i32, self.agents + 1),
            self._vector("row_len", row_len, _i32, rows), qp, qs, rows, self._scale if scale is None else scale, out.data_ptr(), kind,
            0 if lse is None else self._vector("lse", lse, _f32, rows * self.heads),
            0 if weight_in is None else self._vector("weight_in", weight_in, _f32, self._slots),
            0 if weight_out is None else self._vector("weight_out", weight_out, _f32, self._slots), ws, ws_bytes, self._err, stream)
        if st:
            raise _q.QmmError(st, "qmm_kv_attend")

    def evict(self, pool, cache_len, keep, weight, pos, *, weight_out, pos_out, len_out, sink: int = 0, protect_from=None,
              stream: int | None = None) -> None:
        """Cut the sequences to keep[a] tokens by accumulated weight (qmm_kv_evict), in place in the pool.

        cache_len, keep, len_out: int32 [agents] (keep < 0: no limit); protect_from: int32
        [agents] or None; weight_out and pos_out may be weight and pos.  Slots from len_out on
        are free afterwards.  A sequence that is cut shares none of its pages with another: tokens move
        into the slots below keep[a]."""
        at = self._pool(pool)
        stream = self._on(stream)
        ws, ws_bytes, _ = self._space("evict", stream)
        st = self._evict(
            self._ref, at, self._table, self._vector("cache_len", cache_len, _i32, self.agents),
            self._vector("keep", keep, _i32, self.agents), sink,
            0 if protect_from is None else self._vector("protect_from", protect_from, _i32, self.agents),
            self._vector("weight", weight, _f32, self._slots), self._vector("pos", pos, _i32, self._slots),
            self._vector("weight_out", weight_out, _f32, self._slots), self._vector("pos_out", pos_out, _i32, self._slots),
            self._vector("len_out", len_out, _i32, self.agents), ws, ws_bytes, self._err, stream)
        if st:
            raise _q.QmmError(st, "qmm_kv_evict")

    def error(self) -> int:
        """The error word (synchronises): 0, or 1 (a wait ran out) | 2 (page table) | 4 (rows or lengths)."""
        return int(self.error_word.item())


def logprobs(logits, tokens=None, lse=None, logprob=None, entropy=None, top_index=None, top_logprob=None,
             stream: int | None = None) -> None:
    """Log probabilities over rows of logits (qmm_logprobs).

    logits: fp32, fp16 or bf16 [m, n], any row stride.  tokens: int32 [m, given] with logprob
    fp32 [m, given]; lse, entropy: fp32 [m]; top_index: int32 [m, top] with top_logprob fp32
    [m, top], top <= 32.  Outputs left out are not computed."""
    if _torch is None:
        _setup()
    kind = _types.get(logits.dtype)
    if kind is None or logits.dim() != 2 or not logits.is_cuda:
        _refuse("logits", "an fp32, fp16 or bf16 CUDA tensor [m, n]")
    device = logits.get_device()
    _current(device)
    m, n = logits.shape
    st = logits.stride()
    if m > 0 and n > 1 and st[1] != 1:
        _refuse("logits", "contiguous but for the row stride")
    if (tokens is None) != (logprob is None) or (top_index is None) != (top_logprob is None):
        _refuse("tokens and logprob, top_index and top_logprob", "given together")
    given = top = tp = lp = ip = vp = 0
    if tokens is not None:
        # (their second dim is the number per row: a transposed pair would pass for one of other rows)
        if tokens.dim() != 2 or tokens.shape[0] != m or logprob.shape != tokens.shape:
            _refuse("tokens and logprob", f"[{m}, given], both")
        given = tokens.shape[1]
        tp, lp = _vector("tokens", tokens, _i32, m * given, device), _vector("logprob", logprob, _f32, m * given, device)
    if top_index is not None:
        if top_index.dim() != 2 or top_index.shape[0] != m or top_logprob.shape != top_index.shape:
            _refuse("top_index and top_logprob", f"[{m}, top], both")
        top = top_index.shape[1]
        ip, vp = _vector("top_index", top_index, _i32, m * top, device), _vector("top_logprob", top_logprob, _f32, m * top, device)
    status = load().qmm_logprobs(logits.data_ptr(), kind, m, n, st[0] if m > 1 else n, tp, given, top,
                                 0 if lse is None else _vector("lse", lse, _f32, m, device),
                                 0 if entropy is None else _vector("entropy", entropy, _f32, m, device), lp, ip, vp,
                                 _raw(device) if stream is None else stream)
    if status:
        raise _q.QmmError(status, "qmm_logprobs")
