"""ctypes binding of the serving operators (include/qmm_serve.h): argument checks and marshalling.

``KvPlan`` holds what a serving program sets up once for a paged KV cache -- its dims, the page
table, the workspace and the error word -- and appends to the cache, attends over it and evicts
from it; ``logprobs`` reads the lm_head's output.  As in ``qmm``, every step runs in the library's
CUDA kernels, there is no fallback, and PyTorch supplies only device memory and streams.  Calls go
to the current stream unless ``stream`` is given; a tensor last written on another stream has to be
ordered before them by the caller."""
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


_types = None


def _type_of(t) -> int:
    global _types
    if _types is None:
        import torch
        _types = {torch.float32: TYPE_F32, torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16}
    if t.dtype not in _types:
        raise TypeError(f"fp32, fp16 or bf16 expected, got {t.dtype}")
    return _types[t.dtype]


def _opt(t) -> int:
    return 0 if t is None else t.data_ptr()


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class KvPlan:
    """A paged KV cache of one layer: the dims, the page table, the workspace and the error word.

    page_table: int32 CUDA tensor [agents, max_pages], contiguous; its entries may be rewritten
    between calls.  format: "q8_0" (the pool of qmm_attn_decode: head_dim 128, page_tokens 64),
    "f16" or "bf16" (head_dim 64, 128 or 256, page_tokens 16 .. 256).  The pool is passed to each
    call, so that layers can share a plan: a uint8 tensor of pool_pages * kv_heads * 17,408 bytes,
    or a 16-bit one of pool_pages * kv_heads * 2 * page_tokens * head_dim elements.
    max_rows / max_agent_rows bound the rows of an attend call, and those of one sequence.
    Calls of one plan share its workspace: order them on one stream."""

    def __init__(self, page_table, *, format: str, heads: int, kv_heads: int, head_dim: int, page_tokens: int,
                 pool_pages: int, max_rows: int, max_agent_rows: int | None = None):
        import torch
        _need(page_table.dtype == torch.int32 and page_table.dim() == 2 and page_table.is_contiguous() and page_table.is_cuda,
              "page_table: a contiguous int32 CUDA tensor [agents, max_pages]")
        _need(format in FORMATS, f"format: one of {', '.join(FORMATS)}")
        agents, max_pages = page_table.shape
        self.page_table, self.format, self.max_rows = page_table, format, int(max_rows)
        self.dims = KvDims(FORMATS[format], heads, kv_heads, head_dim, page_tokens, agents, max_pages,
                           int(max_agent_rows or max_rows), pool_pages)
        self._ref = ctypes.byref(self.dims)
        self.cap = max_pages * page_tokens
        self._pool_dtype = {"q8_0": torch.uint8, "f16": torch.float16, "bf16": torch.bfloat16}[format]
        self._q_dtype = torch.bfloat16 if format == "bf16" else torch.float16
        self._pool_size = pool_pages * kv_heads * (17408 if format == "q8_0" else 2 * page_tokens * head_dim)
        self._i32, self._f32 = torch.int32, torch.float32
        self.error_word = torch.zeros(1, dtype=torch.int32, device=page_table.device)
        self._workspace = {}
        self._bytes("qmm_kv_evict_workspace_bytes")  # refuses dims that no call takes

    def _bytes(self, name, *args) -> int:
        n = ctypes.c_int64()
        _q._check(getattr(load(), name)(self._ref, *args, ctypes.byref(n)), name)
        return n.value

    def _space(self, kind: str):
        """The workspace of a kind of call, allocated at its first use and kept."""
        t = self._workspace.get(kind)
        if t is None:
            import torch
            n = self._bytes("qmm_kv_evict_workspace_bytes") if kind == "evict" else \
                self._bytes("qmm_kv_attend_workspace_bytes", int(kind == "weights"))
            t = self._workspace[kind] = torch.empty(n, dtype=torch.uint8, device=self.page_table.device)
        return t

    def _check_pool(self, pool):
        _need(pool.dtype == self._pool_dtype and pool.numel() == self._pool_size and pool.is_contiguous() and pool.is_cuda,
              f"pool: a contiguous {self._pool_dtype} CUDA tensor of {self._pool_size} elements")

    def _check_slots(self, name, t, dtype):
        _need(t is None or (t.dtype == dtype and t.is_contiguous() and t.is_cuda and
                            t.numel() == self.dims.agents * self.dims.kv_heads * self.cap),
              f"{name}: a contiguous {dtype} CUDA tensor [agents, kv_heads, {self.cap}]")

    def _check_ints(self, name, t, n):
        _need(t.dtype == self._i32 and t.numel() == n and t.is_contiguous() and t.is_cuda,
              f"{name}: a contiguous int32 CUDA tensor of {n} elements")

    def append(self, pool, agent_rows, cache_len, k, v, *, weight=None, pos=None, row_pos=None, stream: int | None = None) -> None:
        """Write K and V of new rows behind the sequences' cached tokens (qmm_kv_append).

        k, v: fp32, fp16 or bf16 [rows, kv_heads, head_dim], any row stride (columns of the qkv
        projection's output are taken in place).  cache_len: int32 [agents], tokens cached
        before the call (not changed).  weight / pos: the slots' arrays, whose new entries become
        0 and row_pos."""
        d = self.dims
        rows = k.shape[0]
        self._check_pool(pool)
        for name, t in (("k", k), ("v", v)):
            _need(t.shape == (rows, d.kv_heads, d.head_dim) and t.is_cuda and t.dtype == k.dtype and
                  (rows == 0 or t.stride()[1:] == (d.head_dim, 1)),
                  f"{name}: a CUDA tensor [rows, {d.kv_heads}, {d.head_dim}], contiguous but for the row stride")
        self._check_ints("agent_rows", agent_rows, d.agents + 1)
        self._check_ints("cache_len", cache_len, d.agents)
        self._check_slots("weight", weight, self._f32)
        self._check_slots("pos", pos, self._i32)
        if row_pos is not None:
            self._check_ints("row_pos", row_pos, rows)
        width = d.kv_heads * d.head_dim
        # (a single row's stride says nothing)
        ks, vs = (k.stride(0), v.stride(0)) if rows > 1 else (width, width)
        st = _q.current_stream() if stream is None else stream
        _q._check(load().qmm_kv_append(self._ref, pool.data_ptr(), self.page_table.data_ptr(), agent_rows.data_ptr(),
                                       cache_len.data_ptr(), k.data_ptr(), ks, v.data_ptr(), vs, _type_of(k), rows, _opt(weight),
                                       _opt(pos), _opt(row_pos), self.error_word.data_ptr(), st), "qmm_kv_append")

    def attend(self, pool, agent_rows, row_len, q, out, *, lse=None, weight_in=None, weight_out=None,
               scale: float | None = None, stream: int | None = None) -> None:
        """Attention of new tokens over the cache (qmm_kv_attend).

        q: fp16 (bf16 for a bf16 cache) [rows, heads, head_dim], any row stride that is a multiple of
        8; out: contiguous fp16, bf16 or fp32 of the same shape; row_len: int32 [rows], slots
        that the row sees; lse: fp32 [rows, heads]; weight_in / weight_out: the slots' accumulated
        weights before and after (weight_in may be weight_out, or None for zeros); scale: None
        for 1 / sqrt(head_dim)."""
        d = self.dims
        rows = q.shape[0]
        self._check_pool(pool)
        shape = (rows, d.heads, d.head_dim)
        _need(q.shape == shape and q.dtype == self._q_dtype and q.is_cuda and (rows == 0 or q.stride()[1:] == (d.head_dim, 1)),
              f"q: a {self._q_dtype} CUDA tensor [rows, {d.heads}, {d.head_dim}], contiguous but for the row stride")
        _need(out.shape == shape and out.is_contiguous() and out.is_cuda, f"out: a contiguous CUDA tensor [rows, {d.heads}, {d.head_dim}]")
        _need(rows <= self.max_rows, f"q: at most {self.max_rows} rows (the plan's max_rows)")
        self._check_ints("agent_rows", agent_rows, d.agents + 1)
        self._check_ints("row_len", row_len, rows)
        _need(lse is None or (lse.dtype == self._f32 and lse.numel() == rows * d.heads and lse.is_contiguous() and lse.is_cuda),
              f"lse: a contiguous fp32 CUDA tensor [rows, {d.heads}]")
        self._check_slots("weight_in", weight_in, self._f32)
        self._check_slots("weight_out", weight_out, self._f32)
        ws = self._space("weights" if weight_out is not None else "attend")
        st = _q.current_stream() if stream is None else stream
        _q._check(load().qmm_kv_attend(self._ref, pool.data_ptr(), self.page_table.data_ptr(), agent_rows.data_ptr(),
                                       row_len.data_ptr(), q.data_ptr(), q.stride(0) if rows > 1 else d.heads * d.head_dim, rows,
                                       d.head_dim ** -0.5 if scale is None else scale, out.data_ptr(), _type_of(out), _opt(lse),
                                       _opt(weight_in), _opt(weight_out), ws.data_ptr(), ws.numel(), self.error_word.data_ptr(), st),
                  "qmm_kv_attend")

    def evict(self, pool, cache_len, keep, weight, pos, *, weight_out, pos_out, len_out, sink: int = 0, protect_from=None,
              stream: int | None = None) -> None:
        """Cut the sequences to keep[a] tokens by accumulated weight (qmm_kv_evict), in place in the pool.

        cache_len, keep, len_out: int32 [agents] (keep < 0: no limit); protect_from: int32
        [agents] or None; weight_out and pos_out may be weight and pos.  Slots from len_out on
        are free afterwards."""
        d = self.dims
        self._check_pool(pool)
        self._check_ints("cache_len", cache_len, d.agents)
        self._check_ints("keep", keep, d.agents)
        self._check_ints("len_out", len_out, d.agents)
        if protect_from is not None:
            self._check_ints("protect_from", protect_from, d.agents)
        for name, t, dt in (("weight", weight, self._f32), ("weight_out", weight_out, self._f32), ("pos", pos, self._i32),
                            ("pos_out", pos_out, self._i32)):
            _need(t is not None, f"{name}: needed")
            self._check_slots(name, t, dt)
        ws = self._space("evict")
        st = _q.current_stream() if stream is None else stream
        _q._check(load().qmm_kv_evict(self._ref, pool.data_ptr(), self.page_table.data_ptr(), cache_len.data_ptr(), keep.data_ptr(),
                                      sink, _opt(protect_from), weight.data_ptr(), pos.data_ptr(), weight_out.data_ptr(),
                                      pos_out.data_ptr(), len_out.data_ptr(), ws.data_ptr(), ws.numel(), self.error_word.data_ptr(),
                                      st), "qmm_kv_evict")

    def error(self) -> int:
        """The error word (synchronises): 0, or 1 (a wait ran out) | 2 (page table) | 4 (rows or lengths)."""
        return int(self.error_word.item())


def logprobs(logits, tokens=None, lse=None, logprob=None, entropy=None, top_index=None, top_logprob=None,
             stream: int | None = None) -> None:
    """Log probabilities over rows of logits (qmm_logprobs).

    logits: fp32, fp16 or bf16 [m, n], any row stride.  tokens: int32 [m, given] with logprob
    fp32 [m, given]; lse, entropy: fp32 [m]; top_index: int32 [m, top] with top_logprob fp32
    [m, top], top <= 32.  Outputs left out are not computed."""
    import torch
    _need(logits.dim() == 2 and logits.is_cuda and (logits.shape[0] == 0 or logits.stride(1) == 1 or logits.shape[1] == 1),
          "logits: a CUDA tensor [m, n], contiguous but for the row stride")
    m, n = logits.shape
    _need((tokens is None) == (logprob is None) and (top_index is None) == (top_logprob is None),
          "tokens and logprob, top_index and top_logprob: given together")

    def two(name, t, dtype):
        if t is None:
            return 0
        _need(t.dtype == dtype and t.dim() == 2 and t.shape[0] == m and t.is_contiguous() and t.is_cuda,
              f"{name}: a contiguous {dtype} CUDA tensor [{m}, ..]")
        return t.shape[1]

    given, top = two("tokens", tokens, torch.int32), two("top_index", top_index, torch.int32)
    _need(two("logprob", logprob, torch.float32) == given, "logprob: as many columns as tokens")
    _need(two("top_logprob", top_logprob, torch.float32) == top, "top_logprob: as many columns as top_index")
    for name, t in (("lse", lse), ("entropy", entropy)):
        _need(t is None or (t.dtype == torch.float32 and t.numel() == m and t.is_contiguous() and t.is_cuda),
              f"{name}: a contiguous fp32 CUDA tensor [{m}]")
    st = _q.current_stream() if stream is None else stream
    _q._check(load().qmm_logprobs(logits.data_ptr(), _type_of(logits), m, n, logits.stride(0) if m > 1 else n, _opt(tokens), given,
                                  top, _opt(lse), _opt(entropy), _opt(logprob), _opt(top_index), _opt(top_logprob), st),
              "qmm_logprobs")
