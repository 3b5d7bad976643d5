"""Thin Python binding over libdhsa.so (ctypes).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
import threading
from typing import Optional, Tuple

import numpy as np
import torch

from .workloads import Budget

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdhsa.so")
_lib = None
_lib_lock = threading.Lock()

DHSA_BF16 = 0
DHSA_F32 = 1

STATUS_NAMES = {0: "DHSA_OK", 1: "DHSA_ERR_INVALID_ARG", 2: "DHSA_ERR_UNSUPPORTED",
                3: "DHSA_ERR_WORKSPACE", 4: "DHSA_ERR_CUDA", 5: "DHSA_ERR_TIMEOUT",
                6: "DHSA_ERR_DEVICE_CHECK"}

EXPORTED = [
    "dhsa_status_string", "dhsa_validate", "dhsa_plan_nnz", "dhsa_chunk_reduce",
    "dhsa_chunk_similarity", "dhsa_topk_select", "dhsa_plan_workspace_size", "dhsa_plan",
    "dhsa_attention_workspace_size", "dhsa_attention", "dhsa_workspace_status",
    "dhsa_selftest_timeout", "dhsa_plan_noalloc", "dhsa_attention_kv_plan",
    "dhsa_segment_capacity", "dhsa_segment_workspace_size", "dhsa_segment", "dhsa_plan_check",
    "dhsa_plan_margins", "dhsa_rope_init", "dhsa_rope_init_freq", "dhsa_rope", "dhsa_kv_append",
    "dhsa_paged_attention_workspace_size", "dhsa_paged_attention",
]

DHSA_BUDGET_PER_KV_HEAD = 0x100


class DhsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__("%s failed: %s" % (where, STATUS_NAMES.get(code, str(code))))
        self.code = code


class _Budget(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("k", ctypes.c_int32), ("num", ctypes.c_int32),
                ("den", ctypes.c_int32)]


class _Problem(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("total_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("num_chunks", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("chunk_bounds", ctypes.c_void_p),
                ("seq_chunk_ptr", ctypes.c_void_p),
                ("h_cu_seqlens", ctypes.c_void_p), ("h_chunk_bounds", ctypes.c_void_p),
                ("h_seq_chunk_ptr", ctypes.c_void_p)]


class _SegmentRule(ctypes.Structure):
    _fields_ = [("threshold", ctypes.c_float), ("min_len", ctypes.c_int32), ("max_len", ctypes.c_int32)]


ROPE_MAX_PAIRS = 128
ROPE_KINDS = {"linear": 1, "llama3": 2, "yarn": 3}


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


class _RopeTable(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float),
                ("turns", ctypes.c_uint64 * ROPE_MAX_PAIRS)]


class _Tokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64)]


class _PagedCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p)]


class _PagedBatch(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("table_stride", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("group_ptr", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p),
                ("h_cu_q", ctypes.c_void_p), ("h_group_ptr", ctypes.c_void_p)]


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:  # one thread loads the library and sets every signature
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libdhsa.so is missing (build it with "
                               "`python -m dynamic_hierarchical_sparse_b200.build`)")
        L = ctypes.CDLL(_LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        PP = ctypes.POINTER(_Problem)
        PB = ctypes.POINTER(_Budget)
        sig = {
            "dhsa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "dhsa_validate": (ctypes.c_int, [PP, PB]),
            "dhsa_plan_nnz": (ctypes.c_int, [PP, _Budget, ctypes.POINTER(I64)]),
            "dhsa_chunk_reduce": (ctypes.c_int, [P, I32, I32, I32, I32, P, I32, P, P]),
            "dhsa_chunk_similarity": (ctypes.c_int, [P, P, PP, P, P]),
            "dhsa_topk_select": (ctypes.c_int, [P, PP, _Budget, P, P, I64, P, SZ, P]),
            "dhsa_plan_workspace_size": (ctypes.c_int, [PP, _Budget, ctypes.POINTER(SZ)]),
            "dhsa_plan": (ctypes.c_int, [P, P, PP, _Budget, P, P, I64, P, SZ, P]),
            "dhsa_attention_workspace_size": (ctypes.c_int, [PP, ctypes.POINTER(SZ)]),
            "dhsa_attention": (ctypes.c_int, [P, P, P, PP, P, P, I64, ctypes.c_float, P, P, SZ, P]),
            "dhsa_workspace_status": (ctypes.c_int, [P, P]),
            "dhsa_selftest_timeout": (ctypes.c_int, [P, I32, P]),
            "dhsa_plan_noalloc": (ctypes.c_int, [P, P, PP, _Budget, P, P, I64, P]),
            "dhsa_attention_kv_plan": (ctypes.c_int, [P, P, P, PP, P, P, I64, ctypes.c_float, P, P, SZ, P]),
            "dhsa_segment_capacity": (ctypes.c_int, [P, I32, I32, ctypes.POINTER(I64)]),
            "dhsa_segment_workspace_size": (ctypes.c_int, [I32, ctypes.POINTER(SZ)]),
            "dhsa_segment": (ctypes.c_int, [P, I32, I32, I32, I32, P, P, _SegmentRule, P, I64, P, P, P, SZ, P]),
            "dhsa_plan_check": (ctypes.c_int, [PP, P, P, I64, I32, P, SZ, P]),
            "dhsa_plan_margins": (ctypes.c_int, [PP, _Budget, P, P, I64, P, SZ, P, P]),
            "dhsa_rope_init": (ctypes.c_int, [P, I32, I32, ctypes.c_double, P]),
            "dhsa_rope_init_freq": (ctypes.c_int, [P, I32, I32, P, ctypes.c_double]),
            "dhsa_rope": (ctypes.c_int, [P, I32, I32, I32, P, _Tokens, I32, _Tokens, _Tokens, I32, _Tokens, P]),
            "dhsa_kv_append": (ctypes.c_int, [P, P, P, P, _Tokens, _Tokens, _Tokens, _Tokens, _Tokens, I32, P, SZ, P]),
            "dhsa_paged_attention_workspace_size": (ctypes.c_int, [P, P, I32, ctypes.POINTER(SZ)]),
            "dhsa_paged_attention": (ctypes.c_int, [P, P, _Tokens, I32, ctypes.c_float, _Tokens, P, P, SZ, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(code: int, where: str) -> None:
    if code != 0:
        raise DhsaError(code, where)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _enter(stream) -> None:
    """A one-shot call on an explicit stream first waits for the work queued on
    the current stream (its inputs, and outputs this module just zeroed there)."""
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream(stream.device))


def _leave(stream) -> None:
    """... and the current stream waits for the call before its result is used
    (or freed) there."""
    if stream is not None:
        torch.cuda.current_stream(stream.device).wait_stream(stream)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _budget(b: Budget) -> _Budget:
    kind = int(b.kind) | (DHSA_BUDGET_PER_KV_HEAD if getattr(b, "per_kv_head", False) else 0)
    return _Budget(kind, int(b.k), int(b.num), int(b.den))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DHSA_BF16
    if t.dtype == torch.float32:
        return DHSA_F32
    raise TypeError("q/k/v must be bfloat16 or float32, got %s" % t.dtype)


class Problem:
    """Shapes + chunk structure of one packed batch, with host and device mirrors."""

    def __init__(self, cu_seqlens, chunk_bounds, seq_chunk_ptr, num_q_heads: int,
                 num_kv_heads: int, head_dim: int, dtype: torch.dtype,
                 device: Optional[torch.device] = None):
        self.h_cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
        self.h_bounds = np.ascontiguousarray(np.asarray(chunk_bounds, dtype=np.int32))
        self.h_sptr = np.ascontiguousarray(np.asarray(seq_chunk_ptr, dtype=np.int32))
        dev = torch.device("cuda") if device is None else device
        self.d_cu = torch.from_numpy(self.h_cu).to(dev)
        self.d_bounds = torch.from_numpy(self.h_bounds).to(dev)
        self.d_sptr = torch.from_numpy(self.h_sptr).to(dev)
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        self.dtype = dtype
        self.num_chunks = int(self.h_bounds.shape[0] - 1)
        self.num_seqs = int(self.h_cu.shape[0] - 1)
        self.total_tokens = int(self.h_cu[-1])
        self.c = _Problem(
            DHSA_BF16 if dtype == torch.bfloat16 else DHSA_F32, self.num_seqs, self.total_tokens,
            num_q_heads, num_kv_heads, head_dim, self.num_chunks,
            self.d_cu.data_ptr(), self.d_bounds.data_ptr(), self.d_sptr.data_ptr(),
            self.h_cu.ctypes.data, self.h_bounds.ctypes.data, self.h_sptr.ctypes.data)

    @staticmethod
    def from_inputs(inp, device: Optional[torch.device] = None) -> "Problem":
        s = inp.spec
        return Problem(inp.cu_seqlens, inp.chunk_bounds, inp.seq_chunk_ptr, s.num_q_heads,
                       s.num_kv_heads, s.head_dim, inp.q.dtype, device)

    def ref(self):
        return ctypes.byref(self.c)

    def validate(self, budget: Optional[Budget] = None) -> int:
        if budget is None:
            return lib().dhsa_validate(self.ref(), None)
        b = _budget(budget)
        return lib().dhsa_validate(self.ref(), ctypes.byref(b))

    def nnz(self, budget: Budget) -> int:
        out = ctypes.c_int64(0)
        _check(lib().dhsa_plan_nnz(self.ref(), _budget(budget), ctypes.byref(out)), "dhsa_plan_nnz")
        return int(out.value)

    def plan_workspace_bytes(self, budget: Budget) -> int:
        out = ctypes.c_size_t(0)
        _check(lib().dhsa_plan_workspace_size(self.ref(), _budget(budget), ctypes.byref(out)),
               "dhsa_plan_workspace_size")
        return int(out.value)

    def attention_workspace_bytes(self) -> int:
        out = ctypes.c_size_t(0)
        _check(lib().dhsa_attention_workspace_size(self.ref(), ctypes.byref(out)),
               "dhsa_attention_workspace_size")
        return int(out.value)


@dataclasses.dataclass
class Plan:
    row_ptr: torch.Tensor  # int32 [Hq*n+1] device ([Hkv*n+1] for a per-KV-head plan)
    col: torch.Tensor      # int32 [nnz] device
    nnz: int
    per_kv_head: bool = False


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _require(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def chunk_reduce(x: torch.Tensor, problem: Problem, stream=None) -> torch.Tensor:
    """Step 1 for one tensor: [T, H, d] -> fp32 [H, n, d]."""
    _require(x, "x")
    T, H, d = x.shape
    out = torch.empty(H, problem.num_chunks, d, dtype=torch.float32, device=x.device)
    _enter(stream)
    _check(lib().dhsa_chunk_reduce(_ptr(x), _dtype_code(x), T, H, d, _ptr(problem.d_bounds),
                                   problem.num_chunks, _ptr(out), _stream_ptr(stream)),
           "dhsa_chunk_reduce")
    _leave(stream)
    return out


def chunk_similarity(qc: torch.Tensor, kc: torch.Tensor, problem: Problem, stream=None) -> torch.Tensor:
    """Step 2: fp32 [Hq, n, n]; entries outside the causal same-sequence triangle are 0."""
    n = problem.num_chunks
    scores = torch.zeros(problem.num_q_heads, n, n, dtype=torch.float32, device=qc.device)
    _enter(stream)
    _check(lib().dhsa_chunk_similarity(_ptr(qc), _ptr(kc), problem.ref(), _ptr(scores),
                                       _stream_ptr(stream)), "dhsa_chunk_similarity")
    _leave(stream)
    return scores


def topk_select(scores: torch.Tensor, problem: Problem, budget: Budget, stream=None,
                check: bool = False) -> Plan:
    """Step 3 on a given score matrix."""
    nnz = problem.nnz(budget)
    dev = scores.device
    heads = problem.num_kv_heads if budget.per_kv_head else problem.num_q_heads
    row_ptr = torch.empty(heads * problem.num_chunks + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
    ws = _workspace(256, dev)
    st = _stream_ptr(stream)
    _enter(stream)
    _check(lib().dhsa_topk_select(_ptr(scores), problem.ref(), _budget(budget), _ptr(row_ptr), _ptr(col),
                                  nnz, _ptr(ws), ws.numel(), st), "dhsa_topk_select")
    if check:
        _check(lib().dhsa_workspace_status(_ptr(ws), st), "dhsa_topk_select (device)")
    _leave(stream)
    return Plan(row_ptr, col[:nnz], nnz, bool(budget.per_kv_head))


class Planner:
    """Owns the plan workspace and output buffers for repeated dhsa_plan calls.
    With an explicit stream, ordering against other streams is the caller's
    (the one-shot functions below do it themselves)."""

    def __init__(self, problem: Problem, budget: Budget, device=None):
        self.problem, self.budget = problem, budget
        dev = problem.d_bounds.device if device is None else device
        self.nnz = problem.nnz(budget)
        self.ws = _workspace(problem.plan_workspace_bytes(budget), dev)
        heads = problem.num_kv_heads if budget.per_kv_head else problem.num_q_heads
        self.row_ptr = torch.empty(heads * problem.num_chunks + 1, dtype=torch.int32, device=dev)
        self.col = torch.empty(max(self.nnz, 1), dtype=torch.int32, device=dev)
        self._b = _budget(budget)

    def __call__(self, q: torch.Tensor, k: torch.Tensor, stream=None) -> Plan:
        _check(lib().dhsa_plan(_ptr(q), _ptr(k), self.problem.ref(), self._b, _ptr(self.row_ptr),
                               _ptr(self.col), self.nnz, _ptr(self.ws), self.ws.numel(),
                               _stream_ptr(stream)), "dhsa_plan")
        return Plan(self.row_ptr, self.col[:self.nnz], self.nnz, bool(self.budget.per_kv_head))

    def status(self, stream=None) -> int:
        return lib().dhsa_workspace_status(_ptr(self.ws), _stream_ptr(stream))

    def margins(self, stream=None) -> torch.Tensor:
        """Selection margins of the plan the last call wrote (dhsa_plan_margins):
        fp32 [rows, 2], the k-th and (k+1)-th largest admissible scores per row
        (NaN where there is none)."""
        rows = self.row_ptr.numel() - 1
        out = torch.empty(rows, 2, dtype=torch.float32, device=self.row_ptr.device)
        _check(lib().dhsa_plan_margins(self.problem.ref(), self._b, _ptr(self.row_ptr), _ptr(self.col), self.nnz,
                                       _ptr(self.ws), self.ws.numel(), _ptr(out), _stream_ptr(stream)),
               "dhsa_plan_margins")
        return out


def plan(q: torch.Tensor, k: torch.Tensor, problem: Problem, budget: Budget, stream=None,
         check: bool = False) -> Plan:
    """Steps 1-3: returns the per-(head, query chunk) list of kept key chunks."""
    _require(q, "q")
    _require(k, "k")
    p = Planner(problem, budget, q.device)
    _enter(stream)
    out = p(q, k, stream)
    if check:
        _check(p.status(stream), "dhsa_plan (device)")
    _leave(stream)
    return Plan(out.row_ptr.clone(), out.col.clone(), out.nnz, out.per_kv_head)


def check_plan(problem: Problem, row_ptr: torch.Tensor, col: torch.Tensor, per_kv_head: bool = False,
               stream=None) -> int:
    """Device-side structural check of a plan (dhsa_plan_check).  Waits for it
    and returns the status (0 = a valid plan, 6 = DHSA_ERR_DEVICE_CHECK).
    row_ptr / col: int32 device tensors; nnz = col.numel()."""
    _require(row_ptr, "row_ptr")
    _require(col, "col")
    if row_ptr.dtype != torch.int32 or col.dtype != torch.int32:
        raise TypeError("row_ptr and col must be int32")
    ws = _workspace(256, row_ptr.device)
    st = _stream_ptr(stream)
    _enter(stream)
    _check(lib().dhsa_plan_check(problem.ref(), _ptr(row_ptr), _ptr(col), int(col.numel()), int(bool(per_kv_head)),
                                 _ptr(ws), ws.numel(), st), "dhsa_plan_check")
    code = int(lib().dhsa_workspace_status(_ptr(ws), st))
    _leave(stream)
    return code


class Attention:
    """Owns the attention workspace for repeated dhsa_attention calls (stream
    ordering as for Planner)."""

    def __init__(self, problem: Problem, device=None):
        self.problem = problem
        dev = problem.d_bounds.device if device is None else device
        self.ws = _workspace(problem.attention_workspace_bytes(), dev)

    def __call__(self, q, k, v, plan: Plan, out: torch.Tensor, scale: Optional[float] = None,
                 stream=None) -> torch.Tensor:
        fn = lib().dhsa_attention_kv_plan if plan.per_kv_head else lib().dhsa_attention
        _check(fn(_ptr(q), _ptr(k), _ptr(v), self.problem.ref(), _ptr(plan.row_ptr), _ptr(plan.col), plan.nnz,
                  ctypes.c_float(0.0 if scale is None else scale), _ptr(out), _ptr(self.ws), self.ws.numel(),
                  _stream_ptr(stream)), "dhsa_attention")
        return out

    def status(self, stream=None) -> int:
        return lib().dhsa_workspace_status(_ptr(self.ws), _stream_ptr(stream))


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, problem: Problem, plan: Plan,
              scale: Optional[float] = None, stream=None, check: bool = False) -> torch.Tensor:
    """Step 4: sparse causal attention over the plan's kept token pairs."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, name)
    out = torch.empty_like(q)
    a = Attention(problem, q.device)
    _enter(stream)
    a(q, k, v, plan, out, scale, stream)
    if check:
        _check(a.status(stream), "dhsa_attention (device)")
    _leave(stream)
    return out


class Segmenter:
    """Owns the buffers of repeated online chunking calls (dhsa_segment) for
    one batch layout: sequence offsets, KV heads, head dim and rule."""

    def __init__(self, cu_seqlens, num_kv_heads: int, head_dim: int, rule, device=None):
        self.h_cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
        self.num_seqs = int(self.h_cu.shape[0] - 1)
        self.num_kv_heads, self.head_dim = int(num_kv_heads), int(head_dim)
        self.rule = rule
        self._rule = _SegmentRule(float(rule.threshold), int(rule.min_len), int(rule.max_len))
        dev = torch.device("cuda") if device is None else torch.device(device)
        L = lib()
        cap = ctypes.c_int64(0)
        _check(L.dhsa_segment_capacity(self.h_cu.ctypes.data_as(ctypes.c_void_p), self.num_seqs,
                                       int(rule.min_len), ctypes.byref(cap)), "dhsa_segment_capacity")
        self.capacity = int(cap.value)
        ws = ctypes.c_size_t(0)
        _check(L.dhsa_segment_workspace_size(int(self.h_cu[-1]), ctypes.byref(ws)), "dhsa_segment_workspace_size")
        self.ws = _workspace(ws.value, dev)
        self.d_cu = torch.from_numpy(self.h_cu).to(dev)
        self.chunk_bounds = torch.empty(self.capacity + 1, dtype=torch.int32, device=dev)
        self.seq_chunk_ptr = torch.empty(self.num_seqs + 1, dtype=torch.int32, device=dev)
        self.num_chunks = torch.empty(1, dtype=torch.int32, device=dev)

    def __call__(self, k: torch.Tensor, stream=None):
        """Asynchronous: returns the device arrays (chunk_bounds holds
        num_chunks + 1 valid entries)."""
        _require(k, "k")
        _check(lib().dhsa_segment(_ptr(k), _dtype_code(k), self.num_kv_heads, self.head_dim, self.num_seqs,
                                  _ptr(self.d_cu), self.h_cu.ctypes.data_as(ctypes.c_void_p), self._rule,
                                  _ptr(self.chunk_bounds), self.capacity, _ptr(self.seq_chunk_ptr),
                                  _ptr(self.num_chunks), _ptr(self.ws), self.ws.numel(), _stream_ptr(stream)),
               "dhsa_segment")
        return self.chunk_bounds, self.seq_chunk_ptr, self.num_chunks

    def status(self, stream=None) -> int:
        return lib().dhsa_workspace_status(_ptr(self.ws), _stream_ptr(stream))


def segment(k: torch.Tensor, cu_seqlens, rule, stream=None, check: bool = False):
    """Online variable-length chunking of the packed batch ``k`` [T, Hkv, d].

    Waits for the result and returns host int32 arrays (chunk_bounds [n+1],
    seq_chunk_ptr [B+1]), ready for ``Problem``."""
    seg = Segmenter(cu_seqlens, k.shape[1], k.shape[2], rule, k.device)
    _enter(stream)
    bounds, ptr, n = seg(k, stream)
    if check:
        _check(seg.status(stream), "dhsa_segment (device)")
    _leave(stream)
    n = int(n.item())
    return bounds[:n + 1].cpu().numpy(), ptr.cpu().numpy()


def selftest_timeout(limit_us: int = 20000, device=None) -> int:
    """Runs the bounded-wait self test; returns the status it reports (expect 5)."""
    ws = _workspace(256, torch.device("cuda") if device is None else device)
    st = _stream_ptr(None)
    _check(lib().dhsa_selftest_timeout(_ptr(ws), int(limit_us), st), "dhsa_selftest_timeout")
    return int(lib().dhsa_workspace_status(_ptr(ws), st))


# ------------------------------------------------- around the prefill path


# The calls below cost a few microseconds on the GPU at a decode step, so their
# marshalling is kept short: device indexes instead of device objects, the raw
# current stream instead of a Stream object, plain integers for pointers.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


class _on_device:
    """Makes a device the current one for a block (launches go by it); nothing
    to do where it already is."""

    def __init__(self, index: int):
        self.index = index

    def __enter__(self):
        self.before = _current_device()
        if self.before != self.index:
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.before != self.index:
            torch.cuda.set_device(self.before)


def _call(fn, name: str, index: int, args: tuple) -> None:
    """fn(*args) with device `index` current; raises on an error status."""
    if _current_device() == index:
        code = fn(*args)
    else:
        with _on_device(index):
            code = fn(*args)
    if code != 0:
        raise DhsaError(code, name)


def _stream_on(stream, index: int) -> int:
    return _raw_stream(index) if stream is None else stream.cuda_stream


_NO_TOKENS = _Tokens(None, 0)  # passed by value, never written
_I32 = torch.int32


def _tokens(t: Optional[torch.Tensor], name: str, heads: int, head_dim: int, dtype: torch.dtype, tokens: int,
            index: int) -> _Tokens:
    """A packed [T, H, d] operand whose tokens may lie apart (a slice of a fused
    tensor), on CUDA device `index`."""
    if t is None:
        return _NO_TOKENS
    shape = t.shape
    if len(shape) == 3 and t.dtype is dtype and t.get_device() == index:
        n, h, d = shape
        if h == heads and d == head_dim and n >= tokens:
            if t.is_contiguous():
                return _Tokens(t.data_ptr(), h * d)
            st, sh, sd = t.stride()
            if sd == 1 and (sh == d or h == 1) and (st >= h * d or n <= 1):
                return _Tokens(t.data_ptr(), st if n > 1 else h * d)
    # what of it is wrong
    if t.get_device() != index:
        raise ValueError("%s must be a CUDA tensor on device %d, got %s" % (name, index, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if len(shape) != 3 or n < tokens or h != heads or d != head_dim:
        raise ValueError("%s must be [>= %d, %d, %d], got %s" % (name, tokens, heads, head_dim, tuple(shape)))
    if sd != 1 or (sh != d and h > 1):
        raise ValueError("the heads of a token of %s must be contiguous" % name)
    raise ValueError("the tokens of %s overlap (a broadcast tensor must be expanded to memory of its own)" % name)


def _int32(t: torch.Tensor, name: str, shape, index: int) -> None:
    if t.dtype is _I32 and t.shape == shape and t.get_device() == index >= 0 and t.is_contiguous():
        return
    if t.get_device() != index or index < 0:
        raise ValueError("%s must be a CUDA tensor on device %d" % (name, index))
    if t.dtype is not torch.int32:
        raise TypeError("%s must be int32" % name)
    raise ValueError("%s must be a contiguous %s tensor, got %s" % (name, shape, tuple(t.shape)))


class Rope:
    """Rotary frequencies (dhsa_rope_table): host data, usable on any device.

    ``rotary_dim``: the first numbers of a head that turn; pairs are (i, i +
    rotary_dim / 2), or (2i, 2i + 1) when ``interleaved``.  ``scaling``: a
    ``workloads.RopeScaling`` or None.  ``inv_freq`` gives the rotary_dim / 2
    frequencies themselves (then ``base`` and ``scaling`` are not used), with
    ``factor`` on cos and sin."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling=None,
                 inv_freq=None, factor: float = 1.0):
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)
        self.c = _RopeTable()
        self.ref, self.fn = ctypes.byref(self.c), lib().dhsa_rope
        if inv_freq is not None:
            f = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
            if f.shape != (self.rotary_dim // 2,):
                raise ValueError("inv_freq must have rotary_dim / 2 entries")
            _check(lib().dhsa_rope_init_freq(ctypes.byref(self.c), self.rotary_dim, int(self.interleaved),
                                             f.ctypes.data_as(ctypes.c_void_p), float(factor)), "dhsa_rope_init_freq")
            return
        sc = None
        if scaling is not None:
            if scaling.kind not in ROPE_KINDS:
                raise ValueError("unknown rope scaling %r" % (scaling.kind,))
            sc = ctypes.byref(_RopeScaling(ROPE_KINDS[scaling.kind], scaling.factor, scaling.original_len,
                                           scaling.low_freq_factor, scaling.high_freq_factor, scaling.beta_fast,
                                           scaling.beta_slow))
        _check(lib().dhsa_rope_init(ctypes.byref(self.c), self.rotary_dim, int(self.interleaved), float(base), sc),
               "dhsa_rope_init")


def rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor, rope: Rope,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotates packed q [T, Hq, d] and k [T, Hkv, d] (either may be None) at
    ``positions`` (int32 [T]); returns (q_out, k_out).  Outputs are made where
    they are not given; an output may be its own input."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("rope needs q or k")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("an output without its input")
    T, hq, d = x.shape
    dev, dtype = x.get_device(), x.dtype
    hk = 1
    _int32(positions, "positions", (T,), dev)
    if q is not None and q_out is None:
        q_out = torch.empty(T, hq, d, dtype=dtype, device=x.device)
    if k is not None:
        hk = k.shape[1]
        if k_out is None:
            k_out = torch.empty(T, hk, d, dtype=dtype, device=x.device)
    if stream is not None:
        _enter(stream)
    _call(rope.fn, "dhsa_rope", dev,
          (rope.ref, _dtype_code(x), d, T, positions.data_ptr(), _tokens(q, "q", hq, d, dtype, T, dev), hq,
           _tokens(q_out, "q_out", hq, d, dtype, T, dev), _tokens(k, "k", hk, d, dtype, T, dev), hk,
           _tokens(k_out, "k_out", hk, d, dtype, T, dev), _stream_on(stream, dev)))
    if stream is not None:
        _leave(stream)
    return q_out, k_out


class PagedCache:
    """The pages of a K/V cache: ``k_pages`` and ``v_pages`` [pages, Hkv,
    page_size, d] on the device, each page contiguous (pages may lie apart, by
    the same stride in both).  K in bf16 and V in f16, or both in fp32."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor):
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if not t.is_cuda or t.dim() != 4:
                raise ValueError("%s must be a CUDA tensor [pages, Hkv, page_size, d]" % name)
        if k_pages.shape != v_pages.shape or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must have one shape and device")
        want = {torch.bfloat16: torch.float16, torch.float32: torch.float32}.get(k_pages.dtype)
        if want is None or v_pages.dtype != want:
            raise TypeError("pages must be K bfloat16 with V float16, or both float32; got %s, %s"
                            % (k_pages.dtype, v_pages.dtype))
        n, h, p, d = k_pages.shape
        for t in (k_pages, v_pages):
            st = t.stride()
            if st[3] != 1 or (p > 1 and st[2] != d) or (h > 1 and st[1] != p * d):
                raise ValueError("a page must be contiguous")
        if n > 1 and k_pages.stride(0) != v_pages.stride(0):
            raise ValueError("k_pages and v_pages must have one page stride")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = n, h, p, d
        self.dtype, self.device, self.index = k_pages.dtype, k_pages.device, k_pages.get_device()
        self.c = _PagedCache(_dtype_code(k_pages), h, d, p, n, k_pages.stride(0) if n > 1 else h * p * d,
                             k_pages.data_ptr(), v_pages.data_ptr())

    @staticmethod
    def empty(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, dtype: torch.dtype,
              device=None) -> "PagedCache":
        dev = torch.device("cuda") if device is None else torch.device(device)
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        v_dtype = torch.float16 if dtype == torch.bfloat16 else dtype
        return PagedCache(torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=v_dtype, device=dev))


class PagedBatch:
    """One step of a batch over a paged cache (dhsa_paged_batch).

    ``cu_q``: host offsets [B+1] of the sequences' new tokens in the packed
    tensors; ``kv_lens`` int32 [B] on the device: tokens a sequence holds with
    them; ``block_table`` int32 [B, max_pages] on the device.  ``group_ptr``
    (host [G+1]) and ``prefix_lens`` (int32 [G] on the device): the sequences of
    a group share their first prefix_lens[g] tokens.  The device tensors are
    kept and read by every call, so a program may go on writing them."""

    def __init__(self, cu_q, kv_lens: torch.Tensor, block_table: torch.Tensor, group_ptr=None,
                 prefix_lens: Optional[torch.Tensor] = None):
        # copies: the offsets on the host and on the device have to stay the same ones
        self.h_cu = np.asarray(cu_q, dtype=np.int32).copy(order="C")
        if self.h_cu.ndim != 1 or self.h_cu.shape[0] < 1:
            raise ValueError("cu_q must have B + 1 entries")
        self.num_seqs = int(self.h_cu.shape[0] - 1)
        self.total_tokens = int(self.h_cu[-1])
        dev, self.index = kv_lens.device, kv_lens.get_device()
        _int32(kv_lens, "kv_lens", (self.num_seqs,), self.index)
        if not block_table.is_cuda or block_table.device != dev or block_table.dtype != torch.int32:
            raise ValueError("block_table must be an int32 tensor on %s" % dev)
        if block_table.dim() != 2 or block_table.shape[0] != self.num_seqs or block_table.shape[1] < 1 or \
                block_table.stride(1) != 1:
            raise ValueError("block_table must be [B, max_pages] with contiguous rows")
        if (group_ptr is None) != (prefix_lens is None):
            raise ValueError("group_ptr and prefix_lens come together")
        width = int(block_table.shape[1])
        stride = int(block_table.stride(0)) if self.num_seqs > 1 else width
        self.device, self.kv_lens, self.block_table, self.prefix_lens = dev, kv_lens, block_table, prefix_lens
        self.d_cu = torch.from_numpy(self.h_cu).to(dev)
        groups, self.h_groups, self.d_groups = 0, None, None
        if group_ptr is not None:
            self.h_groups = np.asarray(group_ptr, dtype=np.int32).copy(order="C")
            groups = int(self.h_groups.shape[0] - 1)
            if groups < 1:
                raise ValueError("group_ptr must have G + 1 entries, G >= 1")
            _int32(prefix_lens, "prefix_lens", (groups,), self.index)
            self.d_groups = torch.from_numpy(self.h_groups).to(dev)
        self.c = _PagedBatch(self.num_seqs, width, stride, groups, self.d_cu.data_ptr(), kv_lens.data_ptr(),
                             block_table.data_ptr(), 0 if groups == 0 else self.d_groups.data_ptr(),
                             0 if groups == 0 else prefix_lens.data_ptr(), self.h_cu.ctypes.data,
                             0 if groups == 0 else self.h_groups.ctypes.data)


class KvAppender:
    """Repeated dhsa_kv_append calls over one cache, batch and rotation (None:
    keys are stored as they come).  Owns the status word, which gathers reports
    until ``reset``.  Stream ordering as for Planner."""

    def __init__(self, cache: PagedCache, batch: PagedBatch, rope: Optional[Rope] = None):
        if cache.device != batch.device:
            raise ValueError("cache and batch are on different devices")
        self.cache, self.batch, self.rope = cache, batch, rope
        self.ws = torch.zeros(256, dtype=torch.uint8, device=cache.device)
        self._fixed = (ctypes.byref(cache.c), ctypes.byref(batch.c), None if rope is None else rope.ref)
        self._fn, self._ws = lib().dhsa_kv_append, self.ws.data_ptr()

    def __call__(self, k: torch.Tensor, v: torch.Tensor, q: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, stream=None):
        """Stores k and v [T, Hkv, d]; returns (q_out, k_out): q [T, Hq, d]
        rotated (made where q comes without q_out) and, where given, k_out."""
        c, T = self.cache, self.batch.total_tokens
        hk, d, dt, dev, hq, pos = c.num_kv_heads, c.head_dim, c.dtype, c.index, 1, None
        if q is not None:
            hq = q.shape[1]
            if q_out is None:
                q_out = torch.empty(T, hq, d, dtype=dt, device=c.device)
                if stream is not None:  # memory of the current stream, written on another
                    stream.wait_stream(torch.cuda.current_stream(c.device))
                    q_out.record_stream(stream)
        elif q_out is not None:
            raise ValueError("q_out without q")
        if positions is not None:
            _int32(positions, "positions", (T,), dev)
            pos = positions.data_ptr()
        _call(self._fn, "dhsa_kv_append", dev,
              (*self._fixed, pos, _tokens(k, "k", hk, d, dt, T, dev), _tokens(v, "v", hk, d, dt, T, dev),
               _tokens(k_out, "k_out", hk, d, dt, T, dev), _tokens(q, "q", hq, d, dt, T, dev),
               _tokens(q_out, "q_out", hq, d, dt, T, dev), hq, self._ws, 256, _stream_on(stream, dev)))
        return q_out, k_out

    def status(self, stream=None) -> int:
        with _on_device(self.cache.index):
            return lib().dhsa_workspace_status(_ptr(self.ws), _stream_ptr(stream))

    def reset(self) -> None:
        """Clears the status word (on the current stream)."""
        self.ws.zero_()


def append_kv(cache: PagedCache, batch: PagedBatch, k: torch.Tensor, v: torch.Tensor, rope: Optional[Rope] = None,
              q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, stream=None,
              check: bool = False):
    """One-shot append to the paged cache; returns (q_out, k_out) as KvAppender does."""
    a = KvAppender(cache, batch, rope)
    with _on_device(cache.index):
        _enter(stream)
        if q is not None and q_out is None:
            q_out = torch.empty(batch.total_tokens, q.shape[1], cache.head_dim, dtype=cache.dtype,
                                device=cache.device)
        out = a(k, v, q, q_out, k_out, positions, stream)
        if check:
            _check(a.status(stream), "dhsa_kv_append (device)")
        _leave(stream)
    return out


class PagedAttention:
    """Repeated dhsa_paged_attention calls over one cache, batch and number of
    query heads.  Owns the workspace (status word included, which gathers
    reports until ``reset``).  Stream ordering as for Planner."""

    def __init__(self, cache: PagedCache, batch: PagedBatch, num_q_heads: int):
        if cache.device != batch.device:
            raise ValueError("cache and batch are on different devices")
        self.cache, self.batch, self.num_q_heads = cache, batch, int(num_q_heads)
        n = ctypes.c_size_t(0)
        _check(lib().dhsa_paged_attention_workspace_size(ctypes.byref(cache.c), ctypes.byref(batch.c),
                                                         self.num_q_heads, ctypes.byref(n)),
               "dhsa_paged_attention_workspace_size")
        self.ws = _workspace(n.value, cache.device)
        self.reset()
        self._fixed = (ctypes.byref(cache.c), ctypes.byref(batch.c))
        self._fn, self._ws, self._ws_bytes = lib().dhsa_paged_attention, self.ws.data_ptr(), self.ws.numel()

    def __call__(self, q: torch.Tensor, out: torch.Tensor, scale: Optional[float] = None,
                 lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        c, T, hq = self.cache, self.batch.total_tokens, self.num_q_heads
        d, dt, dev, lse_ptr = c.head_dim, c.dtype, c.index, None
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous() \
                    or lse.dim() != 2 or lse.shape[0] < T or lse.shape[1] != hq:
                raise ValueError("lse must be a contiguous float32 [>= %d, %d] tensor on device %d" % (T, hq, dev))
            lse_ptr = lse.data_ptr()
        _call(self._fn, "dhsa_paged_attention", dev,
              (*self._fixed, _tokens(q, "q", hq, d, dt, T, dev), hq, 0.0 if scale is None else scale,
               _tokens(out, "out", hq, d, dt, T, dev), lse_ptr, self._ws, self._ws_bytes, _stream_on(stream, dev)))
        return out

    def status(self, stream=None) -> int:
        with _on_device(self.cache.index):
            return lib().dhsa_workspace_status(_ptr(self.ws), _stream_ptr(stream))

    def reset(self) -> None:
        """Clears the status word (on the current stream)."""
        self.ws[:256].zero_()


def paged_attention(q: torch.Tensor, cache: PagedCache, batch: PagedBatch, scale: Optional[float] = None,
                    lse: Optional[torch.Tensor] = None, stream=None, check: bool = False) -> torch.Tensor:
    """Attention of the new tokens q [T, Hq, d] over the paged cache.  Rows of
    the result behind the last sequence's are zero."""
    a = PagedAttention(cache, batch, q.shape[1])
    with _on_device(cache.index):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        out[batch.total_tokens:].zero_()
        _enter(stream)
        a(q, out, scale, lse, stream)
        if check:
            _check(a.status(stream), "dhsa_paged_attention (device)")
        _leave(stream)
    return out
