"""Exact top-k indexer selection (HyTopK) and selection replay on MI355X, with
the operators around it: rotary positions, the quantised cache, the attention's
mass at the selected entries and the indexer's loss.

A thin ctypes binding over ``libhytopk.so`` (``include/hytopk.h``): it only
marshals torch tensors into pointers and sizes; every step of the selection
runs in the library's HIP kernels on the caller's current stream.  The
library must be built (``python -m exact_top_token_amd.build``); nothing here
falls back to a CPU or PyTorch implementation.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "Problem", "Params", "Stats", "load_library", "library_path", "select", "replay",
    "baseline_select", "select_workspace_bytes", "baseline_workspace_bytes", "HytopkError",
    "EXPORTS", "BF16", "FP8_E4M3", "MXFP8_E4M3", "MXFP4_E2M1", "PATH_AUTO", "PATH_ROWS_ALL", "trace_enable", "trace_read",
    "backward", "backward_workspace_bytes", "select_noalloc", "NOALLOC_SCRATCH_BYTES",
    "select_async", "ASYNC_STATUS_WORDS", "Rotary", "rotary", "cache_write", "cache_read",
    "cache_write_workspace_bytes", "quantize", "attention_mass", "attention_mass_workspace_bytes",
    "index_loss",
]

BF16, FP8_E4M3, MXFP8_E4M3, MXFP4_E2M1 = 0, 1, 2, 3
_FMT = {"bf16": BF16, "fp8": FP8_E4M3, "mxfp8": MXFP8_E4M3, "mxfp4": MXFP4_E2M1}
PATH_AUTO, PATH_ROWS_ALL = 0, 1
EXPORTS = (
    "hytopk_select_workspace", "hytopk_baseline_workspace", "hytopk_select", "hytopk_replay",
    "hytopk_baseline_select", "hytopk_backward_workspace", "hytopk_backward",
    "hytopk_status_string", "hytopk_last_error", "hytopk_trace_enable", "hytopk_trace_read",
    "hytopk_select_noalloc", "hytopk_select_async", "hytopk_rotary_frequencies", "hytopk_rotary",
    "hytopk_cache_write_workspace", "hytopk_cache_write", "hytopk_cache_read",
    "hytopk_attention_mass_workspace", "hytopk_attention_mass", "hytopk_index_loss",
)
NOALLOC_SCRATCH_BYTES = 64 << 20  # HYTOPK_NOALLOC_SCRATCH_BYTES


class Problem(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int64), ("n", ctypes.c_int64), ("q_start", ctypes.c_int64),
                ("H", ctypes.c_int32), ("d", ctypes.c_int32), ("k", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("q_pos", ctypes.c_void_p), ("q_first", ctypes.c_void_p)]


class Params(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in
                ("m_min", "m_max", "m_div", "oversample", "cap", "max_recover", "force_path",
                 "rows_chunk")]


class Stats(ctypes.Structure):
    _fields_ = [("n_overflow", ctypes.c_int32), ("n_underk", ctypes.c_int32),
                ("n_failed", ctypes.c_int32), ("full_rescore", ctypes.c_int32),
                ("cand_total", ctypes.c_int64), ("cand_max", ctypes.c_int32),
                ("path", ctypes.c_int32), ("failed_queries", ctypes.POINTER(ctypes.c_int32)),
                ("failed_capacity", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_
                if f not in ("failed_queries", "failed_capacity", "reserved")}


class TraceEntry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_double)]


class RowsArray(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class RotaryPlan(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("gain", ctypes.c_double), ("dim", ctypes.c_int32),
                ("first", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("L", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Attention(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int64), ("n", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("key_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("k", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class HytopkError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"hytopk status {status}: {msg}")
        self.status = status


_LIB = None


def library_path() -> str:
    return os.environ.get("HYTOPK_LIBRARY",
                          os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhytopk.so"))


def load_library():
    """Load libhytopk.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m exact_top_token_amd.build`")
    lib = ctypes.CDLL(path)
    P, vp, sz = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t
    lib.hytopk_select_workspace.argtypes = [P(Problem), P(Params)]
    lib.hytopk_select_workspace.restype = sz
    lib.hytopk_baseline_workspace.argtypes = [P(Problem)]
    lib.hytopk_baseline_workspace.restype = sz
    lib.hytopk_select.argtypes = [P(Problem), P(Params), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                  P(Stats)]
    lib.hytopk_select.restype = ctypes.c_int
    lib.hytopk_select_noalloc.argtypes = [P(Problem), P(Params), vp, vp, vp, vp, vp, vp, vp, vp,
                                          P(Stats)]
    lib.hytopk_select_noalloc.restype = ctypes.c_int
    lib.hytopk_select_async.argtypes = [P(Problem), P(Params), vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                        vp, vp]
    lib.hytopk_select_async.restype = ctypes.c_int
    lib.hytopk_replay.argtypes = [P(Problem), vp, vp, vp, vp, vp, vp, vp, vp]
    lib.hytopk_replay.restype = ctypes.c_int
    lib.hytopk_baseline_select.argtypes = [P(Problem), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hytopk_baseline_select.restype = ctypes.c_int
    lib.hytopk_backward_workspace.argtypes = [P(Problem)]
    lib.hytopk_backward_workspace.restype = sz
    lib.hytopk_backward.argtypes = [P(Problem), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hytopk_backward.restype = ctypes.c_int
    lib.hytopk_status_string.argtypes = [ctypes.c_int]
    lib.hytopk_status_string.restype = ctypes.c_char_p
    lib.hytopk_last_error.argtypes = []
    lib.hytopk_last_error.restype = ctypes.c_char_p
    lib.hytopk_trace_enable.argtypes = [ctypes.c_int]
    lib.hytopk_trace_enable.restype = ctypes.c_int
    lib.hytopk_trace_read.argtypes = [P(TraceEntry), ctypes.c_int]
    lib.hytopk_trace_read.restype = ctypes.c_int
    i32, i64, dbl = ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    lib.hytopk_rotary_frequencies.argtypes = [i32, dbl, i32, dbl, i64, vp, P(dbl)]
    lib.hytopk_rotary_frequencies.restype = ctypes.c_int
    lib.hytopk_rotary.argtypes = [P(RotaryPlan), i64, i32, i32, P(RowsArray), P(RowsArray), vp, i64,
                                  i32, vp]
    lib.hytopk_rotary.restype = ctypes.c_int
    lib.hytopk_cache_write_workspace.argtypes = [P(Cache), i64, i32]
    lib.hytopk_cache_write_workspace.restype = sz
    lib.hytopk_cache_write.argtypes = [P(Cache), i64, P(RowsArray), vp, i64, P(RotaryPlan), vp, i64,
                                       vp, sz, vp]
    lib.hytopk_cache_write.restype = ctypes.c_int
    lib.hytopk_cache_read.argtypes = [P(Cache), i64, vp, i64, vp, i32, vp]
    lib.hytopk_cache_read.restype = ctypes.c_int
    lib.hytopk_attention_mass_workspace.argtypes = [P(Attention)]
    lib.hytopk_attention_mass_workspace.restype = sz
    lib.hytopk_attention_mass.argtypes = [P(Attention), vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hytopk_attention_mass.restype = ctypes.c_int
    lib.hytopk_index_loss.argtypes = [i64, i32, vp, vp, vp, vp, vp, vp]
    lib.hytopk_index_loss.restype = ctypes.c_int
    _LIB = lib
    return lib


def _check(rc: int) -> None:
    if rc != 0:
        lib = load_library()
        raise HytopkError(rc, lib.hytopk_last_error().decode() or lib.hytopk_status_string(rc).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name: str, shape, dtype, device) -> None:
    """The library writes or reads these buffers by the problem's sizes, so
    a caller-given tensor must have exactly that shape and dtype, be
    contiguous and sit on the inputs' device."""
    if (tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous()
            or t.device != device):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _workspace(t, device):
    """Workspace: contiguous uint8 on the inputs' device (its size is checked by the library)."""
    import torch
    if t.dtype != torch.uint8 or t.dim() != 1 or not t.is_contiguous() or t.device != device:
        raise ValueError(f"workspace must be a contiguous 1-D uint8 tensor on {device}")
    return t


def _scales(prob, q, q_scale, k_scale) -> None:
    """Per-token fp32 scales (FP8) or E8M0 bytes per 32 elements (MX)."""
    import torch
    if prob.dtype == BF16:
        if q_scale is not None or k_scale is not None:
            raise ValueError("bf16 inputs take no q_scale / k_scale")
        return
    if q_scale is None or k_scale is None:
        raise ValueError("fp8 and MX inputs need q_scale and k_scale")
    if prob.dtype == FP8_E4M3:
        _need(q_scale, "q_scale", (prob.n,), torch.float32, q.device)
        _need(k_scale, "k_scale", (prob.L,), torch.float32, q.device)
    else:
        _need(q_scale, "q_scale", (prob.n, prob.H, prob.d // 32), torch.uint8, q.device)
        _need(k_scale, "k_scale", (prob.L, prob.d // 32), torch.uint8, q.device)


def _outputs(out, prob, device):
    import torch
    idx, score = out
    _need(idx, "out[0] (indices)", (prob.n, prob.k), torch.int32, device)
    if score is not None:
        _need(score, "out[1] (scores)", (prob.n, prob.k), torch.float32, device)
    return idx, score


def _dtype_code(q, fmt=None) -> int:
    """Storage format: ``fmt`` ("bf16", "fp8", "mxfp8", "mxfp4") when given,
    else bf16 or per-token FP8 from the tensor dtype."""
    import torch
    if fmt is not None:
        return _FMT[fmt]
    if q.dtype == torch.bfloat16:
        return BF16
    if q.dtype in (torch.float8_e4m3fn, torch.uint8):
        return FP8_E4M3
    raise TypeError(f"q/k must be bfloat16 or float8_e4m3fn, got {q.dtype}")


def _problem(q, k, w, topk: int, q_start, q_pos=None, q_first=None, fmt=None) -> Problem:
    """q [n][H][d] and k [L][d] (MXFP4: the last axis holds d/2 bytes)."""
    import torch
    code = _dtype_code(q, fmt)
    n, H, dq = q.shape
    d = 2 * dq if code == MXFP4_E2M1 else dq
    L = k.shape[0]
    if k.shape[1] != dq or tuple(w.shape) != (n, H):
        raise ValueError("shapes must be q [n][H][d], k [L][d], w [n][H]")
    for t in (q, k, w):
        if not t.is_cuda or not t.is_contiguous() or t.device != q.device:
            raise ValueError("q, k and w must be contiguous and on the same GPU")
    if w.dtype != torch.float32:
        raise ValueError("w must be float32")
    if k.dtype != q.dtype or (code in (MXFP8_E4M3, MXFP4_E2M1) and q.dtype != torch.uint8):
        raise ValueError("q and k must share a dtype (uint8 codes for the MX formats)")
    for t in (q_pos, q_first):
        if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (n,)
                              or t.device != q.device or not t.is_contiguous()):
            raise ValueError("q_pos / q_first must be contiguous int32 [n] tensors on the GPU")
    if q_start is None:
        q_start = 0 if q_pos is not None else L - n
    return Problem(L, n, int(q_start), H, d, int(topk), code,
                   None if q_pos is None else q_pos.data_ptr(),
                   None if q_first is None else q_first.data_ptr())


def _params(params) -> Params | None:
    if params is None:
        return None
    if isinstance(params, Params):
        return params
    p = Params()
    for key, val in dict(params).items():
        setattr(p, key, int(val))
    return p


def _stream(t):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def trace_enable(on: bool = True) -> bool:
    """Bracket every library launch with hipEvents (clears the totals)."""
    return bool(load_library().hytopk_trace_enable(1 if on else 0))


def trace_read() -> dict:
    """{phase: (launches, total_ms)} accumulated since tracing was enabled."""
    lib = load_library()
    n = lib.hytopk_trace_read(None, 0)
    if n < 0:
        _check(n)
    arr = (TraceEntry * max(n, 1))()
    n = lib.hytopk_trace_read(arr, n)
    if n < 0:
        _check(n)
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n)}


def select_workspace_bytes(q, k, w, topk: int, q_start=None, params=None, q_pos=None,
                           q_first=None, fmt=None) -> int:
    lib = load_library()
    prob = _problem(q, k, w, topk, q_start, q_pos, q_first, fmt)
    prm = _params(params)
    return int(lib.hytopk_select_workspace(ctypes.byref(prob), ctypes.byref(prm) if prm else None))


def baseline_workspace_bytes(q, k, w, topk: int, q_start=None, fmt=None) -> int:
    lib = load_library()
    return int(lib.hytopk_baseline_workspace(ctypes.byref(_problem(q, k, w, topk, q_start,
                                                                   fmt=fmt))))


def select(q, k, w, topk: int, *, q_scale=None, k_scale=None, q_start=None, params=None,
           workspace=None, out=None, with_stats: bool = False, q_pos=None, q_first=None,
           fmt=None):
    """Exact top-k per query (HyTopK).  Returns (idx int32 [n][k], score fp32
    [n][k]) and, with ``with_stats``, a dict of what the call did.  q_pos /
    q_first (int32 [n] on the GPU, optional) give each query's position and
    the first key of its context (packed sequences).  ``fmt`` selects the MX
    formats ("mxfp8", "mxfp4"; q_scale / k_scale then hold E8M0 bytes)."""
    import torch
    lib = load_library()
    prob = _problem(q, k, w, topk, q_start, q_pos, q_first, fmt)
    _scales(prob, q, q_scale, k_scale)
    prm = _params(params)
    need = int(lib.hytopk_select_workspace(ctypes.byref(prob), ctypes.byref(prm) if prm else None))
    if need == 0:
        _check(lib.hytopk_select(ctypes.byref(prob), ctypes.byref(prm) if prm else None,
                                 *([None] * 8), 0, None, None))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _workspace(workspace, q.device)
    if out is None:
        idx = torch.empty((prob.n, prob.k), dtype=torch.int32, device=q.device)
        score = torch.empty((prob.n, prob.k), dtype=torch.float32, device=q.device)
    else:
        idx, score = _outputs(out, prob, q.device)
    st = Stats()
    failed_buf = None
    if with_stats:
        failed_buf = (ctypes.c_int32 * int(prob.n))()
        st.failed_queries = ctypes.cast(failed_buf, ctypes.POINTER(ctypes.c_int32))
        st.failed_capacity = int(prob.n)
    _check(lib.hytopk_select(ctypes.byref(prob), ctypes.byref(prm) if prm else None, _ptr(q),
                             _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(idx), _ptr(score),
                             _ptr(workspace), workspace.numel(), _stream(q), ctypes.byref(st)))
    if not with_stats:
        return idx, score
    d = st.as_dict()
    d["failed"] = [failed_buf[i] for i in range(min(st.n_failed, int(prob.n)))]
    return idx, score, d


def select_noalloc(q, k, w, topk: int, out, *, q_scale=None, k_scale=None, q_start=None,
                   params=None, q_pos=None, q_first=None, fmt=None, with_stats: bool = False):
    """hytopk_select_noalloc: select into the caller's ``out`` = (idx, score)
    tensors with the library's static scratch as workspace (no allocation on
    the device).  Returns ``out`` and, with ``with_stats``, the stats dict."""
    lib = load_library()
    prob = _problem(q, k, w, topk, q_start, q_pos, q_first, fmt)
    _scales(prob, q, q_scale, k_scale)
    prm = _params(params)
    idx, score = _outputs(out, prob, q.device)
    st = Stats()
    failed_buf = None
    if with_stats:
        failed_buf = (ctypes.c_int32 * int(prob.n))()
        st.failed_queries = ctypes.cast(failed_buf, ctypes.POINTER(ctypes.c_int32))
        st.failed_capacity = int(prob.n)
    _check(lib.hytopk_select_noalloc(ctypes.byref(prob), ctypes.byref(prm) if prm else None,
                                     _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                                     _ptr(idx), _ptr(score), _stream(q), ctypes.byref(st)))
    if not with_stats:
        return idx, score
    d = st.as_dict()
    d["failed"] = [failed_buf[i] for i in range(min(st.n_failed, int(prob.n)))]
    return idx, score, d


ASYNC_STATUS_WORDS = 8


def select_async(q, k, w, topk: int, *, workspace, out, status, q_scale=None, k_scale=None,
                 q_start=None, params=None, q_pos=None, q_first=None, fmt=None):
    """hytopk_select_async: select into ``out`` = (idx, score) with the caller's
    ``workspace`` (select_workspace_bytes) and no host synchronisation, so the
    call can be recorded in a CUDA/HIP graph.  ``status`` (int32
    [ASYNC_STATUS_WORDS] on the GPU) receives the device status words:
    status[0] == 1 means more than max_recover queries failed and their rows
    are not final.  Returns ``out``."""
    import torch
    lib = load_library()
    prob = _problem(q, k, w, topk, q_start, q_pos, q_first, fmt)
    _scales(prob, q, q_scale, k_scale)
    prm = _params(params)
    idx, score = _outputs(out, prob, q.device)
    _workspace(workspace, q.device)
    if (status.dtype != torch.int32 or status.numel() < ASYNC_STATUS_WORDS
            or not status.is_contiguous() or status.device != q.device):
        raise ValueError("status must be a contiguous int32 tensor of ASYNC_STATUS_WORDS entries "
                         "on the inputs' device")
    _check(lib.hytopk_select_async(ctypes.byref(prob), ctypes.byref(prm) if prm else None,
                                   _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                                   _ptr(idx), _ptr(score), _ptr(workspace), workspace.numel(),
                                   _stream(q), _ptr(status)))
    return idx, score


def replay(q, k, w, idx, *, q_scale=None, k_scale=None, q_start=None, out=None, fmt=None):
    """Selection replay: scores of the saved indices idx [n][k] (-inf at idx < 0)."""
    import torch
    lib = load_library()
    prob = _problem(q, k, w, idx.shape[1], q_start, fmt=fmt)
    _scales(prob, q, q_scale, k_scale)
    _need(idx, "idx", (prob.n, prob.k), torch.int32, q.device)
    if out is None:
        out = torch.empty(idx.shape, dtype=torch.float32, device=q.device)
    _need(out, "out", (prob.n, prob.k), torch.float32, q.device)
    _check(lib.hytopk_replay(ctypes.byref(prob), _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale),
                             _ptr(w), _ptr(idx), _ptr(out), _stream(q)))
    return out


def baseline_select(q, k, w, topk: int, *, q_scale=None, k_scale=None, q_start=None,
                    workspace=None, out=None, q_pos=None, q_first=None, fmt=None):
    """The materialise-then-top-k route (writes the n x L fp32 score table)."""
    import torch
    lib = load_library()
    prob = _problem(q, k, w, topk, q_start, q_pos, q_first, fmt)
    _scales(prob, q, q_scale, k_scale)
    need = int(lib.hytopk_baseline_workspace(ctypes.byref(prob)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _workspace(workspace, q.device)
    if out is None:
        idx = torch.empty((prob.n, prob.k), dtype=torch.int32, device=q.device)
        score = torch.empty((prob.n, prob.k), dtype=torch.float32, device=q.device)
    else:
        idx, score = _outputs(out, prob, q.device)
    _check(lib.hytopk_baseline_select(ctypes.byref(prob), _ptr(q), _ptr(q_scale), _ptr(k),
                                      _ptr(k_scale), _ptr(w), _ptr(idx), _ptr(score),
                                      _ptr(workspace), workspace.numel(), _stream(q)))
    return idx, score


def backward_workspace_bytes(q, k, w, topk: int, q_start=None, fmt=None) -> int:
    lib = load_library()
    return int(lib.hytopk_backward_workspace(ctypes.byref(_problem(q, k, w, topk, q_start,
                                                                   fmt=fmt))))


def backward(q, k, w, idx, d_score, *, q_scale=None, k_scale=None, q_start=None,
             want=("dq", "dw", "dk"), workspace=None, out=None, fmt=None):
    """Indexer backward at the replayed entries idx [n][k] with upstream
    gradient d_score [n][k] (fp32).  Returns a dict with the requested fp32
    gradients: dq [n][H][d], dw [n][H], dk [L][d] (for FP8 / MX inputs, with
    respect to the decoded values)."""
    import torch
    lib = load_library()
    prob = _problem(q, k, w, idx.shape[1], q_start, fmt=fmt)
    _scales(prob, q, q_scale, k_scale)
    _need(idx, "idx", (prob.n, prob.k), torch.int32, q.device)
    _need(d_score, "d_score", (prob.n, prob.k), torch.float32, q.device)
    res = dict(out or {})
    shapes = {"dq": (prob.n, prob.H, prob.d), "dw": (prob.n, prob.H), "dk": (prob.L, prob.d)}
    if set(res) - set(shapes):
        raise ValueError(f"unknown gradient names in out: {sorted(set(res) - set(shapes))}")
    for name in want:
        if name not in res:
            res[name] = torch.empty(shapes[name], dtype=torch.float32, device=q.device)
    for name, t in res.items():
        _need(t, name, shapes[name], torch.float32, q.device)
    if ("dk" in res or prob.dtype != BF16) and workspace is None:
        need = int(lib.hytopk_backward_workspace(ctypes.byref(prob)))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if workspace is not None:
        _workspace(workspace, q.device)
    _check(lib.hytopk_backward(ctypes.byref(prob), _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale),
                               _ptr(w), _ptr(idx), _ptr(d_score), _ptr(res.get("dq")),
                               _ptr(res.get("dw")), _ptr(res.get("dk")), _ptr(workspace),
                               0 if workspace is None else workspace.numel(), _stream(q)))
    return res


# ----------------------------------------- rotary positions and the cache

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def _launch(device, fn, *args) -> None:
    """Calls fn(*args, stream) on the device's current stream, with that device
    current (a call's host time is most of a small operator's, so nothing here
    builds a stream or a guard object that is not needed)."""
    import torch
    index = device.index
    if index == torch.cuda.current_device():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc != 0:
        _check(rc)


def _gpu(t, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")


def _rows_array(t, name: str):
    """[n][d] or [n][heads][d] rows of bf16 or fp32, any strides but the last."""
    import torch
    dtype, stride = t.dtype, t.stride()
    if dtype != torch.bfloat16 and dtype != torch.float32:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    axes = len(stride)
    if axes != 2 and axes != 3:
        raise ValueError(f"{name} must be [n][d] or [n][heads][d], got {tuple(t.shape)}")
    if stride[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return RowsArray(t.data_ptr(), stride[0], stride[1] if axes == 3 else 0,
                     0 if dtype == torch.bfloat16 else 1, 0)


def _address(t):
    return None if t is None else t.data_ptr()


def _ints(t, name: str, n: int, device) -> None:
    import torch
    if t is not None:
        _need(t, name, (n,), torch.int32, device)


class Rotary:
    """A rotation of elements ``first .. first + dim - 1`` of every head: the
    frequencies (``freq``, float64 on the GPU) and the factor on the rotated
    part (``gain``), made once and kept for every call.  ``layout`` pairs
    elements (i, i + dim/2) ("half") or (2i, 2i + 1) ("interleaved");
    ``scaling`` ("none", "linear", "ntk", "yarn") stretches the positions by
    ``factor`` for a model whose positions reached ``original`` before."""

    def __init__(self, dim: int, *, first: int = 0, layout: str = "half", base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, original: int = 0, device="cuda"):
        import torch
        if layout not in _LAYOUTS:
            raise ValueError(f"unknown rotary layout {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"unknown rotary scaling {scaling!r}")
        dim, first, original = int(dim), int(first), int(original)
        if not (0 < dim < 1 << 31 and 0 <= first < 1 << 31):
            raise ValueError("dim must be > 0 and first >= 0, both below 2^31")
        lib = load_library()
        freq = torch.empty(max(min(dim, 1024) // 2, 1), dtype=torch.float64)
        gain = ctypes.c_double()
        _check(lib.hytopk_rotary_frequencies(dim, float(base), _SCALINGS[scaling], float(factor),
                                             original, _ptr(freq), ctypes.byref(gain)))
        self.freq = freq.to(device)
        self.gain, self.dim, self.first, self.layout = gain.value, dim, first, layout
        self._plan = RotaryPlan(self.freq.data_ptr(), self.gain, self.dim, self.first,
                                _LAYOUTS[layout], 0)


def _plan(rot, device):
    if rot is None:
        return None
    if rot.freq.device != device:
        raise ValueError(f"the rotary plan is on {rot.freq.device}, the rows on {device}")
    return rot._plan


def rotary(x, rot: Rotary, *, q_start: int = 0, q_pos=None, backward: bool = False, out=None,
           out_dtype=None):
    """Rotary positions of rows x [n][d] or [n][heads][d] (bf16 or fp32, any
    strides but the last).  Token i sits at ``q_pos[i]`` (int32 [n] on the GPU) or
    ``q_start + i``.  ``backward`` applies the transposed rotation, which
    takes a gradient of the result to one of x.  ``out`` may be x itself."""
    import torch
    lib = _LIB or load_library()
    _gpu(x, "x")
    xa = _rows_array(x, "x")
    shape, device = x.shape, x.device
    n, d = shape[0], shape[-1]
    heads = shape[1] if len(shape) == 3 else 1
    if out is None:
        out = x.new_empty(shape, dtype=out_dtype)
    elif out.shape != x.shape or out.device != x.device or out_dtype not in (None, out.dtype):
        raise ValueError(f"out must have x's shape {tuple(x.shape)} and device, and out_dtype")
    ya = _rows_array(out, "out")
    _ints(q_pos, "q_pos", n, device)
    _launch(device, lib.hytopk_rotary, _plan(rot, device), n, heads, d, xa, ya, _address(q_pos),
            int(q_start), 1 if backward else 0)
    return out


def _cache(codes, scale, fmt):
    """codes [L][d] or [L][heads][d] (MXFP4: the last axis holds d/2 bytes) and
    scales as ``select`` takes them."""
    import torch
    _gpu(codes, "codes")
    code = _dtype_code(codes, fmt)
    shape = codes.shape
    axes = len(shape)
    if axes != 2 and axes != 3:
        raise ValueError(f"codes must be [L][d] or [L][heads][d], got {tuple(shape)}")
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    dtype = codes.dtype
    if dtype != (torch.bfloat16 if code == BF16 else torch.uint8) and not (
            code == FP8_E4M3 and dtype == torch.float8_e4m3fn):
        raise ValueError(f"codes of type {dtype} do not hold this format")
    L, last = shape[0], shape[-1]
    heads = shape[1] if axes == 3 else 1
    d = 2 * last if code == MXFP4_E2M1 else last
    if code == BF16:
        if scale is not None:
            raise ValueError("a bf16 cache takes no scale")
        return Cache(codes.data_ptr(), None, L, heads, d, code, 0)
    if scale is None:
        raise ValueError("fp8 and MX caches need scale")
    if code == FP8_E4M3:
        _need(scale, "scale", (L,), torch.float32, codes.device)
    else:
        _need(scale, "scale", (*shape[:-1], d // 32), torch.uint8, codes.device)
    return Cache(codes.data_ptr(), scale.data_ptr(), L, heads, d, code, 0)


def cache_write_workspace_bytes(codes, scale, n: int, *, fmt=None) -> int:
    """Workspace bytes of a cache_write of n rows by slot (0: none)."""
    return int(load_library().hytopk_cache_write_workspace(
        ctypes.byref(_cache(codes, scale, fmt)), n, 1))


def cache_write(x, codes, scale=None, *, fmt=None, start: int = 0, slots=None, rotary=None,
                q_start: int = 0, q_pos=None, workspace=None) -> None:
    """Quantise rows x ([n][d] or [n][heads][d], bf16 or fp32, any strides but the
    last) into cache rows ``slots[i]`` (int32 [n] on the GPU; rows outside the
    cache are padding and skipped; the last of several rows of one slot is
    kept) or ``start + i``.  ``codes`` and ``scale`` are laid out as ``select`` takes them
    (``fmt`` as there).  ``rotary`` (a Rotary) rotates the rows first, at positions
    ``q_pos`` / ``q_start + i``."""
    import torch
    lib = _LIB or load_library()
    c = _cache(codes, scale, fmt)
    xa = _rows_array(x, "x")
    n = x.shape[0]
    device, shape = x.device, x.shape
    if device != codes.device:
        raise ValueError(f"x is on {device}, the cache on {codes.device}")
    if shape[-1] != c.d or (shape[1] if len(shape) == 3 else 1) != c.heads:
        raise ValueError(f"x {tuple(shape)} does not fit cache rows of {c.heads} x {c.d}")
    _ints(slots, "slots", n, device)
    _ints(q_pos, "q_pos", n, device)
    if workspace is None and slots is not None:
        need = lib.hytopk_cache_write_workspace(c, n, 1)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is not None:
        _workspace(workspace, device)
    _launch(device, lib.hytopk_cache_write, c, n, xa, _address(slots), int(start),
            _plan(rotary, device), _address(q_pos), int(q_start), _address(workspace),
            0 if workspace is None else workspace.numel())


def quantize(x, fmt: str, *, rotary=None, q_start: int = 0, q_pos=None):
    """Rows x ([n][d] or [n][heads][d]) in a storage format of ``select``: new
    (codes, scale), scale None for "bf16".  ``rotary`` as in ``cache_write``."""
    import torch
    if fmt not in _FMT:
        raise ValueError(f"unknown format {fmt!r}")
    _gpu(x, "x")
    code, shape, d = _FMT[fmt], tuple(x.shape), x.shape[-1]
    if code != BF16 and d % 32:
        raise ValueError("quantised rows need d in multiples of 32")
    codes = torch.empty(shape[:-1] + (d // 2 if code == MXFP4_E2M1 else d,), device=x.device,
                        dtype=torch.bfloat16 if code == BF16 else torch.uint8)
    scale = None
    if code == FP8_E4M3:
        scale = torch.empty(shape[0], dtype=torch.float32, device=x.device)
    elif code != BF16:
        scale = torch.empty(shape[:-1] + (d // 32,), dtype=torch.uint8, device=x.device)
    if shape[0]:
        cache_write(x, codes, scale, fmt=fmt, rotary=rotary, q_start=q_start, q_pos=q_pos)
    return codes, scale


def cache_read(codes, scale=None, *, fmt=None, slots=None, start: int = 0, count=None,
               dtype=None, out=None):
    """Cache rows decoded: rows ``slots`` (int32 [n] on the GPU; rows outside the cache read as
    zeros) or ``start .. start + count - 1`` (to the end by default), as [n][d]
    or [n][heads][d] of ``dtype`` (bf16 by default, or fp32)."""
    import torch
    lib = _LIB or load_library()
    c = _cache(codes, scale, fmt)
    n = slots.shape[0] if slots is not None else (c.L - int(start) if count is None else int(count))
    if count is not None and n != count:
        raise ValueError(f"count {count} differs from the {n} slots")
    _ints(slots, "slots", n, codes.device)
    shape = (n, c.d) if codes.dim() == 2 else (n, c.heads, c.d)
    device = codes.device
    if out is None:
        if n < 0:
            raise ValueError("start lies behind the cache")
        out = codes.new_empty(shape, dtype=dtype or torch.bfloat16)
    else:
        _need(out, "out", shape, dtype or out.dtype, device)
    dtype = out.dtype
    if dtype != torch.bfloat16 and dtype != torch.float32:
        raise TypeError(f"rows are read as bfloat16 or float32, got {dtype}")
    _launch(device, lib.hytopk_cache_read, c, n, _address(slots), int(start), out.data_ptr(),
            0 if dtype == torch.bfloat16 else 1)
    return out


# ------------------------------------------- the indexer's target and loss

def _attention(q, k, idx, softmax_scale) -> Attention:
    """q [n][heads][d], k [L][key_heads][d] or [L][d], idx [n][k]."""
    import torch
    if q.dim() != 3 or k.dim() not in (2, 3) or k.shape[-1] != q.shape[-1]:
        raise ValueError("shapes must be q [n][heads][d], k [L][key_heads][d] or [L][d]")
    device = q.device
    for t, name in ((q, "q"), (k, "k")):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.device != device:
            raise ValueError(f"{name} must be contiguous bfloat16 on one GPU")
    n, heads, d = q.shape
    rows = k.shape
    if idx.dim() != 2:
        raise ValueError("idx must be [n][k]")
    count = idx.shape[1]
    _need(idx, "idx", (n, count), torch.int32, device)
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    return Attention(rows[0], n, heads, rows[1] if len(rows) == 3 else 1, d, count, scale, 0)


def attention_mass_workspace_bytes(q, k, idx) -> int:
    """Workspace bytes of attention_mass without lse."""
    return int(load_library().hytopk_attention_mass_workspace(
        ctypes.byref(_attention(q, k, idx, None))))


def attention_mass(q, k, idx, *, softmax_scale=None, lse=None, workspace=None, out=None):
    """The attention's probability at the selected entries idx [n][k], averaged
    over heads (fp32 [n][k]; 0 at padding): the target of ``index_loss``.
    q [n][heads][d] and k [L][key_heads][d] (or [L][d]) are the attention's, bf16;
    ``softmax_scale`` is d ** -0.5 by default; ``lse`` (fp32 [n][heads]) is the attention's
    log-sum-exp, by default taken over the row's entries."""
    import torch
    lib = _LIB or load_library()
    p = _attention(q, k, idx, softmax_scale)
    device = q.device
    if lse is not None:
        _need(lse, "lse", (p.n, p.heads), torch.float32, device)
    if out is None:
        out = q.new_empty((p.n, p.k), dtype=torch.float32)
    else:
        _need(out, "out", (p.n, p.k), torch.float32, device)
    if workspace is None and lse is None:
        workspace = torch.empty(max(lib.hytopk_attention_mass_workspace(p), 1), dtype=torch.uint8,
                                device=device)
    if workspace is not None:
        _workspace(workspace, device)
    _launch(device, lib.hytopk_attention_mass, p, q.data_ptr(), k.data_ptr(), idx.data_ptr(),
            _address(lse), out.data_ptr(), _address(workspace),
            0 if workspace is None else workspace.numel())
    return out


def index_loss(score, mass, *, weight=None, want=("loss", "d_score"), out=None):
    """The indexer's loss per query and its gradient: the divergence of
    softmax(score) from mass / sum(mass) over the entries whose score is not -inf,
    times ``weight`` (fp32 [n], 1 by default).  score (``replay``'s) and mass
    (``attention_mass``'s) are fp32 [n][k].  Returns (loss [n], d_score [n][k]),
    None for one that ``want`` leaves out; ``backward`` takes d_score.  ``out`` gives
    the two tensors instead (either may be None; d_score may be score or mass)."""
    import torch
    lib = _LIB or load_library()
    _gpu(score, "score")
    if score.dim() != 2:
        raise ValueError("score must be [n][k]")
    n, k = score.shape
    dev = score.device
    _need(score, "score", (n, k), torch.float32, dev)
    _need(mass, "mass", (n, k), torch.float32, dev)
    if weight is not None:
        _need(weight, "weight", (n,), torch.float32, dev)
    if out is None:
        loss = score.new_empty(n) if "loss" in want else None
        grad = torch.empty_like(score) if "d_score" in want else None
    else:
        loss, grad = out
        if loss is not None:
            _need(loss, "out[0] (loss)", (n,), torch.float32, dev)
        if grad is not None:
            _need(grad, "out[1] (d_score)", (n, k), torch.float32, dev)
    _launch(dev, lib.hytopk_index_loss, n, k, score.data_ptr(), mass.data_ptr(), _address(weight),
            _address(loss), _address(grad))
    return loss, grad
