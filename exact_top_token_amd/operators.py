"""Bindings of the operators around the selection: layer norm and its 8-bit checkpoints, rotary
positions, the quantised cache, the attention's mass at the selected entries and the indexer's loss.

As in the package's own module only tensors are marshalled here; the kernels run on
the tensors' GPU and its current stream.  A call's host time is most of a small
operator's, so these functions build no stream, guard or pointer object that a
call does not need, and make results like an argument where they can (0.9 us against 1.4).
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import (BF16, FP8_E4M3, MXFP4_E2M1, MXFP8_E4M3, _FMT, Attention, Cache, Norm, RotaryPlan, RowsArray, _check,
               _dtype_code, _workspace, load_library)

__all__ = ["Rotary", "rotary", "cache_write", "cache_read", "cache_write_workspace_bytes",
           "quantize", "NormSaved", "layer_norm", "layer_norm_backward", "layer_norm_backward_workspace_bytes",
           "attention_mass", "attention_mass_workspace_bytes", "index_loss"]

_EWORKSPACE = -3  # HYTOPK_EWORKSPACE
_bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_empty_like, _contiguous = torch.empty_like, torch.contiguous_format


def _call(device, fn, *args) -> int:
    """The status of fn(*args, stream) on the device's current stream, with that device
    current."""
    index = device.index
    if index == _current_device():
        return fn(*args, _raw_stream(index))
    with torch.cuda.device(device):
        return fn(*args, _raw_stream(index))


def _launch(device, fn, *args) -> None:
    rc = _call(device, fn, *args)
    if rc != 0:
        _check(rc)


def _need(t, name: str, shape, dtype, device) -> None:
    """The library reads and writes by sizes, so a tensor must have exactly this
    shape and dtype, be contiguous and sit on the call's device."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _gpu(t, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")


def _rows_array(t, name: str) -> RowsArray:
    """[n][d] or [n][heads][d] rows of bf16 or fp32, any strides but the last."""
    dtype, stride = t.dtype, t.stride()
    if dtype != _bf16 and dtype != _f32:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    axes = len(stride)
    if axes != 2 and axes != 3:
        raise ValueError(f"{name} must be [n][d] or [n][heads][d], got {tuple(t.shape)}")
    if stride[-1] != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError(f"the last axis of {name} must be contiguous")
    return RowsArray(t.data_ptr(), stride[0], stride[1] if axes == 3 else 0,
                     0 if dtype == _bf16 else 1, 0)


def _address(t):
    return None if t is None else t.data_ptr()


# ----------------------------------------- rotary positions and the cache

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class Rotary:
    """A rotation of elements ``first .. first + dim - 1`` of every head: the
    frequencies (``freq``, float64 on the GPU) and the factor on the rotated
    part (``gain``), made once and kept for every call.  ``layout`` pairs
    elements (i, i + dim/2) ("half") or (2i, 2i + 1) ("interleaved");
    ``scaling`` ("none", "linear", "ntk", "yarn") stretches the positions by
    ``factor`` for a model whose positions reached ``original`` before.  ``gain`` replaces the
    scaling's own factor (YaRN: 0.1 ln(factor) + 1; else 1), and ``freq``
    [dim/2] (radians a position) the frequencies, for a model with its own.

    ``sections`` (pairs of each axis, dim/2 in all) is for tokens with a position on
    each of several axes, such as time, height and width; ``q_pos`` is then int32 [n][axes] ([n] for one).  The axes'
    pairs lie one behind the other or, with ``cycle``, in turn: axis a > 0 takes pairs a, a + A, a + 2A, ... of A axes,
    as many as it has, and axis 0 the others.  ``restart`` begins the frequencies anew on each axis, as those of a
    rotation of its pairs alone."""

    def __init__(self, dim: int, *, first: int = 0, layout: str = "half", base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, original: int = 0, gain=None, freq=None,
                 sections=None, cycle: bool = False, restart: bool = False, device="cuda"):
        if layout not in _LAYOUTS:
            raise ValueError(f"unknown rotary layout {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"unknown rotary scaling {scaling!r}")
        dim, first, original = int(dim), int(first), int(original)
        if not (0 < dim < 1 << 31 and 0 <= first < 1 << 31):
            raise ValueError("dim must be > 0 and first >= 0, both below 2^31")
        factor_on = ctypes.c_double()

        def frequencies(dim):
            made = torch.empty(max(min(dim, 1024) // 2, 1), dtype=torch.float64)
            _check(load_library().hytopk_rotary_frequencies(dim, float(base), _SCALINGS[scaling], float(factor),
                                                            original, made.data_ptr(), ctypes.byref(factor_on)))
            return made

        made = frequencies(dim)
        sections = None if sections is None else tuple(sections)
        axis, axes = _axis_of_pairs(dim // 2, sections, cycle), 1 if sections is None else len(sections)
        if freq is not None:
            own = torch.as_tensor(freq).detach().cpu()
            if scaling != "none" or restart or own.shape != made.shape or not torch.isfinite(own).all():
                raise ValueError(f"freq must hold {dim // 2} finite values, and takes no scaling or restart")
            made.copy_(own)
        elif restart:
            if sections is None:
                raise ValueError("restart needs sections")
            for a in range(axes):
                made[axis == a] = frequencies(2 * int(sections[a]))
        gain = factor_on.value if gain is None else float(gain)
        if not math.isfinite(gain):
            raise ValueError("gain must be finite")
        half = made.numel()
        if axes > 1:  # the pairs' axes lie behind the frequencies
            table = torch.zeros(half + (half + 1) // 2, dtype=torch.float64)
            table[:half] = made
            table[half:].view(_i32)[:half] = axis
            made = table
        made = made.to(device)
        self.freq = made[:half]
        self.axis = made[half:].view(_i32)[:half] if axes > 1 else None
        self.gain, self.dim, self.first, self.layout, self.axes = gain, dim, first, layout, axes
        self._plan = RotaryPlan(self.freq.data_ptr(), self.gain, dim, first, _LAYOUTS[layout], axes if axes > 1 else 0)


def _axis_of_pairs(pairs: int, sections, cycle: bool):
    """The axis of each of a rotation's pairs (int32 [pairs])."""
    axis = torch.zeros(pairs, dtype=_i32)
    if sections is None:
        if cycle:
            raise ValueError("cycle needs sections")
        return axis
    counts = [int(s) for s in sections]
    A = len(counts)
    if not 1 <= A <= 16 or min(counts) < 1 or sum(counts) != pairs:
        raise ValueError(f"sections must give 1 to 16 axes one pair or more each, {pairs} in all, got {counts}")
    at = 0
    for a, s in enumerate(counts):
        if not cycle:
            axis[at:at + s] = a
            at += s
        elif a:
            if a + (s - 1) * A >= pairs:
                raise ValueError(f"axis {a} has {s} pairs, more than its turns among {pairs} pairs")
            axis[a:a + s * A:A] = a
    return axis


def _plan(rot, device):
    if rot is None:
        return None
    if rot.freq.device != device:
        raise ValueError(f"the rotary plan is on {rot.freq.device}, the rows on {device}")
    return rot._plan


def _positions(n, rot):
    """The shape of n tokens' positions."""
    return (n,) if rot is None or rot.axes == 1 else (n, rot.axes)


def rotary(x, rot: Rotary, *, q_start: int = 0, q_pos=None, backward: bool = False, out=None,
           out_dtype=None):
    """Rotary positions of rows x [n][d] or [n][heads][d] (bf16 or fp32, any
    strides but the last).  Token i sits at ``q_pos[i]`` (int32 [n] on the GPU) or
    ``q_start + i``.  ``backward`` applies the transposed rotation, which
    takes a gradient of the result to one of x.  A plan of several axes takes ``q_pos``
    [n][axes].  ``out`` may be x itself."""
    _gpu(x, "x")
    xa = _rows_array(x, "x")
    shape, device = x.shape, x.device
    n, d = shape[0], shape[-1]
    heads = shape[1] if len(shape) == 3 else 1
    if out is None and (out_dtype is None or out_dtype == x.dtype):
        out = _empty_like(x, memory_format=_contiguous)
        ya = RowsArray(out.data_ptr(), heads * d, d, xa.dtype, 0)
    else:
        if out is None:
            out = x.new_empty(shape, dtype=out_dtype)
        elif out.shape != shape or out.device != device or out_dtype not in (None, out.dtype):
            raise ValueError(f"out must have x's shape {tuple(shape)} and device, and out_dtype")
        ya = _rows_array(out, "out")
    if q_pos is not None:
        _need(q_pos, "q_pos", _positions(n, rot), _i32, device)
    _launch(device, load_library().hytopk_rotary, _plan(rot, device), n, heads, d, xa, ya,
            _address(q_pos), int(q_start), 1 if backward else 0)
    return out


def _cache(codes, scale, fmt) -> Cache:
    """codes [L][d] or [L][heads][d] (MXFP4: the last axis holds d/2 bytes) and
    scales as ``select`` takes them."""
    _gpu(codes, "codes")
    code = _dtype_code(codes) if fmt is None else _FMT[fmt]
    shape, dtype = codes.shape, codes.dtype
    axes = len(shape)
    if axes != 2 and axes != 3:
        raise ValueError(f"codes must be [L][d] or [L][heads][d], got {tuple(shape)}")
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    if dtype != (_bf16 if code == BF16 else _u8) and not (
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
        _need(scale, "scale", (L,), _f32, codes.device)
    else:
        _need(scale, "scale", (*shape[:-1], d // 32), _u8, codes.device)
    return Cache(codes.data_ptr(), scale.data_ptr(), L, heads, d, code, 0)


def cache_write_workspace_bytes(codes, scale, n: int, *, fmt=None) -> int:
    """Workspace bytes of a cache_write of n rows by slot (0: none)."""
    return int(load_library().hytopk_cache_write_workspace(_cache(codes, scale, fmt), n, 1))


def cache_write(x, codes, scale=None, *, fmt=None, start: int = 0, slots=None, rotary=None,
                q_start: int = 0, q_pos=None, workspace=None) -> None:
    """Quantise rows x ([n][d] or [n][heads][d], bf16 or fp32, any strides but the
    last) into cache rows ``slots[i]`` (int32 [n] on the GPU; rows outside the
    cache are padding and skipped; the last of several rows of one slot is
    kept) or ``start + i``.  ``codes`` and ``scale`` are laid out as ``select`` takes them
    (``fmt`` as there).  ``rotary`` (a Rotary) rotates the rows first, at positions
    ``q_pos`` / ``q_start + i``."""
    lib = load_library()
    c = _cache(codes, scale, fmt)
    xa = _rows_array(x, "x")
    device, shape = x.device, x.shape
    n = shape[0]
    if device != codes.device:
        raise ValueError(f"x is on {device}, the cache on {codes.device}")
    if shape[-1] != c.d or (shape[1] if len(shape) == 3 else 1) != c.heads:
        raise ValueError(f"x {tuple(shape)} does not fit cache rows of {c.heads} x {c.d}")
    if q_pos is not None:
        _need(q_pos, "q_pos", _positions(n, rotary), _i32, device)
    if slots is not None:
        _need(slots, "slots", (n,), _i32, device)
    if workspace is not None:
        _workspace(workspace, device)
    args = (c, n, xa, _address(slots), int(start), _plan(rotary, device), _address(q_pos), int(q_start))
    rc = _call(device, lib.hytopk_cache_write, *args, _address(workspace),
               0 if workspace is None else workspace.numel())
    if rc == _EWORKSPACE and workspace is None:  # many rows by slot; few need none, so it is not asked before
        workspace = torch.empty(lib.hytopk_cache_write_workspace(c, n, 1), dtype=_u8, device=device)
        rc = _call(device, lib.hytopk_cache_write, *args, workspace.data_ptr(), workspace.numel())
    if rc != 0:
        _check(rc)


def quantize(x, fmt: str, *, rotary=None, q_start: int = 0, q_pos=None):
    """Rows x ([n][d] or [n][heads][d]) in a storage format of ``select``: new
    (codes, scale), scale None for "bf16".  ``rotary`` as in ``cache_write``."""
    if fmt not in _FMT:
        raise ValueError(f"unknown format {fmt!r}")
    _gpu(x, "x")
    code, shape = _FMT[fmt], tuple(x.shape)
    d = shape[-1]
    if code != BF16 and d % 32:
        raise ValueError("quantised rows need d in multiples of 32")
    codes = x.new_empty(shape[:-1] + (d // 2 if code == MXFP4_E2M1 else d,),
                        dtype=_bf16 if code == BF16 else _u8)
    scale = None
    if code == FP8_E4M3:
        scale = x.new_empty(shape[0], dtype=_f32)
    elif code != BF16:
        scale = x.new_empty(shape[:-1] + (d // 32,), dtype=_u8)
    if shape[0]:
        cache_write(x, codes, scale, fmt=fmt, rotary=rotary, q_start=q_start, q_pos=q_pos)
    return codes, scale


def cache_read(codes, scale=None, *, fmt=None, slots=None, start: int = 0, count=None,
               dtype=None, out=None):
    """Cache rows decoded: rows ``slots`` (int32 [n] on the GPU; rows outside the cache read as
    zeros) or ``start .. start + count - 1`` (to the end by default), as [n][d]
    or [n][heads][d] of ``dtype`` (bf16 by default, or fp32)."""
    c = _cache(codes, scale, fmt)
    device = codes.device
    if slots is not None:
        n = slots.shape[0]
        _need(slots, "slots", (n,), _i32, device)
        if count is not None and n != count:
            raise ValueError(f"count {count} differs from the {n} slots")
    else:
        n = c.L - int(start) if count is None else int(count)
    shape = (n, c.d) if codes.dim() == 2 else (n, c.heads, c.d)
    if out is None:
        if n < 0:
            raise ValueError("start lies behind the cache")
        out = codes.new_empty(shape, dtype=dtype or _bf16)
    else:
        _need(out, "out", shape, dtype or out.dtype, device)
    dtype = out.dtype
    if dtype != _bf16 and dtype != _f32:
        raise TypeError(f"rows are read as bfloat16 or float32, got {dtype}")
    _launch(device, load_library().hytopk_cache_read, c, n, _address(slots), int(start),
            out.data_ptr(), 0 if dtype == _bf16 else 1)
    return out


# ------------------------------------------ layer norm and its checkpoints

_CHECKPOINTS = {"fp8": FP8_E4M3, "mxfp8": MXFP8_E4M3}


class NormSaved(NamedTuple):
    """What a layer norm keeps for its backward: its input (``fmt`` None, ``scale`` None) or the
    input's codes and scales in 8 bits (``fmt`` "fp8": uint8 of x's shape, fp32 a row; "mxfp8":
    one uint8 per 32 elements), and each row's mean and reciprocal deviation (``stats``, fp32 [..., 2])."""
    rows: torch.Tensor
    scale: torch.Tensor | None
    stats: torch.Tensor
    fmt: str | None


def _norm_shape(shape, name: str):
    """n, heads and d of rows [n][d] or [n][heads][d]."""
    if len(shape) == 2:
        return shape[0], 1, shape[1]
    if len(shape) == 3:
        return shape
    raise ValueError(f"{name} must be [n][d] or [n][heads][d], got {tuple(shape)}")


def _norm(weight, bias, d, eps, device) -> Norm:
    if weight is None and bias is None:
        return Norm(None, None, 1, eps)
    dtype = bias.dtype if weight is None else weight.dtype
    if dtype != _f32 and dtype != _bf16:
        raise TypeError(f"weight and bias must be bfloat16 or float32, got {dtype}")
    if weight is not None:
        _need(weight, "weight", (d,), dtype, device)
    if bias is not None:
        _need(bias, "bias", (d,), dtype, device)
    return Norm(_address(weight), _address(bias), 0 if dtype == _bf16 else 1, eps)


def _saved(s: NormSaved, shape, device):
    """The rows or the cache that a NormSaved stands for."""
    rows, scale, stats, fmt = s
    lead = shape[:-1]
    _need(stats, "stats", (*lead, 2), _f32, device)
    if fmt is None:
        if scale is not None:
            raise ValueError("rows that are kept as they are take no scale")
        if rows.shape != shape or rows.device != device:
            raise ValueError(f"saved rows must have the shape {tuple(shape)} and be on {device}")
        return _rows_array(rows, "saved rows"), None
    if fmt not in _CHECKPOINTS:
        raise ValueError(f"unknown checkpoint format {fmt!r}: fp8 or mxfp8")
    if scale is None:
        raise ValueError("fp8 and mxfp8 checkpoints need scale")
    _need(rows, "saved codes", shape, _u8, device)
    if fmt == "fp8":
        _need(scale, "scale", lead, _f32, device)
    else:
        _need(scale, "scale", (*lead, shape[-1] // 32), _u8, device)
    return None, _checkpoint(s, shape)


def _checkpoint(s: NormSaved, shape) -> Cache:
    return Cache(s.rows.data_ptr(), s.scale.data_ptr(), math.prod(shape[:-1]), 1, shape[-1], _CHECKPOINTS[s.fmt], 0)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, out=None, out_dtype=None, save=None):
    """Layer norm of rows x [n][d] or [n][heads][d] (bf16 or fp32, any strides but the last), each
    over its d elements: (x - mean) / sqrt(var + eps) * weight + bias, with weight and bias [d]
    (fp32 or bf16, one type; None: ones and zeros).  ``out`` may be x itself.  With ``save`` the result is
    (y, saved) and ``layer_norm_backward`` takes ``saved``: "x" keeps x itself (not a copy), "fp8" or "mxfp8"
    a checkpoint of it in 8 bits (d a multiple of 32), made in the same pass, and a NormSaved names the buffers to fill."""
    _gpu(x, "x")
    shape, device = x.shape, x.device
    n, heads, d = _norm_shape(shape, "x")
    xa = _rows_array(x, "x")
    if out is None and (out_dtype is None or out_dtype == x.dtype):
        out = _empty_like(x, memory_format=_contiguous)
        ya = RowsArray(out.data_ptr(), heads * d, d, xa.dtype, 0)
    else:
        if out is None:
            out = x.new_empty(shape, dtype=out_dtype)
        elif out.shape != shape or out.device != device or out_dtype not in (None, out.dtype):
            raise ValueError(f"out must have x's shape {tuple(shape)} and device, and out_dtype")
        ya = _rows_array(out, "out")
    p = _norm(weight, bias, d, eps, device)
    lib = load_library()
    if save is None:
        _launch(device, lib.hytopk_layer_norm, p, n, heads, d, xa, ya, None, None)
        return out
    cache = None
    if isinstance(save, NormSaved):
        rows, cache = _saved(save, shape, device)
        if cache is None and (rows.data != xa.data or save.rows.dtype != x.dtype or save.rows.stride() != x.stride()):
            raise ValueError("a NormSaved without a format keeps x itself")
    else:
        stats = x.new_empty((*shape[:-1], 2), dtype=_f32)
        if save == "x":
            save = NormSaved(x, None, stats, None)
        elif save in _CHECKPOINTS:
            if d % 32:
                raise ValueError("checkpoints in 8 bits need d in multiples of 32")
            scale = (x.new_empty(shape[:-1], dtype=_f32) if save == "fp8"
                     else x.new_empty((*shape[:-1], d // 32), dtype=_u8))
            save = NormSaved(_empty_like(x, dtype=_u8, memory_format=_contiguous), scale, stats, save)
            cache = _checkpoint(save, shape)
        else:
            raise ValueError(f"save must be 'x', 'fp8', 'mxfp8' or a NormSaved, got {save!r}")
    if cache is None and xa.data == ya.data and xa.data:
        raise ValueError("x is kept for the backward: out must not be x")
    _launch(device, lib.hytopk_layer_norm, p, n, heads, d, xa, ya, save.stats.data_ptr(), cache)
    return out, save


def layer_norm_backward_workspace_bytes(dy) -> int:
    """Workspace bytes of layer_norm_backward for dweight or dbias (0: none)."""
    return int(load_library().hytopk_layer_norm_backward_workspace(*_norm_shape(dy.shape, "dy")))


def layer_norm_backward(dy, saved: NormSaved, weight=None, *, want=("dx", "dweight", "dbias"), dx_dtype=None,
                        workspace=None, out=None):
    """Gradients of ``layer_norm`` from dy (the result's shape; bf16 or fp32, any strides but the last)
    and what it saved: a dict with dx (dy's shape, dy's type or ``dx_dtype``), dweight and dbias (fp32 [d], summed
    over all rows in a fixed order), those of ``want``.  ``weight`` is the forward's.  ``out`` gives tensors for some
    of them; dx may be dy or the saved rows themselves."""
    _gpu(dy, "dy")
    shape, device = dy.shape, dy.device
    n, heads, d = _norm_shape(shape, "dy")
    ga = _rows_array(dy, "dy")
    p = _norm(weight, None, d, 0.0, device)
    rows, cache = _saved(saved, shape, device)
    res = {} if out is None else dict(out)
    for name in want:
        if name not in res:
            if name == "dx":
                res[name] = (_empty_like(dy, memory_format=_contiguous) if dx_dtype is None
                             else dy.new_empty(shape, dtype=dx_dtype))
            else:
                res[name] = dy.new_empty(d, dtype=_f32)
    xa = dweight = dbias = None
    for name, t in res.items():
        if name == "dx":
            if t.shape != shape or t.device != device or dx_dtype not in (None, t.dtype):
                raise ValueError(f"dx must have dy's shape {tuple(shape)} and device, and dx_dtype")
            xa = _rows_array(t, "dx")
            continue
        _need(t, name, (d,), _f32, device)
        if name == "dweight":
            dweight = t.data_ptr()
        elif name == "dbias":
            dbias = t.data_ptr()
        else:
            raise ValueError(f"unknown gradient name {name!r}")
    lib = load_library()
    if workspace is not None:
        _workspace(workspace, device)
    elif dweight or dbias:
        need = lib.hytopk_layer_norm_backward_workspace(n, heads, d)
        if need:
            workspace = dy.new_empty(need, dtype=_u8)
    _launch(device, lib.hytopk_layer_norm_backward, p, n, heads, d, ga, rows, cache, saved.stats.data_ptr(), xa,
            dweight, dbias, _address(workspace), 0 if workspace is None else workspace.numel())
    return res


# ------------------------------------------- the indexer's target and loss

def _attention(q, k, idx, softmax_scale) -> Attention:
    """q [n][heads][d], k [L][key_heads][d] or [L][d], idx [n][k]."""
    shape, rows, device = q.shape, k.shape, q.device
    if len(shape) != 3 or len(rows) not in (2, 3) or rows[-1] != shape[-1]:
        raise ValueError("shapes must be q [n][heads][d], k [L][key_heads][d] or [L][d]")
    for t, name in ((q, "q"), (k, "k")):
        if t.dtype != _bf16 or not t.is_cuda or not t.is_contiguous() or t.device != device:
            raise ValueError(f"{name} must be contiguous bfloat16 on one GPU")
    n, heads, d = shape
    if idx.dim() != 2:
        raise ValueError("idx must be [n][k]")
    count = idx.shape[1]
    _need(idx, "idx", (n, count), _i32, device)
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    return Attention(rows[0], n, heads, rows[1] if len(rows) == 3 else 1, d, count, scale, 0)


def attention_mass_workspace_bytes(q, k, idx) -> int:
    """Workspace bytes of attention_mass without lse."""
    return int(load_library().hytopk_attention_mass_workspace(_attention(q, k, idx, None)))


def attention_mass(q, k, idx, *, softmax_scale=None, lse=None, workspace=None, out=None):
    """The attention's probability at the selected entries idx [n][k], averaged
    over heads (fp32 [n][k]; 0 at padding): the target of ``index_loss``.
    q [n][heads][d] and k [L][key_heads][d] (or [L][d]) are the attention's, bf16;
    ``softmax_scale`` is d ** -0.5 by default; ``lse`` (fp32 [n][heads]) is the attention's
    log-sum-exp, by default taken over the row's entries."""
    lib = load_library()
    p = _attention(q, k, idx, softmax_scale)
    device = q.device
    if lse is not None:
        _need(lse, "lse", (p.n, p.heads), _f32, device)
    if out is None:
        out = _empty_like(idx, dtype=_f32)
    else:
        _need(out, "out", (p.n, p.k), _f32, device)
    if workspace is None and lse is None:
        workspace = torch.empty(max(lib.hytopk_attention_mass_workspace(p), 1), dtype=_u8,
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
    _gpu(score, "score")
    if score.dim() != 2:
        raise ValueError("score must be [n][k]")
    shape, device = score.shape, score.device
    n, k = shape
    _need(score, "score", shape, _f32, device)
    _need(mass, "mass", shape, _f32, device)
    if weight is not None:
        _need(weight, "weight", (n,), _f32, device)
    if out is None:
        loss = grad = None
        if "loss" in want:
            loss = score.new_empty(n) if weight is None else _empty_like(weight)
        if "d_score" in want:
            grad = _empty_like(score)
    else:
        loss, grad = out
        if loss is not None:
            _need(loss, "out[0] (loss)", (n,), _f32, device)
        if grad is not None:
            _need(grad, "out[1] (d_score)", shape, _f32, device)
    _launch(device, load_library().hytopk_index_loss, n, k, score.data_ptr(), mass.data_ptr(),
            _address(weight), _address(loss), _address(grad))
    return loss, grad
