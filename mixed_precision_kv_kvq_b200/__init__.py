"""libkvq for Python: the B200 hot path of PM-KVQ's progressive
mixed-precision KV cache (quantize-on-append, Equivalent Right Shift shrink,
GQA decode attention over packed codes).

The functions named ``kvq_*`` mirror the C ABI of include/kvq.h one to one
(torch tensors in, raw pointers out).  ``KVQCache`` is the same API as an
object that owns its device pool and workspace as torch tensors.  PyTorch is
used for device memory and streams only; all arithmetic runs in libkvq.
"""
from __future__ import annotations

import ctypes as C
import struct
from typing import Optional, Sequence

import numpy as np
import torch

from ._lib import (KVQ_DTYPE_BF16, KVQ_DTYPE_F32, KVQ_POS_I32, KVQ_POS_I64, KVQ_ROPE_HALF, KVQ_ROPE_INTERLEAVED,  # noqa: F401
                   KVQ_ROPE_LINEAR, KVQ_ROPE_NONE, KVQ_ROPE_NTK, KVQ_ROPE_YARN, TREE_MAX_NODES, KVQ_OPT_KEY_CHANNEL, KVQ_OPT_SINK_WINDOW, KVQ_SHIFT_DIRECT,  # noqa: F401
                   KVQ_SHIFT_EQUIVALENT, KEY_BLOCK, WINDOW_TOKENS, KVQError, check, load)

HEAD_DIM = 128

__all__ = [
    "KVQCache", "KVQError", "Rope", "load",
    "kvq_pool_bytes", "kvq_pool_bytes_ex", "kvq_alloc", "kvq_alloc_ex", "kvq_export_window", "kvq_set_lambda", "kvq_append", "kvq_shrink", "kvq_set_shift_mode",
    "kvq_decode_workspace", "kvq_decode_attn", "kvq_decode_attn_noalloc", "kvq_append_decode", "kvq_dims", "kvq_query", "kvq_max_tokens", "kvq_export",
    "kvq_rope_freqs", "kvq_rope", "kvq_tree_workspace", "kvq_tree_attn", "kvq_read",
    "kvq_device_status", "kvq_selftest_timeout", "kvq_last_error", "kvq_free", "kvq_allocate_bits",
]


def _stream_ptr(stream) -> C.c_void_p:
    if stream is None:
        if torch.cuda.is_available() and torch.cuda.is_initialized():
            return C.c_void_p(torch.cuda.current_stream().cuda_stream)
        return C.c_void_p(None)
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def _fbit_array(fbit: Sequence[int]):
    arr = (C.c_int * len(fbit))(*[int(f) for f in fbit])
    return arr


def _dptr(t: torch.Tensor) -> C.c_void_p:
    return C.c_void_p(t.data_ptr())


class _Handle(C.c_void_p):
    """A cache's handle, with what kvq_dims says of it."""

    dims = None


def _check_cache(cache, k, v, names=("k", "v")) -> None:
    """That [batch][n][heads][128] tensors (or None) have the cache's batch and KV heads: the kernels go by the cache's."""
    _, batch, heads = getattr(cache, "dims", None) or kvq_dims(cache)
    for t in (k, v):
        if t is not None:
            s = t.shape
            if len(s) != 4 or s[0] != batch or s[2] != heads:
                raise ValueError(f"{names[t is not k]} must be [{batch}][n][{heads}][{HEAD_DIM}], got {list(s)}")


def _check_queries(cache, q: torch.Tensor, out: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> int:
    """The same of [batch][q_heads][128] queries, with an output like them and a workspace whose bytes neighbour.  -> q_heads"""
    batch = (getattr(cache, "dims", None) or kvq_dims(cache))[1]
    s = q.shape
    if len(s) != 3 or s[0] != batch:
        raise ValueError(f"q must be [{batch}][q_heads][{HEAD_DIM}], got {list(s)}")
    if q.dtype is not torch.bfloat16 or s[2] != HEAD_DIM or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 [batch][q_heads][128] tensor")
    if out.dtype is not torch.float32 or out.shape != s or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 tensor shaped like q")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return s[1]


def _check_tokens(cache, k: torch.Tensor, v: torch.Tensor, one: bool) -> int:
    """The same of contiguous Keys and Values alike, of one token a sequence if `one`.  -> tokens a sequence"""
    _, batch, heads = getattr(cache, "dims", None) or kvq_dims(cache)
    s = k.shape
    if len(s) != 4 or s[0] != batch or s[2] != heads:
        raise ValueError(f"k must be [{batch}][n][{heads}][{HEAD_DIM}], got {list(s)}")
    if v.shape != s or k.dtype is not v.dtype or s[3] != HEAD_DIM or (one and s[1] != 1):
        raise ValueError(f"k and v must both be [batch][{1 if one else 'n'}][kv_heads][128] of one dtype")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous")
    return s[1]


# ---------------------------------------------------------------- C ABI mirror

def kvq_pool_bytes(layers: int, batch: int, kv_heads: int, head_dim: int, budget_bytes: int,
                   fbit: Sequence[int]) -> int:
    return load().kvq_pool_bytes(layers, batch, kv_heads, head_dim, budget_bytes, _fbit_array(fbit))


def kvq_pool_bytes_ex(layers: int, batch: int, kv_heads: int, head_dim: int, budget_bytes: int,
                      fbit: Sequence[int], options: int) -> int:
    return load().kvq_pool_bytes_ex(layers, batch, kv_heads, head_dim, budget_bytes, _fbit_array(fbit), options)


def kvq_alloc(layers: int, batch: int, kv_heads: int, head_dim: int, budget_bytes: int,
              fbit: Sequence[int], dev_pool: Optional[torch.Tensor] = None) -> C.c_void_p:
    return kvq_alloc_ex(layers, batch, kv_heads, head_dim, budget_bytes, fbit, dev_pool, 0)


def kvq_alloc_ex(layers: int, batch: int, kv_heads: int, head_dim: int, budget_bytes: int,
                 fbit: Sequence[int], dev_pool: Optional[torch.Tensor] = None, options: int = 0) -> C.c_void_p:
    h = _Handle()
    pool_ptr = _dptr(dev_pool) if dev_pool is not None else C.c_void_p(None)
    pool_bytes = dev_pool.numel() * dev_pool.element_size() if dev_pool is not None else 0
    check(load().kvq_alloc_ex(C.byref(h), layers, batch, kv_heads, head_dim, budget_bytes,
                              _fbit_array(fbit), pool_ptr, pool_bytes, options))
    h.dims = kvq_dims(h)
    return h


def kvq_set_lambda(cache, layer: int, lam: np.ndarray) -> None:
    lam = np.ascontiguousarray(lam, dtype=np.float32)
    check(load().kvq_set_lambda(cache, layer, lam.ctypes.data_as(C.c_void_p)))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KVQ_DTYPE_BF16
    if t.dtype == torch.float32:
        return KVQ_DTYPE_F32
    raise TypeError(f"k/v must be bf16 or fp32, got {t.dtype}")


def kvq_append(cache, layer: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """k, v: device [batch][n][kv_heads][128], bf16 or fp32, contiguous."""
    n = _check_tokens(cache, k, v, False)
    if not (k.is_cuda and v.is_cuda):
        raise ValueError("k and v must be CUDA tensors")
    check(load().kvq_append(cache, layer, _dptr(k), _dptr(v), _dtype_code(k), n, _stream_ptr(stream)))


def kvq_shrink(cache, layer: int, stream=None) -> None:
    check(load().kvq_shrink(cache, layer, _stream_ptr(stream)))


def kvq_set_shift_mode(cache, layer: int, mode: int) -> None:
    """KVQ_SHIFT_EQUIVALENT (default) or KVQ_SHIFT_DIRECT, before the block's first shrink."""
    check(load().kvq_set_shift_mode(cache, layer, int(mode)))


def kvq_decode_workspace(cache, layer: int, q_heads: int) -> int:
    return load().kvq_decode_workspace(cache, layer, q_heads)


def kvq_decode_attn(cache, layer: int, q: torch.Tensor, sm_scale: float, out: torch.Tensor,
                    workspace: torch.Tensor, stream=None) -> None:
    """q: device bf16 [batch][q_heads][128]; out: device fp32, same shape."""
    heads = _check_queries(cache, q, out, workspace)
    if not (q.is_cuda and out.is_cuda and workspace.is_cuda):
        raise ValueError("q, out and workspace must be CUDA tensors")
    ws_bytes = workspace.numel() * workspace.element_size()
    check(load().kvq_decode_attn(cache, layer, _dptr(q), heads, float(sm_scale), _dptr(out),
                                 _dptr(workspace), ws_bytes, _stream_ptr(stream)))


def kvq_append_decode(cache, layer: int, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, sm_scale: float,
                      out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """One decode step in one launch: append k, v (device [batch][1][kv_heads][128])
    then attend with q (device bf16 [batch][q_heads][128]) into out (fp32)."""
    _check_tokens(cache, k, v, True)
    heads = _check_queries(cache, q, out, workspace)
    if not (k.is_cuda and v.is_cuda and q.is_cuda and out.is_cuda and workspace.is_cuda):
        raise ValueError("k, v, q, out and workspace must be CUDA tensors")
    ws_bytes = workspace.numel() * workspace.element_size()
    check(load().kvq_append_decode(cache, layer, _dptr(k), _dptr(v), _dtype_code(k), _dptr(q), heads,
                                   float(sm_scale), _dptr(out), _dptr(workspace), ws_bytes, _stream_ptr(stream)))


def kvq_decode_attn_noalloc(cache, layer: int, q: torch.Tensor, sm_scale: float, out: torch.Tensor,
                            stream=None) -> None:
    """Decode attention without a workspace: for callers that cannot allocate
    device memory where they run decode.  The library's own fixed 24 MiB
    scratch buffer (one per GPU, kept until exit) holds the split partials;
    calls that can overlap on the GPU share it and must be serialised."""
    heads = _check_queries(cache, q, out)
    if not (q.is_cuda and out.is_cuda):
        raise ValueError("q and out must be CUDA tensors")
    check(load().kvq_decode_attn_noalloc(cache, layer, _dptr(q), heads, float(sm_scale), _dptr(out),
                                         _stream_ptr(stream)))


_ROWS = struct.Struct("Pqqq").pack  # kvq_rows


def _rows(t: Optional[torch.Tensor]):
    """kvq_rows of a [batch][n][heads][128] tensor or view (None: NULL)."""
    if t is None:
        return None
    b, n, h, _ = t.stride()
    return _ROWS(t.data_ptr(), b, n, h)


def _take(name: str, t: torch.Tensor, dtype, device, shape=None):
    """kvq_rows of a [batch][n][heads][128] CUDA tensor of this type and device whose channels are neighbours; these
    calls last a few microseconds on the GPU, so what is checked is read once."""
    s, x = t.stride(), t.shape
    if t.dtype is dtype and t.device == device and len(x) == 4 and x[3] == HEAD_DIM and (s[3] == 1 or not t.numel()):
        if shape is not None and x != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x)}")
        if device.type == "cuda":
            return _ROWS(t.data_ptr(), s[0], s[1], s[2])
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must be a CUDA tensor [batch][n][heads][128] with neighbouring channels")


class _On:
    """Device guard, launch stream and allocator of one call on `device`: the
    given stream, or the device's current one."""

    __slots__ = ("device", "guard", "given", "ptr")

    def __init__(self, device, stream):
        self.device, self.given = device, stream
        self.guard = torch.cuda.device(device) if torch._C._cuda_getDevice() != device.index else None
        if stream is None:
            self.ptr = torch._C._cuda_getCurrentRawStream(device.index)
        elif isinstance(stream, torch.cuda.Stream):
            self.ptr = stream.cuda_stream
        else:
            self.ptr = int(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def _stream(self):
        """The given stream; of a raw handle, what the call allocates belongs to it and not to the current stream."""
        if isinstance(self.given, torch.cuda.Stream):
            return self.given
        return torch.cuda.ExternalStream(self.ptr, self.device) if self.ptr else torch.cuda.default_stream(self.device)

    def empty(self, shape, dtype) -> torch.Tensor:
        """A new tensor that belongs to the call's stream."""
        if self.given is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self._stream()):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def like(self, t: torch.Tensor) -> torch.Tensor:
        """The same, contiguous and shaped like t."""
        if self.given is None:
            return torch.empty_like(t, memory_format=torch.contiguous_format)
        with torch.cuda.stream(self._stream()):
            return torch.empty_like(t, memory_format=torch.contiguous_format)


_SCALINGS = {"none": KVQ_ROPE_NONE, "linear": KVQ_ROPE_LINEAR, "ntk": KVQ_ROPE_NTK, "yarn": KVQ_ROPE_YARN}
_LAYOUTS = {"half": KVQ_ROPE_HALF, "interleaved": KVQ_ROPE_INTERLEAVED}


def kvq_rope_freqs(rot_dim: int, theta: float = 10000.0, scaling: int = KVQ_ROPE_NONE, factor: float = 1.0,
                   original_tokens: int = 0):
    """-> (inv_freq [rot_dim / 2] float64 numpy, magnitude)."""
    for name, x in (("rot_dim", rot_dim), ("scaling", scaling), ("original_tokens", original_tokens)):
        if not -2 ** 31 <= x < 2 ** 31:  # a C int would keep its low 32 bits
            raise KVQError(1, f"{name} {x} is out of range")
    inv = np.zeros(min(max(rot_dim, 2), HEAD_DIM) // 2, np.float64)
    mag = C.c_float()
    check(load().kvq_rope_freqs(int(rot_dim), float(theta), int(scaling), float(factor), int(original_tokens), inv.ctypes.data_as(C.c_void_p), C.byref(mag)))
    return inv, mag.value


class Rope:
    """A rotary schedule: which channels form pairs and how fast each turns.

    scaling: "none", "linear" (positional interpolation), "ntk" or "yarn" with
    `factor` (and `original_tokens` for "yarn"); or inv_freq (and magnitude)
    of any other schedule."""

    def __init__(self, rot_dim: int = HEAD_DIM, theta: float = 10000.0, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original_tokens: int = 0, inv_freq=None, magnitude: float = 1.0):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
        self.rot_dim, self.layout = int(rot_dim), layout
        if inv_freq is None:
            inv_freq, magnitude = kvq_rope_freqs(self.rot_dim, theta, _SCALINGS[scaling], factor, original_tokens)
        inv_freq = np.array(inv_freq, dtype=np.float64)  # a copy: the schedule does not change under its user
        if inv_freq.shape != (self.rot_dim // 2,):
            raise ValueError(f"inv_freq must hold rot_dim / 2 = {self.rot_dim // 2} values")
        self.__setstate__({"rot_dim": self.rot_dim, "layout": layout, "inv_freq": inv_freq, "magnitude": float(magnitude)})

    def __getstate__(self):
        return {"rot_dim": self.rot_dim, "layout": self.layout, "inv_freq": self.inv_freq, "magnitude": self.magnitude}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self.inv_freq.flags.writeable = False
        self._code = _LAYOUTS[self.layout]
        self._ptr = self.inv_freq.ctypes.data_as(C.c_void_p)


def kvq_rope(rope: Rope, positions: torch.Tensor, q: Optional[torch.Tensor], k: Optional[torch.Tensor] = None,
             q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions of q and k (either may be None), in one launch.

    q, k: device [batch][n][heads][128], bf16 or fp32, any strides with
    neighbouring channels (slices of a fused projection are read in place).
    positions: device int32 or int64, [batch][n], or [n] for every sequence.
    q_out, k_out: outputs shaped like q and k (an input itself: in place);
    allocated contiguous by default.  -> (q_out, k_out), which carry no
    gradient (as everything here: the path is inference)."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q and k are both None")
    dtype, dt, device = _dtype_code(first), first.dtype, first.device
    qr = _take("q", q, dt, device) if q is not None else None
    kr = _take("k", k, dt, device) if k is not None else None
    batch, n = first.shape[:2]
    if q is not None and k is not None and k.shape[:2] != (batch, n):
        raise ValueError(f"q and k must agree in batch and tokens, got {list(q.shape)} and {list(k.shape)}")
    if (q_out is not None and q is None) or (k_out is not None and k is None):
        raise ValueError("an output without its input")
    pt, shape = positions.dtype, positions.shape
    if (pt is not torch.int64 and pt is not torch.int32) or positions.device != device:
        raise ValueError("positions must be an int32 or int64 tensor on the device of q and k")
    if shape == (batch, n):
        ps_b, ps_t = positions.stride()
    elif shape == (n,):
        ps_b, ps_t = 0, positions.stride(0)
    else:
        raise ValueError(f"positions must be [{batch}][{n}] or [{n}], got {list(shape)}")
    qo = ko = None
    with _On(device, stream) as on:
        if q is not None:
            if q_out is None:
                q_out = on.like(q)
                qo = _rows(q_out)
            else:
                qo = _take("q_out", q_out, dt, device, q.shape)
        if k is not None:
            if k_out is None:
                k_out = on.like(k)
                ko = _rows(k_out)
            else:
                ko = _take("k_out", k_out, dt, device, k.shape)
        check(load().kvq_rope(rope.rot_dim, rope._code, rope._ptr, rope.magnitude, positions.data_ptr(),
                              KVQ_POS_I64 if pt is torch.int64 else KVQ_POS_I32, ps_b, ps_t, batch, n, dtype,
                              qr, qo, q.shape[2] if q is not None else 0, kr, ko, k.shape[2] if k is not None else 0, on.ptr))
    return q_out, k_out


def kvq_tree_workspace(cache, layer: int, q_heads: int, n_nodes: int) -> int:
    return load().kvq_tree_workspace(cache, layer, q_heads, n_nodes)


def kvq_tree_attn(cache, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: Optional[torch.Tensor],
                  sm_scale: float, out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """q: device bf16 [batch][n][q_heads][128]; k, v: device [batch][n][kv_heads][128], bf16 or fp32 (strided views
    allowed); mask: device bool or uint8 [batch][n][n] or [n][n] (contiguous), None: a chain; out: contiguous bf16,
    shaped like q."""
    _check_cache(cache, k, v)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    with _On(q.device, stream) as on:
        _tree_attn(cache, layer, q, k, v, mask, sm_scale, out, workspace, on.ptr)


def _tree_attn(cache, layer, q, k, v, mask, sm_scale, out, workspace, ptr) -> None:
    """kvq_tree_attn with k and v of the cache's shape and q's device current, on the stream handle ptr."""
    dtype, dt, device = _dtype_code(k), k.dtype, q.device
    qr, kr = _take("q", q, torch.bfloat16, device), _take("k", k, dt, device)
    vr = _take("v", v, dt, device, k.shape)
    _take("out", out, torch.bfloat16, device, q.shape)
    b, n, q_heads, _ = q.shape
    if k.shape[:2] != (b, n):
        raise ValueError(f"k must be [{b}][{n}][kv_heads][128], got {list(k.shape)}")
    if not out.is_contiguous() or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("out and workspace must be contiguous and on one device")
    mask_ptr, mask_b = None, 0
    if mask is not None:
        mt, ms = mask.dtype, mask.shape
        if (mt is not torch.bool and mt is not torch.uint8) or mask.device != device or not mask.is_contiguous():
            raise ValueError("mask must be a contiguous bool or uint8 tensor on the device of q")
        if ms == (b, n, n):
            mask_b = n * n
        elif ms != (n, n):
            raise ValueError(f"mask must be [{b}][{n}][{n}] or [{n}][{n}], got {list(ms)}")
        mask_ptr = mask.data_ptr()
    check(load().kvq_tree_attn(cache, layer, qr, q_heads, n, kr, vr, dtype, mask_ptr, mask_b, float(sm_scale),
                               out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), ptr))


def kvq_read(cache, layer: int, start: int, count: int, k_out: Optional[torch.Tensor], v_out: Optional[torch.Tensor],
             stream=None) -> None:
    """k_out, v_out: device [batch][count][kv_heads][128], both bf16 or both fp32, any strides with neighbouring
    channels; either may be None."""
    first = k_out if k_out is not None else v_out
    if first is None:
        raise ValueError("k_out and v_out are both None")
    _check_cache(cache, k_out, v_out, ("k_out", "v_out"))
    if not first.is_cuda:
        raise ValueError("k_out and v_out must be CUDA tensors")
    with _On(first.device, stream) as on:
        _read(cache, layer, start, count, k_out, v_out, on.ptr)


def _read(cache, layer, start, count, k_out, v_out, ptr) -> None:
    """kvq_read with outputs of the cache's shape and their device current, on the stream handle ptr."""
    first = k_out if k_out is not None else v_out
    start, count = int(start), int(count)
    dtype, dt, device = _dtype_code(first), first.dtype, first.device
    kr = _take("k_out", k_out, dt, device) if k_out is not None else None
    vr = _take("v_out", v_out, dt, device, first.shape) if v_out is not None else None
    if not -2 ** 31 <= start < 2 ** 31:  # a C int would keep its low 32 bits
        raise KVQError(1, f"tokens [{start}, {start} + {count}) are not within what layer {layer} holds")
    if first.shape[1] != count:
        raise ValueError(f"the outputs must hold {count} tokens, got {first.shape[1]}")
    check(load().kvq_read(cache, layer, start, count, dtype, kr, vr, ptr))


def kvq_dims(cache) -> tuple:
    """-> (layers, batch, kv_heads) of a cache."""
    n, b, h = C.c_int(), C.c_int(), C.c_int()
    check(load().kvq_dims(cache, C.byref(n), C.byref(b), C.byref(h)))
    return n.value, b.value, h.value


def kvq_query(cache, layer: int) -> dict:
    t, b, cap, ns = C.c_int(), C.c_int(), C.c_int(), C.c_int()
    check(load().kvq_query(cache, layer, C.byref(t), C.byref(b), C.byref(cap), C.byref(ns)))
    return {"tokens": t.value, "bits": b.value, "capacity": cap.value, "n_shrinks": ns.value}


def kvq_max_tokens(cache) -> int:
    return load().kvq_max_tokens(cache)


def kvq_export(cache, layer: int, b: int, j: int, stream=None, sink_window: bool = False,
               key_channel: bool = False):
    """-> (k_codes [T][128], v_codes [T][128], k_meta [T][2], v_meta [T][2]) uint16 numpy.
    With the sink + window option (sink_window=True) T counts the
    progressive cache only: tokens 1 .. n - 129.  With per-channel Key
    groups (key_channel=True) T counts the progressive cache (whole blocks of
    128) and k_meta row 128 k + c is Key channel c of block k."""
    T = kvq_query(cache, layer)["tokens"]
    if sink_window:
        T = max(0, T - WINDOW_TOKENS - 1)
    if key_channel:
        T = T // KEY_BLOCK * KEY_BLOCK
    kc = np.zeros((T, HEAD_DIM), np.uint16)
    vc = np.zeros((T, HEAD_DIM), np.uint16)
    km = np.zeros((T, 2), np.uint16)
    vm = np.zeros((T, 2), np.uint16)
    p = lambda a: a.ctypes.data_as(C.c_void_p)  # noqa: E731
    check(load().kvq_export(cache, layer, b, j, p(kc), p(vc), p(km), p(vm), _stream_ptr(stream)))
    return kc, vc, km, vm


def kvq_export_window(cache, layer: int, b: int, j: int, stream=None):
    """-> (k_codes [n][128], v_codes, k_meta [n][2], v_meta) uint16 numpy: the
    sink and window tokens (or, with per-channel Key groups, the staged
    tokens) at 16 bits, oldest first."""
    n1 = WINDOW_TOKENS + 1
    kc = np.zeros((n1, HEAD_DIM), np.uint16)
    vc = np.zeros((n1, HEAD_DIM), np.uint16)
    km = np.zeros((n1, 2), np.uint16)
    vm = np.zeros((n1, 2), np.uint16)
    n = C.c_int()
    p = lambda a: a.ctypes.data_as(C.c_void_p)  # noqa: E731
    check(load().kvq_export_window(cache, layer, b, j, p(kc), p(vc), p(km), p(vm), C.byref(n), _stream_ptr(stream)))
    return kc[:n.value], vc[:n.value], km[:n.value], vm[:n.value]


def kvq_device_status(cache, stream=None) -> None:
    check(load().kvq_device_status(cache, _stream_ptr(stream)))


def kvq_selftest_timeout(cache, stream=None) -> None:
    check(load().kvq_selftest_timeout(cache, _stream_ptr(stream)))


def kvq_allocate_bits(sens, bits: Sequence[int], batch: int, kv_heads: int, max_tokens: int,
                      budget_bytes: int, head_dim: int = HEAD_DIM):
    """sens: [layers][n_opts] sensitivities (host).  -> (fbit list, objective)."""
    sens = np.ascontiguousarray(sens, dtype=np.float64)
    if sens.ndim != 2 or sens.shape[1] != len(bits):
        raise ValueError("sens must be [layers][len(bits)]")
    layers = sens.shape[0]
    b = (C.c_int * len(bits))(*[int(x) for x in bits])
    out = (C.c_int * layers)()
    obj = C.c_double()
    check(load().kvq_allocate_bits(layers, len(bits), b, sens.ctypes.data_as(C.c_void_p), batch, kv_heads,
                                   head_dim, max_tokens, budget_bytes, out, C.byref(obj)))
    return list(out), obj.value


def kvq_last_error() -> str:
    m = load().kvq_last_error()
    return m.decode() if m else ""


def kvq_free(cache) -> None:
    load().kvq_free(cache)


# ---------------------------------------------------------------- object API

class KVQCache:
    """A progressive mixed-precision KV cache for `layers` transformer blocks.

    The device pool is a torch uint8 tensor sized by kvq_pool_bytes; the
    decode workspace is a torch tensor sized by kvq_decode_workspace.
    Host (CPU) inputs of append, decode_attn and append_decode are copied to
    the device on the current stream before the call (pinned memory makes the
    copy asynchronous); tree_attn and read take device tensors."""

    def __init__(self, layers: int, batch: int, kv_heads: int, budget_bytes: int,
                 fbit: Sequence[int], head_dim: int = HEAD_DIM, device=None, sink_window: bool = False,
                 key_channel: bool = False):
        self.layers, self.batch, self.kv_heads = layers, batch, kv_heads
        self.fbit = list(fbit)
        self.device = torch.device(device if device is not None else "cuda")
        self.sink_window = sink_window
        self.key_channel = key_channel
        options = (KVQ_OPT_SINK_WINDOW if sink_window else 0) | (KVQ_OPT_KEY_CHANNEL if key_channel else 0)
        nbytes = kvq_pool_bytes_ex(layers, batch, kv_heads, head_dim, budget_bytes, fbit, options)
        if nbytes == 0:
            raise KVQError(1, "invalid cache parameters or budget too small")
        self.pool = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.handle = kvq_alloc_ex(layers, batch, kv_heads, head_dim, budget_bytes, fbit, self.pool, options)
        self._ws = {}
        self._tree_ws = {}
        self._stage = {}

    # -- helpers
    def _dev(self, t: torch.Tensor) -> torch.Tensor:
        if t.is_cuda:
            return t if t.is_contiguous() else t.contiguous()
        return t.to(self.device, non_blocking=True)

    def workspace(self, layer: int, q_heads: int) -> torch.Tensor:
        n = kvq_decode_workspace(self.handle, layer, q_heads)
        if n == 0:
            raise KVQError(1, f"no workspace size for layer {layer}, q_heads {q_heads}")
        ws = self._ws.get(n)
        if ws is None:
            ws = torch.empty((n + 3) // 4, dtype=torch.float32, device=self.device)
            self._ws[n] = ws
        return ws

    # -- the hot path
    def set_lambda(self, layer: int, lam) -> None:
        if isinstance(lam, torch.Tensor):
            lam = lam.detach().float().cpu().numpy()
        kvq_set_lambda(self.handle, layer, lam)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        kvq_append(self.handle, layer, self._dev(k), self._dev(v), stream)

    def shrink(self, layer: int, stream=None) -> None:
        kvq_shrink(self.handle, layer, stream)

    def set_shift_mode(self, layer: int, mode: int) -> None:
        kvq_set_shift_mode(self.handle, layer, mode)

    def decode_attn(self, layer: int, q: torch.Tensor, sm_scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        q = self._dev(q)
        if sm_scale is None:
            sm_scale = HEAD_DIM ** -0.5
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=self.device)
        kvq_decode_attn(self.handle, layer, q, sm_scale, out, self.workspace(layer, q.shape[1]), stream)
        return out

    def append_decode(self, layer: int, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor,
                      sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """append(layer, k, v) of one token per sequence, then decode_attn(layer, q), in one launch."""
        k, v, q = self._dev(k), self._dev(v), self._dev(q)
        if sm_scale is None:
            sm_scale = HEAD_DIM ** -0.5
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=self.device)
        kvq_append_decode(self.handle, layer, k, v, q, sm_scale, out, self.workspace(layer, q.shape[1]), stream)
        return out

    def tree_attn(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: Optional[torch.Tensor] = None,
                  sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of n drafted tokens per sequence over the block's cache and over one another.

        q: bf16 [batch][n][q_heads][128]; k, v: the drafted tokens' Keys and Values [batch][n][kv_heads][128], bf16 or
        fp32; mask: bool or uint8 [batch][n][n] or [n][n], mask[i][j]: node i sees node j (None: a chain, j <= i).
        -> bf16, shaped like q.  The drafted tokens do not enter the cache."""
        device = self.pool.device
        if q.dim() != 4 or q.shape[0] != self.batch or q.device != device:
            raise ValueError(f"q must be [{self.batch}][n][q_heads][128] on {device}, got {list(q.shape)} on {q.device}")
        _check_cache(self.handle, k, v)
        with _On(device, stream) as on:
            # the workspace belongs to this call alone: calls on other streams and captured graphs have their own
            size = (q.shape[2], q.shape[1])
            nbytes = self._tree_ws.get(size)
            if nbytes is None:
                nbytes = kvq_tree_workspace(self.handle, layer, *size)
                if nbytes:
                    self._tree_ws[size] = nbytes
            if out is None:
                out = on.like(q)
            _tree_attn(self.handle, layer, q, k, v, mask, HEAD_DIM ** -0.5 if sm_scale is None else sm_scale, out,
                       on.empty((nbytes,), torch.uint8), on.ptr)
        return out

    def read(self, layer: int, start: int = 0, count: Optional[int] = None, dtype: torch.dtype = torch.bfloat16,
             k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None, stream=None):
        """Tokens start .. start + count - 1 as values in the order they were appended -> (k, v), each
        [batch][count][kv_heads][128]: what append was given, up to the quantization.  With k_out or v_out only the
        given ones are written (and returned)."""
        if count is None:
            count = self.query(layer)["tokens"] - start
        if count < 0:
            raise ValueError(f"count {count} < 0")
        device = self.pool.device
        with _On(device, stream) as on:
            if k_out is None and v_out is None:
                shape = (self.batch, count, self.kv_heads, HEAD_DIM)
                k_out = on.empty(shape, dtype)
                v_out = on.like(k_out)
            else:
                _check_cache(self.handle, k_out, v_out, ("k_out", "v_out"))
                for name, x in (("k_out", k_out), ("v_out", v_out)):
                    if x is not None and x.device != device:
                        raise ValueError(f"{name} must be on the cache's device {device}, got {x.device}")
            _read(self.handle, layer, start, count, k_out, v_out, on.ptr)
        return k_out, v_out

    def query(self, layer: int) -> dict:
        return kvq_query(self.handle, layer)

    @property
    def max_tokens(self) -> int:
        return kvq_max_tokens(self.handle)

    def export(self, layer: int, b: int, j: int, stream=None):
        return kvq_export(self.handle, layer, b, j, stream, self.sink_window, self.key_channel)

    def export_window(self, layer: int, b: int, j: int, stream=None):
        return kvq_export_window(self.handle, layer, b, j, stream)

    def device_status(self, stream=None) -> None:
        kvq_device_status(self.handle, stream)

    def free(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            kvq_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
