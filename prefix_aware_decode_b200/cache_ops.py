"""Operators on the paged cache of device-resident sessions (pa.h, "session
caches on the device"): append with rotary positions, attention with a sliding
window and sinks, accumulated attention weights, and eviction.

Every call takes the sessions' block table [S][max_pages], cached lengths [S]
and row offsets [S + 1] as int32 CUDA tensors and reads them when its kernels
run: nothing is planned on the host or copied back, so a call can be captured
into a CUDA graph and replayed as the lengths and tables change in place.

All tensors of a call live on one device, which need not be the current one.
A call runs on `stream` (a torch stream of that device), or on the device's
current stream; outputs and workspaces that it allocates belong to that stream.
Argument errors raise ValueError, errors of the library PaError.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from ._binding import PaRope, PaSessions, _check, lib

_ref = ctypes.byref
_I32, _F32, _F64, _BF16 = torch.int32, torch.float32, torch.float64, torch.bfloat16
_Tensor, _empty_strided = torch.Tensor, torch.empty_strided


def _ptr(t, name: str, dtype, index: int, align: int = 16) -> int:
    """Address of a contiguous tensor of one type on CUDA device `index`."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.is_contiguous() and t.get_device() == index:
        p = t.data_ptr()
        if p % align == 0:
            return p
        raise ValueError(f"{name} must be {align}-byte aligned")
    if not isinstance(t, _Tensor) or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the pools' device")
    raise ValueError(f"{name} must be contiguous")


def _rows_ptr(t, name: str, heads: int, rows: int, D: int, index: int) -> Tuple[int, int]:
    """Address and row stride of [rows][heads][D] rows, which may be slices of wider ones."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.shape != (rows, heads, D):
        raise ValueError(f"{name} must be a bf16 tensor [{rows}][{heads}][{D}]")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the pools' device")
    s = t.stride()
    if (D > 1 and s[2] != 1) or (heads > 1 and s[1] != D):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    stride = s[0] if rows > 1 else heads * D
    p = t.data_ptr()
    if stride < heads * D or stride % 8 or p % 16:
        raise ValueError(f"{name}: rows must not overlap and must be 16-byte aligned")
    return p, stride


class _On:
    """Makes a device, or a stream of it, current for a call's launches and allocations."""

    def __init__(self, index: int, stream):
        device = torch.device("cuda", index)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream is not None and stream.device != device:
            raise ValueError(f"stream must be a stream of {device}")
        self.ctx = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


class _Here:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_HERE = _Here()


def _on(index: int, stream):
    if stream is None and index == torch.cuda.current_device():
        return _HERE
    return _On(index, stream)


def _current(index: int) -> int:
    """The device's current stream (cudaStream_t); the private call costs a thirtieth of the public one."""
    return _raw_stream(index)


try:
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:  # not in this torch
    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _index(k_pool) -> int:
    """The device of a call: k_pool's."""
    if not isinstance(k_pool, _Tensor) or k_pool.dim() != 4:
        raise ValueError("k_pool must be a tensor [num_pages][Hkv][P][D]")
    if not k_pool.is_cuda:
        raise ValueError("k_pool must be a CUDA tensor")
    return k_pool.get_device()


def _sessions(k_pool, block_table, kv_lens, cu_rows, num_rows: int, num_q_heads: Optional[int], index: int) -> PaSessions:
    num_pages, Hkv, P, D = k_pool.shape
    bt = _ptr(block_table, "block_table", _I32, index, 4)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [S][max_pages]")
    S, max_pages = block_table.shape
    kv = _ptr(kv_lens, "kv_lens", _I32, index, 4)
    if kv_lens.shape != (S,):
        raise ValueError("kv_lens must be [S], S the rows of block_table")
    if num_q_heads is None:
        return PaSessions(S, 0, Hkv, Hkv, D, P, max_pages, num_pages, bt, kv, None)
    cu = _ptr(cu_rows, "cu_rows", _I32, index, 4)
    if cu_rows.shape != (S + 1,):
        raise ValueError("cu_rows must be [S + 1], S the rows of block_table")
    return PaSessions(S, num_rows, num_q_heads, Hkv, D, P, max_pages, num_pages, bt, kv, cu)


def _v_ptr(v_pool, k_pool, index: int) -> int:
    p = _ptr(v_pool, "v_pool", _BF16, index)
    if v_pool.shape != k_pool.shape:
        raise ValueError("v_pool must have k_pool's shape")
    return p


def _q_ptr(q, k_pool, index: int) -> int:
    p = _ptr(q, "q", _BF16, index)
    if q.dim() != 3 or q.shape[2] != k_pool.shape[3]:
        raise ValueError("q must be [rows][Hq][D], D that of the pools")
    return p


def _out(t, name: str, shape, dtype, index: int, align: int = 16):
    """(tensor, address) of an output: the caller's, checked, or a new one."""
    if t is None:
        t = _new(shape, dtype, index)
        return t, t.data_ptr()
    p = _ptr(t, name, dtype, index, align)
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    return t, p


def _new(shape, dtype, index: int):
    """A new contiguous tensor of at most three dimensions (empty_strided costs two thirds of empty)."""
    n = len(shape)
    strides = (1,) if n == 1 else (shape[1], 1) if n == 2 else (shape[1] * shape[2], shape[2], 1)
    return _empty_strided(shape, strides, dtype=dtype, device=_device(index))


_devices = {}


def _device(index: int):
    d = _devices.get(index)
    if d is None:
        d = _devices[index] = torch.device("cuda", index)
    return d


def rope_append(q, k, v, positions, inv_freq, k_pool, v_pool, block_table, kv_lens, cu_rows, *,
                axes: Optional[Sequence[int]] = None, interleaved: bool = False, q_out=None, stream=None):
    """Rotates the rows' q and k and writes k and v into their cache slots
    (pa_rope_append).  Returns q_out bf16 [rows][Hq][D].

    q bf16 [rows][Hq][D], k, v bf16 [rows][Hkv][D]: heads contiguous, rows at any
    stride (slices of one projection).  positions int32 [rows] or [n_axes][rows];
    inv_freq fp64 [R/2] (radians per position; R the rotated dims); axes: the axis
    of each of the R/2 pairs (default: all 0).  kv_lens counts the rows: the i-th
    of a session's n rows goes to cached token kv_len - n + i.
    """
    index = _index(k_pool)
    if not isinstance(q, _Tensor) or q.dim() != 3:
        raise ValueError("q must be [rows][Hq][D]")
    rows, Hq, _ = q.shape
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, rows, Hq, index)
    D, Hkv = b.head_dim, b.num_kv_heads
    qp, qs = _rows_ptr(q, "q", Hq, rows, D, index)
    kp, ks = _rows_ptr(k, "k", Hkv, rows, D, index)
    vp, vs = _rows_ptr(v, "v", Hkv, rows, D, index)
    pos = _ptr(positions, "positions", _I32, index, 4)
    ps = positions.shape
    if len(ps) not in (1, 2) or ps[-1] != rows:
        raise ValueError("positions must be [rows] or [n_axes][rows]")
    inv = _ptr(inv_freq, "inv_freq", _F64, index, 8)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [R / 2]")
    pairs = inv_freq.shape[0]
    if axes is not None:
        axes = bytes(axes)
        if len(axes) != pairs:
            raise ValueError("axes must name the axis of each of inv_freq's pairs")
    kpool, vpool = _ptr(k_pool, "k_pool", _BF16, index), _v_ptr(v_pool, k_pool, index)
    rope = PaRope(2 * pairs, 1 if len(ps) == 1 else ps[0], 1 if interleaved else 0, axes, pos, inv)
    with _on(index, stream):
        q_out, op = _out(q_out, "q_out", (rows, Hq, D), _BF16, index)
        _check(lib().pa_rope_append(_ref(b), _ref(rope), qp, qs, kp, ks, vp, vs, kpool, vpool, op, _current(index)),
               "pa_rope_append")
    return q_out


def window_workspace(q, k_pool, block_table, kv_lens, cu_rows, *, window: int = 0, sinks: int = 0):
    """A workspace for window_attend calls of these shapes (pa_window_workspace_size):
    one serves any number of calls in stream order, calls that may overlap on the
    GPU need one each."""
    index = _index(k_pool)
    _q_ptr(q, k_pool, index)
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, q.shape[0], q.shape[1], index)
    return _new((_workspace_bytes(b, window, sinks, index),), torch.uint8, index)


_sizes = {}


def _workspace_bytes(b: PaSessions, window: int, sinks: int, index: int) -> int:
    """pa_window_workspace_size, which depends on the sizes of a call only."""
    key = (b.n_sessions, b.num_rows, b.num_q_heads, b.num_kv_heads, b.head_dim, b.page_size, b.max_pages,
           b.num_pages_in_pool, window, sinks, index)
    size = _sizes.get(key)
    if size is None:
        n = ctypes.c_size_t()
        with _on(index, None):
            _check(lib().pa_window_workspace_size(_ref(b), window, sinks, _ref(n)), "pa_window_workspace_size")
        if len(_sizes) >= 1024:
            _sizes.clear()
        size = _sizes[key] = n.value
    return size


def window_status(workspace, stream=None) -> int:
    """The device status word of the last window_attend on this workspace
    (pa_window_status; PA_OK unless a bounded wait gave up).  Synchronises the stream."""
    out = ctypes.c_int()
    index = workspace.get_device()
    wp = _ptr(workspace, "workspace", torch.uint8, index, 256)
    with _on(index, stream):
        _check(lib().pa_window_status(wp, _current(index), _ref(out)), "pa_window_status")
    return out.value


def window_attend(q, k_pool, v_pool, block_table, kv_lens, cu_rows, *, window: int = 0, sinks: int = 0,
                  softmax_scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of the last rows of every session over its cache, with a
    sliding window and sinks (pa_window_attend): the row at position p sees token
    t when t <= p and (window == 0 or t > p - window or t < sinks).

    q bf16 [rows][Hq][D]; pools bf16 [num_pages][Hkv][P][D].  Returns (out bf16
    [rows][Hq][D], lse fp32 [rows][Hq]); rows that see nothing get 0 and -inf.
    `workspace` (window_workspace) is allocated by the call when not given.
    """
    index = _index(k_pool)
    qp = _q_ptr(q, k_pool, index)
    rows, Hq, D = q.shape
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, rows, Hq, index)
    kp, vp = _ptr(k_pool, "k_pool", _BF16, index), _v_ptr(v_pool, k_pool, index)
    with _on(index, stream):
        out, op = _out(out, "out", (rows, Hq, D), _BF16, index)
        lse, lp = _out(lse, "lse", (rows, Hq), _F32, index, 4)
        if workspace is None:
            workspace = _new((_workspace_bytes(b, window, sinks, index),), torch.uint8, index)
        wp = _ptr(workspace, "workspace", torch.uint8, index, 256)
        _check(lib().pa_window_attend(_ref(b), window, sinks, softmax_scale, qp, kp, vp, wp, workspace.numel(), op, lp,
                                      _current(index)), "pa_window_attend")
    return out, lse


def weigh_tokens(q, k_pool, lse, block_table, kv_lens, cu_rows, scores, *, window: int = 0, sinks: int = 0,
                 softmax_scale: float = 0.0, stream=None):
    """Adds to scores fp32 [S][Hkv][max_tokens], in place, the attention weight that
    each cached token draws from the batch's rows (pa_weigh_tokens): lse is
    window_attend's for the same q, window, sinks and scale.  Returns scores."""
    index = _index(k_pool)
    qp, kp = _q_ptr(q, k_pool, index), _ptr(k_pool, "k_pool", _BF16, index)
    rows, Hq, _ = q.shape
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, rows, Hq, index)
    lp = _ptr(lse, "lse", _F32, index, 4)
    if lse.shape != (rows, Hq):
        raise ValueError("lse must be [rows][Hq]")
    sp = _ptr(scores, "scores", _F32, index, 4)
    ss = scores.shape
    if len(ss) != 3 or ss[0] != b.n_sessions or ss[1] != b.num_kv_heads:
        raise ValueError("scores must be [S][Hkv][max_tokens]")
    with _on(index, stream):
        _check(lib().pa_weigh_tokens(_ref(b), window, sinks, softmax_scale, qp, kp, lp, sp, ss[2], _current(index)),
               "pa_weigh_tokens")
    return scores


def weigh_status(device=None, stream=None) -> int:
    """The first failure of a bounded wait of weigh_tokens on the device since this
    call last returned one (pa_weigh_status; PA_OK: none).  Synchronises the stream."""
    out = ctypes.c_int()
    index = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    with _on(index, stream):
        _check(lib().pa_weigh_status(_current(index), _ref(out)), "pa_weigh_status")
    return out.value


def evict_tokens(scores, k_pool, v_pool, block_table, kv_lens, dst_table, budget: int, *, sinks: int = 0,
                 recent: int = 0, scores_out=None, stream=None):
    """Keeps, per (session, kv head), the first `sinks`, the last `recent` and the
    highest-scoring other tokens, `budget` in all, and copies their K and V in
    order to the pages of dst_table int32 [S][n] (pa_evict_tokens; pages that no
    row of block_table names).  Returns (new_lens int32 [S], kept int32
    [S][Hkv][budget] former indices then -1, scores_out fp32 [S][Hkv][max_tokens])."""
    index = _index(k_pool)
    b = _sessions(k_pool, block_table, kv_lens, None, 0, None, index)
    S, Hkv = b.n_sessions, b.num_kv_heads
    kp, vp = _ptr(k_pool, "k_pool", _BF16, index), _v_ptr(v_pool, k_pool, index)
    sp = _ptr(scores, "scores", _F32, index, 4)
    ss = scores.shape
    if len(ss) != 3 or ss[0] != S or ss[1] != Hkv:
        raise ValueError("scores must be [S][Hkv][max_tokens]")
    dp = _ptr(dst_table, "dst_table", _I32, index, 4)
    ds = dst_table.shape
    if len(ds) != 2 or ds[0] != S:
        raise ValueError("dst_table must be [S][pages]")
    if budget < 1:
        raise ValueError("budget must be positive")
    with _on(index, stream):
        scores_out, xp = _out(scores_out, "scores_out", ss, _F32, index, 4)
        kept, new_lens = _new((S, Hkv, budget), _I32, index), _new((S,), _I32, index)
        _check(lib().pa_evict_tokens(_ref(b), sp, ss[2], kp, vp, dp, ds[1], budget, sinks, recent, xp, kept.data_ptr(),
                                     new_lens.data_ptr(), _current(index)), "pa_evict_tokens")
    return new_lens, kept, scores_out
