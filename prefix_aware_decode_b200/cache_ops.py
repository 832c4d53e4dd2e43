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

_I32, _F32, _F64, _BF16 = torch.int32, torch.float32, torch.float64, torch.bfloat16


def _ptr(t, name: str, dtype, device, align: int = 16) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, the pools' device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    p = t.data_ptr()
    if p % align:
        raise ValueError(f"{name} must be {align}-byte aligned")
    return p


def _rows_ptr(t, name: str, heads: int, rows: int, D: int, device) -> Tuple[int, int]:
    """Address and row stride of [rows][heads][D] rows, which may be slices of wider ones."""
    if not isinstance(t, torch.Tensor) or t.dtype != _BF16 or tuple(t.shape) != (rows, heads, D):
        raise ValueError(f"{name} must be a bf16 tensor [{rows}][{heads}][{D}]")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, the pools' device")
    s = t.stride()
    if (D > 1 and s[2] != 1) or (heads > 1 and s[1] != D):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    stride = s[0] if rows > 1 else heads * D
    if stride < heads * D or stride % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: rows must not overlap and must be 16-byte aligned")
    return t.data_ptr(), stride


class _Call:
    """The device and stream of a call, made current for its launches and allocations."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError("the pools must be CUDA tensors")
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream is not None and stream.device != device:
            raise ValueError(f"stream must be a stream of {device}")
        self.device, self.stream, self.ctx = device, stream, None

    def __enter__(self) -> int:
        if self.stream is not None:
            self.ctx = torch.cuda.stream(self.stream)
        elif self.device.index != torch.cuda.current_device():
            self.ctx = torch.cuda.device(self.device)
        if self.ctx is not None:
            self.ctx.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _sessions(k_pool, block_table, kv_lens, cu_rows, num_rows: int, num_q_heads: Optional[int]) -> PaSessions:
    if not isinstance(k_pool, torch.Tensor) or k_pool.dim() != 4:
        raise ValueError("k_pool must be a tensor [num_pages][Hkv][P][D]")
    dev = k_pool.device
    num_pages, Hkv, P, D = k_pool.shape
    bt = _ptr(block_table, "block_table", _I32, dev, 4)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [S][max_pages]")
    S, max_pages = block_table.shape
    kv = _ptr(kv_lens, "kv_lens", _I32, dev, 4)
    if tuple(kv_lens.shape) != (S,):
        raise ValueError("kv_lens must be [S], S the rows of block_table")
    cu = None
    if cu_rows is not None:
        cu = _ptr(cu_rows, "cu_rows", _I32, dev, 4)
        if tuple(cu_rows.shape) != (S + 1,):
            raise ValueError("cu_rows must be [S + 1], S the rows of block_table")
    return PaSessions(S, num_rows, Hkv if num_q_heads is None else num_q_heads, Hkv, D, P, max_pages, num_pages, bt, kv,
                      cu)


def _pools(k_pool, v_pool) -> Tuple[int, int]:
    dev = k_pool.device
    if v_pool.shape != k_pool.shape:
        raise ValueError("v_pool must have k_pool's shape")
    return _ptr(k_pool, "k_pool", _BF16, dev), _ptr(v_pool, "v_pool", _BF16, dev)


def _q(q, D: int, device) -> int:
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[2] != D:
        raise ValueError("q must be [rows][Hq][D], D that of the pools")
    return _ptr(q, "q", _BF16, device)


def _out(t, name: str, shape, dtype, device, align: int = 16):
    """(tensor, address) of an output: the caller's, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    return t, _ptr(t, name, dtype, device, align)


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
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [rows][Hq][D]")
    rows, Hq = q.shape[0], q.shape[1]
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, rows, Hq)
    if cu_rows is None:
        raise ValueError("cu_rows is needed")
    dev, D, Hkv = k_pool.device, b.head_dim, b.num_kv_heads
    qp, qs = _rows_ptr(q, "q", Hq, rows, D, dev)
    kp, ks = _rows_ptr(k, "k", Hkv, rows, D, dev)
    vp, vs = _rows_ptr(v, "v", Hkv, rows, D, dev)
    pos = _ptr(positions, "positions", _I32, dev, 4)
    if positions.dim() not in (1, 2) or positions.shape[-1] != rows:
        raise ValueError("positions must be [rows] or [n_axes][rows]")
    n_axes = 1 if positions.dim() == 1 else positions.shape[0]
    inv = _ptr(inv_freq, "inv_freq", _F64, dev, 8)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [R / 2]")
    pairs = inv_freq.shape[0]
    if axes is not None:
        axes = bytes(axes)
        if len(axes) != pairs:
            raise ValueError("axes must name the axis of each of inv_freq's pairs")
    pools = _pools(k_pool, v_pool)
    rope = PaRope(2 * pairs, n_axes, 1 if interleaved else 0, axes, pos, inv)
    with _Call(dev, stream) as cs:
        q_out, op = _out(q_out, "q_out", (rows, Hq, D), _BF16, dev)
        _check(lib().pa_rope_append(ctypes.byref(b), ctypes.byref(rope), qp, qs, kp, ks, vp, vs, *pools, op, cs),
               "pa_rope_append")
    return q_out


def window_workspace(q, k_pool, block_table, kv_lens, cu_rows, *, window: int = 0, sinks: int = 0):
    """A workspace for window_attend calls of these shapes (pa_window_workspace_size):
    one serves any number of calls in stream order, calls that may overlap on the
    GPU need one each."""
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, q.shape[0], q.shape[1])
    return _workspace(b, window, sinks, k_pool.device)


def _workspace(b: PaSessions, window: int, sinks: int, device):
    n = ctypes.c_size_t()
    _check(lib().pa_window_workspace_size(ctypes.byref(b), window, sinks, ctypes.byref(n)), "pa_window_workspace_size")
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def window_status(workspace, stream=None) -> int:
    """The device status word of the last window_attend on this workspace
    (pa_window_status; PA_OK unless a bounded wait gave up).  Synchronises the stream."""
    out = ctypes.c_int()
    wp = _ptr(workspace, "workspace", torch.uint8, workspace.device, 256)
    with _Call(workspace.device, stream) as cs:
        _check(lib().pa_window_status(wp, cs, ctypes.byref(out)), "pa_window_status")
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
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [rows][Hq][D]")
    rows, Hq = q.shape[0], q.shape[1]
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, rows, Hq)
    dev, D = k_pool.device, b.head_dim
    qp = _q(q, D, dev)
    pools = _pools(k_pool, v_pool)
    with _Call(dev, stream) as cs:
        out, op = _out(out, "out", (rows, Hq, D), _BF16, dev)
        lse, lp = _out(lse, "lse", (rows, Hq), _F32, dev, 4)
        if workspace is None:
            workspace = _workspace(b, window, sinks, dev)
        wp = _ptr(workspace, "workspace", torch.uint8, dev, 256)
        _check(lib().pa_window_attend(ctypes.byref(b), window, sinks, softmax_scale, qp, *pools, wp, workspace.numel(),
                                      op, lp, cs), "pa_window_attend")
    return out, lse


def weigh_tokens(q, k_pool, lse, block_table, kv_lens, cu_rows, scores, *, window: int = 0, sinks: int = 0,
                 softmax_scale: float = 0.0, stream=None):
    """Adds to scores fp32 [S][Hkv][max_tokens], in place, the attention weight that
    each cached token draws from the batch's rows (pa_weigh_tokens): lse is
    window_attend's for the same q, window, sinks and scale.  Returns scores."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [rows][Hq][D]")
    rows, Hq = q.shape[0], q.shape[1]
    b = _sessions(k_pool, block_table, kv_lens, cu_rows, rows, Hq)
    dev = k_pool.device
    qp, kp = _q(q, b.head_dim, dev), _ptr(k_pool, "k_pool", _BF16, dev)
    lp = _ptr(lse, "lse", _F32, dev, 4)
    if tuple(lse.shape) != (rows, Hq):
        raise ValueError("lse must be [rows][Hq]")
    sp = _ptr(scores, "scores", _F32, dev, 4)
    if scores.dim() != 3 or scores.shape[0] != b.n_sessions or scores.shape[1] != b.num_kv_heads:
        raise ValueError("scores must be [S][Hkv][max_tokens]")
    with _Call(dev, stream) as cs:
        _check(lib().pa_weigh_tokens(ctypes.byref(b), window, sinks, softmax_scale, qp, kp, lp, sp, scores.shape[2], cs),
               "pa_weigh_tokens")
    return scores


def weigh_status(device=None, stream=None) -> int:
    """The first failure of a bounded wait of weigh_tokens on the device since this
    call last returned one (pa_weigh_status; PA_OK: none).  Synchronises the stream."""
    out = ctypes.c_int()
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _Call(device, stream) as cs:
        _check(lib().pa_weigh_status(cs, ctypes.byref(out)), "pa_weigh_status")
    return out.value


def evict_tokens(scores, k_pool, v_pool, block_table, kv_lens, dst_table, budget: int, *, sinks: int = 0,
                 recent: int = 0, scores_out=None, stream=None):
    """Keeps, per (session, kv head), the first `sinks`, the last `recent` and the
    highest-scoring other tokens, `budget` in all, and copies their K and V in
    order to the pages of dst_table int32 [S][n] (pa_evict_tokens; pages that no
    row of block_table names).  Returns (new_lens int32 [S], kept int32
    [S][Hkv][budget] former indices then -1, scores_out fp32 [S][Hkv][max_tokens])."""
    b = _sessions(k_pool, block_table, kv_lens, None, 0, None)
    dev, S, Hkv = k_pool.device, b.n_sessions, b.num_kv_heads
    pools = _pools(k_pool, v_pool)
    sp = _ptr(scores, "scores", _F32, dev, 4)
    if scores.dim() != 3 or scores.shape[0] != S or scores.shape[1] != Hkv:
        raise ValueError("scores must be [S][Hkv][max_tokens]")
    dp = _ptr(dst_table, "dst_table", _I32, dev, 4)
    if dst_table.dim() != 2 or dst_table.shape[0] != S:
        raise ValueError("dst_table must be [S][pages]")
    if budget < 1:
        raise ValueError("budget must be positive")
    with _Call(dev, stream) as cs:
        scores_out, xp = _out(scores_out, "scores_out", scores.shape, _F32, dev, 4)
        kept = torch.empty((S, Hkv, budget), dtype=_I32, device=dev)
        new_lens = torch.empty((S,), dtype=_I32, device=dev)
        _check(lib().pa_evict_tokens(ctypes.byref(b), sp, scores.shape[2], *pools, dp, dst_table.shape[1], budget, sinks,
                                     recent, xp, kept.data_ptr(), new_lens.data_ptr(), cs), "pa_evict_tokens")
    return new_lens, kept, scores_out
