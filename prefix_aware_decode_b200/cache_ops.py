"""Operators on the paged cache of device-resident sessions (pa.h, "session
caches on the device"): append with rotary positions, attention with a sliding
window and sinks, accumulated attention weights, and eviction.

Every call takes the sessions' block table [S][max_pages], cached lengths [S]
and row offsets [S + 1] as int32 CUDA tensors and reads them when its kernels
run: nothing is planned on the host or copied back, so a call can be captured
into a CUDA graph and replayed as the lengths and tables change in place.  Kernels
are chosen by the table's width, which bounds the lengths: a table no wider than the
steps need is the faster one.

All tensors of a call live on one device, which need not be the current one.
A call runs on `stream` (a torch stream of that device, or a cudaStream_t), or on
the device's current stream; outputs and workspaces that it allocates belong to
that stream.  There is no backward: tensors that require grad are refused unless
grad mode is off.  Argument errors raise ValueError (TypeError for what is no tensor),
errors of the library PaError.
"""
from __future__ import annotations

import os
from typing import Optional, Sequence

import torch

from ._binding import LIB_PATH

if not os.path.exists(LIB_PATH) or not os.path.exists(os.path.join(os.path.dirname(LIB_PATH), "_cache_ops.so")):
    raise RuntimeError("libpa.so or _cache_ops.so is missing: build them first (python -c 'import __graft_entry__ as g; "
                       "g.build()'); there is no fallback path")
from . import _cache_ops as _ops  # noqa: E402  (needs torch loaded)


def _on(stream, device):
    """Makes a stream current: a torch stream of the device, or a cudaStream_t."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError(f"stream must be a stream of {device}")
    return torch.cuda.stream(stream)


def _index(device) -> int:
    index = None if device is None else torch.device(device).index
    return torch.cuda.current_device() if index is None else index


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
    if axes is not None:
        axes = bytes(axes)
    if stream is not None:
        with _on(stream, k_pool.device):
            return _ops.rope_append(q, k, v, positions, inv_freq, k_pool, v_pool, block_table, kv_lens, cu_rows, axes,
                                    interleaved, q_out)
    return _ops.rope_append(q, k, v, positions, inv_freq, k_pool, v_pool, block_table, kv_lens, cu_rows, axes,
                            interleaved, q_out)


def window_workspace(q, k_pool, block_table, kv_lens, cu_rows, *, window: int = 0, sinks: int = 0):
    """A workspace for window_attend calls of these shapes (pa_window_workspace_size):
    one serves any number of calls in stream order, calls that may overlap on the
    GPU need one each."""
    return _ops.window_workspace(q, k_pool, block_table, kv_lens, cu_rows, window, sinks)


def window_status(workspace=None, stream=None, device=None) -> int:
    """The device status word of the last window_attend on this workspace
    (pa_window_status; PA_OK unless a bounded wait gave up: the results are then not
    to be used).  Without a workspace: the first failure of any window_attend on the
    device since this call last returned one.  Synchronises the stream."""
    index = _index(device) if workspace is None else -1
    if stream is not None:
        with _on(stream, torch.device("cuda", index) if workspace is None else workspace.device):
            return _ops.window_status(workspace, index)
    return _ops.window_status(workspace, index)


def window_attend(q, k_pool, v_pool, block_table, kv_lens, cu_rows, *, window: int = 0, sinks: int = 0,
                  softmax_scale: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of the last rows of every session over its cache, with a
    sliding window and sinks (pa_window_attend): the row at position p sees token
    t when t <= p and (window == 0 or t > p - window or t < sinks).

    q bf16 [rows][Hq][D]; pools bf16 [num_pages][Hkv][P][D].  Returns (out bf16
    [rows][Hq][D], lse fp32 [rows][Hq]); rows that see nothing get 0 and -inf, rows
    of no session are not written (undefined in tensors that the call allocates).
    `workspace` (window_workspace) is allocated by the call when not given;
    window_status() then tells whether a call gave up.
    """
    if stream is not None:
        with _on(stream, k_pool.device):
            return _ops.window_attend(q, k_pool, v_pool, block_table, kv_lens, cu_rows, window, sinks, softmax_scale,
                                      out, lse, workspace)
    return _ops.window_attend(q, k_pool, v_pool, block_table, kv_lens, cu_rows, window, sinks, softmax_scale, out, lse,
                              workspace)


def weigh_tokens(q, k_pool, lse, block_table, kv_lens, cu_rows, scores, *, window: int = 0, sinks: int = 0,
                 softmax_scale: float = 0.0, stream=None):
    """Adds to scores fp32 [S][Hkv][max_tokens], in place, the attention weight that
    each cached token draws from the batch's rows (pa_weigh_tokens): lse is
    window_attend's for the same q, window, sinks and scale.  Returns scores."""
    if stream is not None:
        with _on(stream, k_pool.device):
            return _ops.weigh_tokens(q, k_pool, lse, block_table, kv_lens, cu_rows, scores, window, sinks, softmax_scale)
    return _ops.weigh_tokens(q, k_pool, lse, block_table, kv_lens, cu_rows, scores, window, sinks, softmax_scale)


def weigh_status(device=None, stream=None) -> int:
    """The first failure of a bounded wait of weigh_tokens on the device since this
    call last returned one (pa_weigh_status; PA_OK: none).  Synchronises the stream."""
    index = _index(device)
    if stream is not None:
        with _on(stream, torch.device("cuda", index)):
            return _ops.weigh_status(index)
    return _ops.weigh_status(index)


def evict_tokens(scores, k_pool, v_pool, block_table, kv_lens, dst_table, budget: int, *, sinks: int = 0,
                 recent: int = 0, scores_out=None, stream=None):
    """Keeps, per (session, kv head), the first `sinks`, the last `recent` and the
    highest-scoring other tokens, `budget` in all, and copies their K and V in
    order to the pages of dst_table int32 [S][n] (pa_evict_tokens; pages that no
    row of block_table names, as SessionPool.compact and then tables(sessions,
    max_pages=the budget's pages) give them; n pages hold the budget; a kept
    token in a hole becomes one of zeros).  Returns (new_lens int32 [S], kept int32
    [S][Hkv][budget] former indices then -1, scores_out fp32 [S][Hkv][max_tokens])."""
    if stream is not None:
        with _on(stream, k_pool.device):
            return _ops.evict_tokens(scores, k_pool, v_pool, block_table, kv_lens, dst_table, budget, sinks, recent,
                                     scores_out)
    return _ops.evict_tokens(scores, k_pool, v_pool, block_table, kv_lens, dst_table, budget, sinks, recent, scores_out)
