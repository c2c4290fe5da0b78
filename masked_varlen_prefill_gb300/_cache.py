"""Bindings of the bounded paged cache's steps (include/mvp.h): rotary
positions written into the cache, the weight each key received, and eviction
by it.  Argument marshalling only, like ``_lib``.

These calls run once per layer and step on small decode batches, where the
host time of the binding is what a caller waits for; so arguments are checked
in one pass over the tensors and pointers go to ctypes as plain integers.
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch

from ._lib import MVP_OK, MvpError, _on, _rows_of_blocks, _stream, load_library

_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16


def _need(dev, dtype, *named):
    """name, tensor, name, tensor, ...: every tensor given (not None) is
    contiguous, of ``dtype``, on ``dev``."""
    for t in named[1::2]:
        if t is not None and not (t.dtype is dtype and t.device == dev and t.is_contiguous()):
            break
    else:
        return
    for name, t in zip(named[::2], named[1::2]):
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"{name} must be a CUDA tensor on {dev}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _cuda_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _p(t):
    return None if t is None else t.data_ptr()


def _call(fn_name, dev, stream, *args):
    """The C call with ``dev`` current (its tensors' device) on ``stream`` or
    the device's current stream; raises on a non-zero status."""
    st = _on(dev, getattr(load_library(), fn_name), (*args, _stream(stream, dev)))
    if st != MVP_OK:
        raise MvpError(fn_name, st)


def _caches(k_cache, v_cache, block_size):
    """The caches as [rows, Hkv, D], views of the caller's memory, and their
    number of blocks."""
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("the caches differ in shape")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous")
    if len(shape) == 4:
        if shape[1] != block_size:
            raise ValueError(f"the caches' blocks have {shape[1]} rows, not block_size ({block_size})")
        k_cache = k_cache.view(-1, *shape[2:])
        v_cache = v_cache.view(-1, *shape[2:])
        shape = k_cache.shape
    if len(shape) != 3:
        raise ValueError("the caches must be [num_blocks * block_size, Hkv, D]")
    if block_size < 1 or shape[0] % block_size != 0:
        raise ValueError("cache rows must be a multiple of block_size")
    return k_cache, v_cache, shape[0] // block_size


# ------------------------------------------------------------------ rotary positions
class RopeTable:
    """The frequencies and axes of ``rope_append_paged``'s pairs on a device
    (``mvp_rope_table_pack``'s entries).  Made once by ``rope_table``."""

    def __init__(self, entries, num_axes):
        self.entries = entries  # int32 [pairs, 4]
        self.num_axes = num_axes
        self.rot_dim = 2 * entries.shape[0]


def rope_table(inv_freq, axes=None, num_axes=None, device=None) -> RopeTable:
    """Table of rotary pairs: ``inv_freq`` [pairs] (host, radians per position;
    float64, so that far positions keep their angle) and ``axes`` [pairs], the
    position axis each pair follows (None: all follow axis 0)."""
    f = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
    if f.ndim != 1 or f.shape[0] < 1:
        raise ValueError("inv_freq must be a 1-D array of rotary pairs")
    a = np.zeros(f.shape[0], dtype=np.int32) if axes is None else np.ascontiguousarray(np.asarray(axes, np.int32))
    if a.shape != f.shape:
        raise ValueError("axes must give one axis per pair")
    if num_axes is None:
        num_axes = int(a.max()) + 1
    table = np.zeros((f.shape[0], 4), dtype=np.int32)
    st = load_library().mvp_rope_table_pack(f.ctypes.data, a.ctypes.data, f.shape[0], int(num_axes), table.ctypes.data)
    if st != MVP_OK:
        raise MvpError("mvp_rope_table_pack", st)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return RopeTable(torch.from_numpy(table).to(device), int(num_axes))


def _rows_of(name, t, dtype, dev):
    """Shape and row stride of a [total_q, heads, D] tensor whose heads are
    contiguous."""
    shape = t.shape
    if len(shape) != 3 or t.device != dev or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor [total_q, heads, D] on {dev}")
    row, head, one = t.stride()
    rows, heads, d = shape
    if one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name}'s heads must be contiguous")
    return shape, row if rows > 1 else max(row, heads * d)


def rope_append_paged(q, k, v, q_out, k_cache, v_cache, positions, table, cu_seqlens_q, seq_lens_k, block_table,
                      block_size, *, adjacent=False, stream=None):
    """Rotate q into ``q_out`` and k into the paged cache, and copy v into it
    (see ``mvp_rope_append_paged`` in include/mvp.h): the step before
    ``attn_fwd_paged`` with the same offsets and block table.

    q [total_q, Hq, D], k/v [total_q, Hkv, D] bf16 or fp32, rows any stride
    (views of one projection); q_out bf16 like q, contiguous; the caches
    [num_blocks * block_size, Hkv, D] or [num_blocks, block_size, Hkv, D],
    contiguous; positions int32 [num_axes, total_q]; table a ``RopeTable``.
    """
    dev = _cuda_device(q_out, "q_out")
    block_size = int(block_size)
    dtype = q.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise ValueError(f"q must be bfloat16 or float32, got {dtype}")
    q_shape, qs = _rows_of("q", q, dtype, dev)
    k_shape, ks = _rows_of("k", k, dtype, dev)
    v_shape, vs = _rows_of("v", v, dtype, dev)
    k_cache, v_cache, num_blocks = _caches(k_cache, v_cache, block_size)
    _need(dev, _BF16, "q_out", q_out, "k_cache", k_cache, "v_cache", v_cache)
    _need(dev, _I32, "positions", positions, "table", table.entries, "cu_seqlens_q", cu_seqlens_q, "seq_lens_k",
          seq_lens_k, "block_table", block_table)
    total, hq, d = q_shape
    _, hkv, dk = k_cache.shape
    if q_out.shape != q_shape or k_shape != (total, hkv, d) or v_shape != k_shape or dk != d:
        raise ValueError("q and q_out must be [total_q, Hq, D], k and v [total_q, Hkv, D], the caches [.., Hkv, D]")
    if positions.shape != (table.num_axes, total):
        raise ValueError(f"positions must be [{table.num_axes}, total_q]")
    num_reqs = seq_lens_k.shape[0]
    bt_shape = block_table.shape
    if cu_seqlens_q.shape != (num_reqs + 1,) or len(bt_shape) != 2 or bt_shape[0] != num_reqs:
        raise ValueError("cu_seqlens_q must be [B + 1], seq_lens_k [B] and block_table [B, max_blocks_per_seq]")
    _call("mvp_rope_append_paged", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), dtype is _F32,
          q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), positions.data_ptr(), table.entries.data_ptr(),
          table.num_axes, table.rot_dim, bool(adjacent), cu_seqlens_q.data_ptr(), seq_lens_k.data_ptr(),
          block_table.data_ptr(), block_size, bt_shape[1], num_blocks, num_reqs, total, hq, hkv, d, qs, ks, vs)


# ------------------------------------------------------------------ weights
def key_weights_workspace_size(num_reqs, num_heads_kv, max_q_len, max_k_len) -> int:
    return int(load_library().mvp_key_weights_workspace_size(num_reqs, num_heads_kv, max_q_len, max_k_len))


def _key_weights(fn_name, q, k, lse, weights, slots, accumulate, cu_seqlens_q, key_args, context_lens, max_q_len,
                 max_k_len, total_k, num_decode_reqs, range_table, range_covered, causal, window_left, window_right,
                 first_tokens, sinks, sink_mode, scale, workspace, stream):
    dev = _cuda_device(q, "q")
    _need(dev, _BF16, "q", q, "k", k)
    _need(dev, _F32, "lse", lse, "sinks", sinks)
    _need(dev, _I32, "cu_seqlens_q", cu_seqlens_q, "context_lens", context_lens, "range_table", range_table,
          "range_covered", range_covered)
    if q.dim() != 3 or k.dim() != 3 or q.shape[2] != k.shape[2]:
        raise ValueError("q must be [total_q, Hq, D] and the keys [.., Hkv, D]")
    total_q, hq, d = q.shape
    hkv = k.shape[1]
    num_reqs = cu_seqlens_q.shape[0] - 1
    if lse.shape != (hq, total_q):
        raise ValueError("lse must be [Hq, total_q]")
    if sinks is not None and sinks.shape != (hq,):
        raise ValueError("sinks must be [Hq]")
    if range_table is not None and range_table.shape != (total_q, 2):
        raise ValueError("range_table must be [total_q, 2]")
    if context_lens is not None and context_lens.shape != (num_reqs,):
        raise ValueError("context_lens must be [B]")
    _weight_args(weights, slots, num_reqs, hkv, dev)
    ws = 0
    if workspace is not None:
        _need(dev, torch.uint8, "workspace", workspace)
        ws = workspace.numel()
    rows = (total_q,) if total_k is None else (total_q, total_k)
    scale = d ** -0.5 if scale is None else float(scale)
    _call(fn_name, dev, stream, q.data_ptr(), k.data_ptr(), lse.data_ptr(), weights.data_ptr(), weights.shape[0],
          weights.shape[2], _p(slots), bool(accumulate), cu_seqlens_q.data_ptr(), *key_args, _p(context_lens),
          num_reqs, *rows, int(max_q_len), int(max_k_len), int(num_decode_reqs), hq, hkv, d, _p(range_table),
          _p(range_covered), bool(causal), int(window_left), int(window_right), int(first_tokens), _p(sinks),
          int(sink_mode), scale, _p(workspace), ws)


def attn_key_weights_varlen(q, k, lse, weights, cu_seqlens_q, cu_seqlens_k, max_q_len, max_k_len, *, slots=None,
                            context_lens=None, range_table=None, range_covered=None, causal=True, window_left=-1,
                            window_right=-1, first_tokens=0, sinks=None, sink_mode=0, scale=None, accumulate=True,
                            workspace=None, num_decode_reqs=-1, stream=None):
    """Add (or, with ``accumulate=False``, write) the attention weight each
    key received to ``weights`` fp32 [num_slots, Hkv, max_len]: the column
    sums of the probabilities of the ``attn_fwd_varlen`` call with these
    arguments that wrote ``lse`` (see ``mvp_attn_key_weights_varlen``)."""
    dev = _cuda_device(q, "q")
    _need(dev, _I32, "cu_seqlens_k", cu_seqlens_k)
    if cu_seqlens_k.shape != cu_seqlens_q.shape:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must be [B + 1]")
    _key_weights("mvp_attn_key_weights_varlen", q, k, lse, weights, slots, accumulate, cu_seqlens_q,
                 (cu_seqlens_k.data_ptr(),), context_lens, max_q_len, max_k_len, k.shape[0], num_decode_reqs,
                 range_table, range_covered, causal, window_left, window_right, first_tokens, sinks, sink_mode, scale,
                 workspace, stream)


def attn_key_weights_paged(q, k_cache, lse, weights, cu_seqlens_q, seq_lens_k, block_table, block_size, max_q_len,
                           max_k_len, *, slots=None, context_lens=None, range_table=None, range_covered=None,
                           causal=True, window_left=-1, window_right=-1, first_tokens=0, sinks=None, sink_mode=0,
                           scale=None, accumulate=True, workspace=None, num_decode_reqs=-1, stream=None):
    """``attn_key_weights_varlen`` over a paged cache: the weights of the
    ``attn_fwd_paged`` call with these arguments."""
    dev = _cuda_device(q, "q")
    block_size = int(block_size)
    if len(k_cache.shape) == 4 and k_cache.shape[1] == block_size:
        k_cache = _rows_of_blocks(k_cache, stream)
    k_cache, _, num_blocks = _caches(k_cache, k_cache, block_size)
    _need(dev, _I32, "seq_lens_k", seq_lens_k, "block_table", block_table)
    num_reqs = seq_lens_k.shape[0]
    if cu_seqlens_q.shape != (num_reqs + 1,) or block_table.dim() != 2 or block_table.shape[0] != num_reqs:
        raise ValueError("cu_seqlens_q must be [B + 1], seq_lens_k [B] and block_table [B, max_blocks_per_seq]")
    _key_weights("mvp_attn_key_weights_paged", q, k_cache, lse, weights, slots, accumulate, cu_seqlens_q,
                 (seq_lens_k.data_ptr(), block_table.data_ptr(), block_size, block_table.shape[1], num_blocks),
                 context_lens, max_q_len, max_k_len, None, num_decode_reqs, range_table, range_covered, causal,
                 window_left, window_right, first_tokens, sinks, sink_mode, scale, workspace, stream)


# ------------------------------------------------------------------ eviction
def kv_evict_workspace_size(num_reqs, num_heads_kv, budget) -> int:
    return int(load_library().mvp_kv_evict_workspace_size(num_reqs, num_heads_kv, budget))


def _weight_args(weights, slots, num_reqs, hkv, dev, name="weights"):
    _need(dev, _F32, name, weights)
    if weights.dim() != 3 or weights.shape[1] != hkv:
        raise ValueError(f"{name} must be [num_slots, Hkv, max_len]")
    if slots is not None:
        _need(dev, _I32, "slots", slots)
        if slots.shape != (num_reqs,):
            raise ValueError("slots must be [B]")


def kv_evict_paged(k_cache, v_cache, weights, seq_lens_k, block_table, block_size, budget, new_seq_lens, kept,
                   workspace, max_k_len, *, first_tokens=0, recent_tokens=0, block_table_out=None, weights_out=None,
                   slots=None, stream=None):
    """Evict each request's keys down to ``budget`` per KV head by their
    weights, keeping the first and the most recent ones (see
    ``mvp_kv_evict_paged`` in include/mvp.h).

    The caches are [num_blocks * block_size, Hkv, D] or [num_blocks,
    block_size, Hkv, D], contiguous; weights fp32 [num_slots, Hkv, max_len];
    new_seq_lens int32 [B] and kept int32 [B, Hkv, budget] are written;
    workspace uint8 of ``kv_evict_workspace_size(B, Hkv, budget)`` bytes.  In
    place unless ``block_table_out`` / ``weights_out`` say where the kept keys
    go.
    """
    dev = _cuda_device(k_cache, "k_cache")
    block_size, budget = int(block_size), int(budget)
    k_cache, v_cache, num_blocks = _caches(k_cache, v_cache, block_size)
    _need(dev, _BF16, "k_cache", k_cache, "v_cache", v_cache)
    _need(dev, _I32, "seq_lens_k", seq_lens_k, "block_table", block_table, "block_table_out", block_table_out,
          "new_seq_lens", new_seq_lens, "kept", kept)
    _need(dev, torch.uint8, "workspace", workspace)
    num_reqs, hkv, d = seq_lens_k.shape[0], k_cache.shape[1], k_cache.shape[2]
    _weight_args(weights, slots, num_reqs, hkv, dev)
    if weights_out is not None:
        _need(dev, _F32, "weights_out", weights_out)
        if weights_out.shape != weights.shape:
            raise ValueError("weights_out must be like weights")
    for t in (block_table, block_table_out):
        if t is not None and (t.dim() != 2 or t.shape[0] != num_reqs):
            raise ValueError("block tables must be [B, max_blocks_per_seq]")
    if new_seq_lens.shape != (num_reqs,) or kept.shape != (num_reqs, hkv, budget):
        raise ValueError("new_seq_lens must be [B] and kept [B, Hkv, budget]")
    _call("mvp_kv_evict_paged", dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(),
          _p(weights_out), weights.shape[0], weights.shape[2], _p(slots), seq_lens_k.data_ptr(),
          block_table.data_ptr(), _p(block_table_out), block_size, block_table.shape[1],
          0 if block_table_out is None else block_table_out.shape[1], num_blocks, num_reqs, int(max_k_len), hkv, d, budget,
          int(first_tokens), int(recent_tokens), new_seq_lens.data_ptr(), kept.data_ptr(), workspace.data_ptr(),
          workspace.numel())
