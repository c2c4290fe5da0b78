"""Bindings of a page pool's steps (include/mvp.h): pages of paged K/V caches
taken, shared, freed and compacted.  Argument marshalling only, like ``_lib``.

A pool is ``refs`` int32 [num_blocks] (the holders of each page; free when
<= 0), the block tables and lengths that the attention calls read, and the
caches of every layer that goes by them (a ``KVCaches``).
"""

from __future__ import annotations

import ctypes

import torch

from ._cache import _I32, _call, _cuda_device, _need
from ._lib import load_library


class KVCaches:
    """The caches of a pool, as ``kv_extend_paged`` and ``kv_compact_paged``
    take them.  Made once by ``kv_caches``."""

    def __init__(self, tensors, block_size, num_blocks, row_bytes):
        self.tensors = tensors  # (kept alive: the pointers are theirs)
        self.block_size = block_size
        self.num_blocks = num_blocks
        self.row_bytes = row_bytes
        self.device = tensors[0].device
        self.count = len(tensors)
        self._array = (ctypes.c_void_p * self.count)(*[t.data_ptr() for t in tensors])
        self.pointers = ctypes.addressof(self._array)


def kv_caches(caches, block_size) -> KVCaches:
    """The K and V caches of every layer that goes by the same block tables:
    tensors [num_blocks, block_size, Hkv, D] or [num_blocks * block_size, Hkv,
    D], contiguous, alike in shape, type (any) and device."""
    tensors, block_size = list(caches), int(block_size)
    if not tensors:
        raise ValueError("a pool needs at least one cache")
    dev, shape = _cuda_device(tensors[0], "caches"), tensors[0].shape
    for t in tensors:
        _need(dev, tensors[0].dtype, "caches", t)
        if t.shape != shape:
            raise ValueError("the caches differ in shape")
    if len(shape) not in (3, 4) or (len(shape) == 4 and shape[1] != block_size):
        raise ValueError("the caches must be [num_blocks, block_size, Hkv, D] or [num_blocks * block_size, Hkv, D]")
    rows = shape[0] * (block_size if len(shape) == 4 else 1)
    if block_size < 1 or rows < block_size or rows % block_size != 0:
        raise ValueError("cache rows must be a multiple of block_size")
    return KVCaches(tensors, block_size, rows // block_size, shape[-1] * shape[-2] * tensors[0].element_size())


# These calls run every step on small arrays, where their host time is what a
# caller waits for: one pass over the tensors, and messages only when it fails.
def _checked(refs, num_blocks, *named):
    """refs [num_blocks] and name, tensor, shape, name, tensor, shape, ...: all
    int32, contiguous and on refs' device, which is returned.  A shape of None:
    a table of two dimensions."""
    dev = refs.device
    if refs.is_cuda and refs.dtype is _I32 and refs.is_contiguous() and refs.shape == (num_blocks,):
        for t, shape in zip(named[1::3], named[2::3]):
            if not (t.dtype is _I32 and t.device == dev and t.is_contiguous() and
                    (t.shape == shape if shape is not None else t.dim() == 2)):
                break
        else:
            return dev
    _need(_cuda_device(refs, "refs"), _I32, "refs", refs)
    if refs.shape != (num_blocks,):
        raise ValueError(f"refs must be [{num_blocks}]")
    for name, t, shape in zip(named[::3], named[1::3], named[2::3]):
        _need(dev, _I32, name, t)
        if shape is None and t.dim() != 2:
            raise ValueError(f"{name} must be [B, max_blocks]")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError("arguments of a pool must be int32 tensors on one device")


def _workspace(workspace, dev):
    if not (workspace.dtype is torch.uint8 and workspace.device == dev and workspace.is_contiguous()):
        _need(dev, torch.uint8, "workspace", workspace)
    return workspace.data_ptr(), workspace.numel()


def kv_extend_workspace_size(num_reqs) -> int:
    return int(load_library().mvp_kv_extend_workspace_size(num_reqs))


def kv_compact_workspace_size(num_blocks) -> int:
    return int(load_library().mvp_kv_compact_workspace_size(num_blocks))


def kv_extend_paged(caches, refs, block_table, seq_lens_k, add_lens, new_seq_lens, missing, workspace, *, stream=None):
    """Take pages for ``add_lens`` more tokens in each request, lowest ids
    first; a partly filled page with other holders is copied (see
    ``mvp_kv_extend_paged`` in include/mvp.h).

    caches a ``KVCaches``; refs int32 [num_blocks], block_table int32 [B,
    max_blocks] and missing int32 [1] are written, new_seq_lens int32 [B] too
    (it may be seq_lens_k); workspace uint8 of ``kv_extend_workspace_size(B)``
    bytes.  All or nothing: ``missing`` is 0, or says how many pages the pool
    lacks (-1: a length that the table cannot hold) and nothing has changed.
    """
    b = block_table.shape[:1]
    dev = _checked(refs, caches.num_blocks, "block_table", block_table, None, "seq_lens_k", seq_lens_k, b, "add_lens",
                   add_lens, b, "new_seq_lens", new_seq_lens, b, "missing", missing, (1,))
    if caches.device != dev:
        raise ValueError(f"the caches must be on {dev}")
    _call("mvp_kv_extend_paged", dev, stream, caches.pointers, caches.count, caches.row_bytes, refs.data_ptr(),
          caches.num_blocks, block_table.data_ptr(), block_table.shape[1], caches.block_size, seq_lens_k.data_ptr(),
          add_lens.data_ptr(), new_seq_lens.data_ptr(), b[0], missing.data_ptr(), *_workspace(workspace, dev))


def kv_fork_paged(refs, block_table, seq_lens_k, parents, block_table_out, seq_lens_out, block_size, *, stream=None):
    """A new batch whose row i continues row ``parents[i]`` of the old one,
    sharing its pages; rows that nothing continues give theirs up (see
    ``mvp_kv_fork_paged`` in include/mvp.h).  parents int32 [B_out]; the new
    table int32 [B_out, >= max_blocks] and lengths int32 [B_out] are written,
    in memory of their own."""
    num_blocks, b, b_out = refs.numel(), block_table.shape[:1], block_table_out.shape[:1]
    dev = _checked(refs, num_blocks, "block_table", block_table, None, "seq_lens_k", seq_lens_k, b, "parents", parents,
                   b_out, "block_table_out", block_table_out, None, "seq_lens_out", seq_lens_out, b_out)
    _call("mvp_kv_fork_paged", dev, stream, refs.data_ptr(), num_blocks, block_table.data_ptr(), seq_lens_k.data_ptr(),
          b[0], block_table.shape[1], parents.data_ptr(), b_out[0], block_table_out.data_ptr(),
          block_table_out.shape[1], seq_lens_out.data_ptr(), int(block_size))


def kv_trim_paged(refs, block_table, seq_lens_k, new_seq_lens, block_size, *, stream=None):
    """Cut requests to ``new_seq_lens`` (0 frees them): their pages past it
    lose a holder, seq_lens_k is written (see ``mvp_kv_trim_paged`` in
    include/mvp.h)."""
    num_blocks, b = refs.numel(), block_table.shape[:1]
    dev = _checked(refs, num_blocks, "block_table", block_table, None, "seq_lens_k", seq_lens_k, b, "new_seq_lens",
                   new_seq_lens, b)
    _call("mvp_kv_trim_paged", dev, stream, refs.data_ptr(), num_blocks, block_table.data_ptr(), block_table.shape[1],
          seq_lens_k.data_ptr(), new_seq_lens.data_ptr(), b[0], int(block_size))


def kv_compact_paged(caches, refs, block_table, seq_lens_k, block_map, num_live, workspace, *, stream=None):
    """Move the live pages of a pool to its lowest ids, in every cache, and
    rewrite the block table (see ``mvp_kv_compact_paged`` in include/mvp.h).
    block_map int32 [num_blocks] (each page's new id, -1: free) and num_live
    int32 [1] are written; workspace uint8 of
    ``kv_compact_workspace_size(num_blocks)`` bytes."""
    num_blocks, b = caches.num_blocks, block_table.shape[:1]
    dev = _checked(refs, num_blocks, "block_table", block_table, None, "seq_lens_k", seq_lens_k, b, "block_map",
                   block_map, (num_blocks,), "num_live", num_live, (1,))
    if caches.device != dev:
        raise ValueError(f"the caches must be on {dev}")
    _call("mvp_kv_compact_paged", dev, stream, caches.pointers, caches.count, caches.row_bytes, refs.data_ptr(),
          num_blocks, block_table.data_ptr(), block_table.shape[1], caches.block_size, seq_lens_k.data_ptr(), b[0],
          block_map.data_ptr(), num_live.data_ptr(), *_workspace(workspace, dev))
