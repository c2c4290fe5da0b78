"""The pages of a pool without a GPU: the oracle's own properties, refusals
before any launch, and what the binding hands over."""

import ctypes

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import _pages
from oracle import pages as op

from . import test_binding_host as tb
from .test_binding_host import BF16, FakeTensor, calls  # noqa: F401

P = 1 << 20
U8 = torch.uint8


@pytest.fixture(scope="module")
def lib():
    return mvp.load_library()


def _pointers(*p):
    return (ctypes.c_void_p * len(p))(*p)


def _extend(lib, **over):
    a = dict(caches=_pointers(P, P), n=2, row=256, refs=P, blocks=8, bt=P, width=4, block=16, lens=P, add=P, new=P, reqs=3,
             missing=P, ws=P, ws_bytes=4096, stream=None)
    return lib.mvp_kv_extend_paged(*{**a, **over}.values())


def test_extend_argument_errors(lib):
    for bad in (dict(block=8), dict(block=48), dict(block=512), dict(blocks=0), dict(width=0), dict(reqs=-1), dict(n=-1),
                dict(caches=None), dict(caches=_pointers(P, None)), dict(refs=None), dict(bt=None), dict(lens=None),
                dict(add=None), dict(new=None), dict(missing=None), dict(ws=None)):
        assert _extend(lib, **bad) == mvp.MVP_ERR_ARG, bad
    for bad in (dict(row=24), dict(row=0), dict(row=(1 << 24) + 16), dict(caches=_pointers(P, P + 8)), dict(ws=P + 4),
                dict(n=257, caches=_pointers(*[P] * 257)), dict(reqs=65536, ws_bytes=1 << 30)):
        assert _extend(lib, **bad) == mvp.MVP_ERR_UNSUPPORTED, bad
    assert _extend(lib, ws_bytes=mvp.kv_extend_workspace_size(3) - 1) == mvp.MVP_ERR_CAPACITY


def test_fork_argument_errors(lib):
    a = dict(refs=P, blocks=8, bt=P, lens=P, reqs=3, width=4, parents=P, out=2, bt_out=2 * P, width_out=4, lens_out=2 * P,
             block=16, stream=None)
    call = lambda **over: lib.mvp_kv_fork_paged(*{**a, **over}.values())  # noqa: E731
    for bad in (dict(block=20), dict(blocks=0), dict(reqs=-1), dict(out=-1), dict(width=0), dict(width_out=3), dict(refs=None),
                dict(bt=None), dict(lens=None), dict(parents=None), dict(bt_out=None), dict(lens_out=None), dict(bt_out=P),
                dict(lens_out=P)):
        assert call(**bad) == mvp.MVP_ERR_ARG, bad
    assert call(reqs=0, out=0) == mvp.MVP_OK
    assert call(out=1 << 25) == mvp.MVP_ERR_UNSUPPORTED


def test_trim_argument_errors(lib):
    a = dict(refs=P, blocks=8, bt=P, width=4, lens=P, keep=P, reqs=3, block=16, stream=None)
    call = lambda **over: lib.mvp_kv_trim_paged(*{**a, **over}.values())  # noqa: E731
    for bad in (dict(block=0), dict(blocks=0), dict(width=0), dict(reqs=-1), dict(refs=None), dict(bt=None), dict(lens=None),
                dict(keep=None)):
        assert call(**bad) == mvp.MVP_ERR_ARG, bad
    assert call(reqs=0) == mvp.MVP_OK


def test_compact_argument_errors(lib):
    a = dict(caches=_pointers(P, P), n=2, row=256, refs=P, blocks=8, bt=P, width=4, block=16, lens=P, reqs=3, map=P, live=P,
             ws=P, ws_bytes=4096, stream=None)
    call = lambda **over: lib.mvp_kv_compact_paged(*{**a, **over}.values())  # noqa: E731
    for bad in (dict(block=3), dict(blocks=0), dict(width=0), dict(reqs=-1), dict(refs=None), dict(bt=None), dict(lens=None),
                dict(map=None), dict(live=None), dict(ws=None), dict(caches=None)):
        assert call(**bad) == mvp.MVP_ERR_ARG, bad
    for bad in (dict(row=8), dict(caches=_pointers(P + 4, P)), dict(ws=P + 8)):
        assert call(**bad) == mvp.MVP_ERR_UNSUPPORTED, bad
    assert call(ws_bytes=mvp.kv_compact_workspace_size(8) - 1) == mvp.MVP_ERR_CAPACITY


def test_workspace_sizes(lib):
    assert mvp.kv_extend_workspace_size(0) == mvp.kv_compact_workspace_size(0) == 0
    assert mvp.kv_extend_workspace_size(-3) == mvp.kv_compact_workspace_size(-1) == 0
    assert mvp.kv_extend_workspace_size(10) == 256 + 240
    assert mvp.kv_compact_workspace_size(9) == 256 + 40


# ------------------------------------------------------------------ the binding
def _handle():
    return mvp.kv_caches([FakeTensor((4, 16, 2, 64), BF16), FakeTensor((4, 16, 2, 64), BF16)], 16)


T = FakeTensor
CALLS = [
    ("mvp_kv_extend_paged", lambda **kw: mvp.kv_extend_paged(_handle(), T((4,)), T((3, 5)), T((3,)), T((3,)), T((3,)),
                                                            T((1,)), T((512,), U8), **kw)),
    ("mvp_kv_fork_paged", lambda **kw: mvp.kv_fork_paged(T((4,)), T((3, 5)), T((3,)), T((2,)), T((2, 5)), T((2,)), 16,
                                                         **kw)),
    ("mvp_kv_trim_paged", lambda **kw: mvp.kv_trim_paged(T((4,)), T((3, 5)), T((3,)), T((3,)), 16, **kw)),
    ("mvp_kv_compact_paged", lambda **kw: mvp.kv_compact_paged(_handle(), T((4,)), T((3, 5)), T((3,)), T((4,)), T((1,)),
                                                               T((512,), U8), **kw)),
]


@pytest.mark.parametrize("name,call", CALLS, ids=[n for n, _ in CALLS])
def test_the_tensors_device_is_current_in_the_call(calls, name, call):  # noqa: F811
    call()
    assert calls[0][:2] == (name, 1) and 101 in calls[0][2]

    class Stream:
        device = tb.DEV
        cuda_stream = 777

    call(stream=Stream())
    assert calls[1][:2] == (name, 1) and 777 in calls[1][2]


def test_a_pools_caches():
    h = _handle()
    assert (h.num_blocks, h.block_size, h.row_bytes, h.count) == (4, 16, 256, 2)
    h = mvp.kv_caches([FakeTensor((64, 2, 64), torch.float32)], 32)
    assert (h.num_blocks, h.row_bytes) == (2, 512)
    for bad in ([], [FakeTensor((4, 16, 2, 64), BF16), FakeTensor((4, 16, 2, 32), BF16)],
                [FakeTensor((4, 16, 2, 64), BF16), FakeTensor((4, 16, 2, 64), torch.float32)],
                [FakeTensor((4, 8, 2, 64), BF16)], [FakeTensor((60, 2, 64), BF16)], [FakeTensor((0, 16, 2, 64), BF16)],
                [FakeTensor((64, 2), BF16)], [torch.zeros((4, 16, 2, 64))]):
        with pytest.raises(ValueError):
            mvp.kv_caches(bad, 16)
    apart = FakeTensor((4, 16, 2, 64), BF16)
    apart.is_contiguous = lambda: False
    with pytest.raises(ValueError):
        mvp.kv_caches([apart], 16)


def test_the_bindings_refusals(calls):  # noqa: F811
    def extend(refs=T((4,)), bt=T((3, 5)), lens=T((3,)), add=T((3,)), new=T((3,)), missing=T((1,)), ws=T((512,), U8)):
        mvp.kv_extend_paged(_handle(), refs, bt, lens, add, new, missing, ws)

    i64 = torch.int64
    for bad in (dict(refs=T((5,))), dict(refs=T((4,), i64)), dict(bt=T((3,))), dict(bt=T((3, 5), i64)), dict(lens=T((2,))),
                dict(add=T((4,))), dict(new=T((3,), i64)), dict(missing=T((2,))), dict(ws=T((512,), BF16))):
        with pytest.raises(ValueError):
            extend(**bad)
    for refs, bt, lens, parents, out, lens_out in ((T((2, 2)), T((3, 5)), T((3,)), T((2,)), T((2, 5)), T((2,))),
                                                   (T((4,)), T((3, 5)), T((2,)), T((2,)), T((2, 5)), T((2,))),
                                                   (T((4,)), T((3, 5)), T((3,)), T((3,)), T((2, 5)), T((2,))),
                                                   (T((4,)), T((3, 5)), T((3,)), T((2,)), T((2, 5)), T((3,)))):
        with pytest.raises(ValueError):
            mvp.kv_fork_paged(refs, bt, lens, parents, out, lens_out, 16)
    with pytest.raises(ValueError):
        mvp.kv_trim_paged(T((4,)), T((3, 5)), T((3,)), T((4,)), 16)
    with pytest.raises(ValueError):
        mvp.kv_compact_paged(_handle(), T((4,)), T((3, 5)), T((3,)), T((5,)), T((1,)), T((512,), U8))
    assert calls == []


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("seed", range(5))
def test_the_oracles_pool_stays_consistent(seed):
    """Random steps: refs are the holders, no page is given out twice, and each request's tokens stay its own."""
    rng = np.random.RandomState(seed)
    block, blocks, width = 4, 80, 12
    refs, rows, lens = [0] * blocks, [[] for _ in range(6)], [0] * 6
    held = [[None] * block for _ in range(blocks)]  # token written at each place
    tokens, stamp = [[] for _ in range(6)], 0
    for _ in range(60):
        what = rng.randint(5)
        if what <= 1:
            add = rng.randint(0, 7, len(rows)).tolist()
            missing, copies = op.extend(refs, rows, lens, add, block, width)
            for old, new, n in copies:
                held[new][:n] = held[old][:n]
            if missing == 0:
                for b, a in enumerate(add):
                    for j in range(lens[b] - a, lens[b]):
                        held[rows[b][j // block]][j % block] = stamp
                        tokens[b].append(stamp)
                        stamp += 1
        elif what == 2:
            parents = rng.randint(-1, len(rows), rng.randint(1, 9)).tolist()
            rows, lens = op.fork(refs, rows, lens, parents)
            tokens = [list(tokens[p]) if p >= 0 else [] for p in parents]
        elif what == 3:
            keep = [int(rng.randint(0, n + 3)) for n in lens]
            op.trim(refs, rows, lens, keep, block)
            tokens = [t[:k] for t, k in zip(tokens, keep)]
        else:
            _, moves, n = op.compact(refs, rows)
            for src, dst in moves:
                held[dst] = list(held[src])
            assert all((r > 0) == (i < n) for i, r in enumerate(refs))
        count = [0] * blocks
        for row, n in zip(rows, lens):
            assert len(row) == op.pages_of(n, block)
            for page in row:
                count[page] += 1
        assert refs == count
        for row, t in zip(rows, tokens):
            assert [held[row[j // block]][j % block] for j in range(len(t))] == t
