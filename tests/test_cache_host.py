"""The bounded paged cache's steps without a GPU: the rotary table against
exact arithmetic, the oracle's own pins, and the refusals, which return
before anything is launched."""

from fractions import Fraction

import numpy as np
import pytest

import masked_varlen_prefill_gb300 as mvp
from oracle import cache as oc

A = 1 << 20  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(mvp.library_path()):
        from masked_varlen_prefill_gb300 import _build

        _build.build()
    return mvp.load_library()


# ------------------------------------------------------------------ rotary table
def _turns(inv):
    """inv / (2 pi) as an exact-enough fraction (pi to 60 digits)."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    return Fraction(inv) / (2 * pi)


def test_rope_table_is_the_frequency_in_turns(lib):
    inv = np.concatenate([10000.0 ** (-np.arange(64) / 64), [6.0, -1.0, 1e-9, 0.0, 2.0 ** -60]])
    axes = (np.arange(inv.size) % 3).astype(np.int32)
    table = np.zeros((inv.size, 4), dtype=np.uint32)
    assert lib.mvp_rope_table_pack(inv.ctypes.data, axes.ctypes.data, inv.size, 3, table.ctypes.data) == mvp.MVP_OK
    assert (table[:, 2] == axes).all()
    for f, (lo, hi, _, _) in zip(inv, table.tolist()):
        got = Fraction((hi << 32) | lo, 1 << 64)
        err = (got - _turns(float(f))) % 1
        assert min(err, 1 - err) <= Fraction(1, 1 << 62), f  # a position of 2^31 stays within 2^-31 of a turn
        for pos in (1, -1, 12345, 2 ** 31 - 1, -2 ** 31):
            turn = ((pos * ((hi << 32) | lo)) % (1 << 64)) >> 32
            want = (pos * _turns(float(f))) % 1
            err = (Fraction(turn, 1 << 32) - want) % 1
            assert min(err, 1 - err) <= Fraction(1, 1 << 30)


def test_rope_table_refusals(lib):
    inv = np.ones(4)
    ax = np.array([0, 1, 2, 3], dtype=np.int32)
    out = np.zeros((4, 4), dtype=np.int32)
    f = lib.mvp_rope_table_pack
    assert f(None, None, 4, 1, out.ctypes.data) == mvp.MVP_ERR_ARG
    assert f(inv.ctypes.data, None, 0, 1, out.ctypes.data) == mvp.MVP_ERR_ARG
    assert f(inv.ctypes.data, None, 257, 1, out.ctypes.data) == mvp.MVP_ERR_ARG
    assert f(inv.ctypes.data, ax.ctypes.data, 4, 3, out.ctypes.data) == mvp.MVP_ERR_ARG  # axis 3 of 3
    assert f(inv.ctypes.data, None, 4, 5, out.ctypes.data) == mvp.MVP_ERR_ARG
    for bad in (np.nan, np.inf, 6.5):
        inv[2] = bad
        assert f(inv.ctypes.data, None, 4, 1, out.ctypes.data) == mvp.MVP_ERR_ARG
    with pytest.raises(ValueError):
        mvp.rope_table([])
    with pytest.raises(ValueError):
        mvp.rope_table([1.0, 0.5], axes=[0])


def _rope(lib, **over):
    a = dict(q=A, k=A, v=A, fp32=0, q_out=A, kc=A, vc=A, pos=A, table=A, axes=1, rot=64, adj=0, cu=A, sk=A, bt=A,
             block=16, max_blocks=4, blocks=8, reqs=1, total=4, hq=4, hkv=2, d=128, qs=512, ks=256, vs=256, stream=None)
    a.update(over)
    return lib.mvp_rope_append_paged(*a.values())


def test_rope_refusals(lib):
    for name in ("q", "k", "v", "q_out", "kc", "vc", "pos", "table", "cu", "sk", "bt"):
        assert _rope(lib, **{name: None}) == mvp.MVP_ERR_ARG, name
    for over in (dict(reqs=0), dict(total=-1), dict(hq=0), dict(hkv=0), dict(rot=8), dict(rot=144), dict(axes=0),
                 dict(axes=5), dict(fp32=2), dict(adj=2), dict(block=8), dict(block=48), dict(block=512),
                 dict(blocks=0), dict(max_blocks=0), dict(qs=511), dict(ks=255), dict(vs=0)):
        assert _rope(lib, **over) == mvp.MVP_ERR_ARG, over
    for over in (dict(d=100), dict(d=1024, rot=64), dict(rot=40), dict(q=A + 8), dict(k=A + 2), dict(v=A + 4),
                 dict(q_out=A + 8), dict(kc=A + 8), dict(table=A + 8), dict(qs=516), dict(fp32=1, vs=258)):
        assert _rope(lib, **over) == mvp.MVP_ERR_UNSUPPORTED, over
    assert _rope(lib, total=0) == mvp.MVP_OK


# ------------------------------------------------------------------ the oracle's own pins
def test_oracle_rotation_keeps_lengths_and_composes():
    rng = np.random.RandomState(0)
    x = rng.randn(5, 2, 16)
    inv, axes = np.array([1.0, 0.3, 0.1, 0.01]), [0, 1, 1, 0]
    p1, p2 = rng.randint(-9, 99, (2, 5)), rng.randint(-9, 99, (2, 5))
    for adj in (False, True):
        y = oc.rotate(x, p1, inv, axes, adj)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 8:], x[..., 8:])
        assert np.allclose(oc.rotate(y, p2, inv, axes, adj), oc.rotate(x, p1 + p2, inv, axes, adj))
        assert np.allclose(oc.rotate(y, -p1, inv, axes, adj), x)
    z = oc.rotate(np.eye(8)[:, None, :] * 1.0, np.ones((1, 8), int), [0.5] * 4, [0] * 4, False)[:, 0]
    assert np.isclose(z[0, 0], np.cos(0.5)) and np.isclose(z[0, 4], np.sin(0.5)) and np.isclose(z[4, 0], -np.sin(0.5))


def test_oracle_first_tokens_mask():
    m = oc.mask_first(3, 8, 5, True, 1, 0, 2)  # rows at 5, 6, 7, window of two keys
    assert [list(np.nonzero(r)[0]) for r in m] == [[0, 1, 4, 5], [0, 1, 5, 6], [0, 1, 6, 7]]
    m = oc.mask_first(3, 8, 0, True, 0, 0, 2)  # the causal rule bounds them
    assert [list(np.nonzero(r)[0]) for r in m] == [[0], [0, 1], [0, 1, 2]]
    m = oc.mask_first(2, 6, 0, False, 1, 1, 4)  # and the right window
    assert [list(np.nonzero(r)[0]) for r in m] == [[0, 1], [0, 1, 2]]
    assert oc.mask_first(4, 9, 5, True, -1, 0, 3).sum() == oc.mask_first(4, 9, 5, True, -1, 0, 0).sum()
    rng = np.random.RandomState(1)
    q, k, v = rng.randn(4, 4, 8), rng.randn(9, 2, 8), rng.randn(9, 2, 8)
    from oracle import attention as oatt

    for mode in (0, 1, 2):
        sinks = rng.randn(4)
        a = oc.attend(q, k, v, oc.mask_first(4, 9, 5, True, 3, 0, 0), 0.3, sinks, mode)
        b = oatt.attend_rows(np.arange(4), q, k, v, 5, True, 3, 0, None, sinks, mode, 0.3)
        assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


def test_first_tokens_refusals(lib):
    def call(first, paged, **over):
        a = dict(q=A, k=A, v=A, out=A, lse=None, cu_q=A, cu_k=A)
        if paged:
            a.update(bt=A, block=16, max_blocks=4, blocks=8)
        a.update(ctx=None, reqs=1, total_q=4)
        if not paged:
            a.update(total_k=4)
        a.update(max_q=4, max_k=4, ndec=-1, hq=4, hkv=2, d=128, table=None, covered=None, causal=1, wl=3, wr=0,
                 first=first, sinks=None, mode=0, scale=0.1, ws=None, wsb=0, stream=None)
        a.update(over)
        return (lib.mvp_attn_fwd_paged_first if paged else lib.mvp_attn_fwd_varlen_first)(*a.values())

    for paged in (False, True):
        assert call(-1, paged) == mvp.MVP_ERR_ARG
        assert call(3, paged, d=96) == mvp.MVP_ERR_UNSUPPORTED
        assert call(3, paged, q=None) == mvp.MVP_ERR_ARG
        assert call(3, paged, total_q=0) == mvp.MVP_OK
    assert call(3, True, block=24) == mvp.MVP_ERR_ARG


# ------------------------------------------------------------------ eviction
def test_oracle_evict():
    w = np.array([5, 1, 4, 4, np.nan, 4, 9, 0], dtype=np.float32)
    assert oc.evict(w, 8, 8, 0, 0).tolist() == list(range(8))
    assert oc.evict(w, 8, 3, 0, 0).tolist() == [0, 2, 6]  # of three equal weights the first
    assert oc.evict(w, 8, 4, 2, 1).tolist() == [0, 1, 6, 7]
    assert oc.evict(w, 8, 7, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]  # NaN goes first
    assert oc.evict(w, 6, 3, 1, 2).tolist() == [0, 4, 5]


def test_evict_refusals(lib):
    def call(**over):
        a = dict(k=A, v=A, w=A, w_out=None, slots_n=2, stride=100, slots=None, sk=A, bt=A, bt_out=None, block=16,
                 max_blocks=8, max_out=0, blocks=20, reqs=2, max_k=100, hkv=2, d=64, budget=50, first=4, recent=10,
                 new=A + 64, kept=A, ws=A, wsb=1 << 20, stream=None)
        a.update(over)
        return lib.mvp_kv_evict_paged(*a.values())

    for name in ("k", "v", "w", "sk", "bt", "new", "kept", "ws"):
        assert call(**{name: None}) == mvp.MVP_ERR_ARG, name
    for over in (dict(reqs=-1), dict(hkv=0), dict(max_k=-1), dict(slots_n=-1), dict(budget=0), dict(first=-1),
                 dict(recent=-1), dict(first=41), dict(block=8), dict(block=24), dict(block=512), dict(blocks=0),
                 dict(max_blocks=6), dict(new=A), dict(stride=99), dict(slots_n=1), dict(bt_out=A, max_out=3),
                 dict(first=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert call(**over) == mvp.MVP_ERR_ARG, over
    for over in (dict(d=8), dict(d=100), dict(d=520), dict(budget=(1 << 30) + 1), dict(k=A + 8), dict(v=A + 2), dict(ws=A + 4)):
        assert call(**over) == mvp.MVP_ERR_UNSUPPORTED, over
    assert call(wsb=256) == mvp.MVP_ERR_CAPACITY
    assert call(reqs=0) == mvp.MVP_OK
    assert mvp.kv_evict_workspace_size(2, 3, 65) == 256 + 2 * 3 * 5 * 4
    assert mvp.kv_evict_workspace_size(0, 3, 65) == 0


# ------------------------------------------------------------------ key weights
def test_oracle_key_weights():
    rng = np.random.RandomState(2)
    q, k = rng.randn(5, 4, 8), rng.randn(9, 2, 8)
    mask = oc.mask_first(5, 9, 4, True, 3, 0, 1)
    sinks = rng.randn(4)
    for mode in (0, 1, 2):
        v = np.zeros((9, 2, 9))  # v = one-hot of the key: the output is the row of probabilities
        v[np.arange(9), :, np.arange(9)] = 1
        probs, lse = np.zeros((5, 4, 9)), None
        for h in range(4):
            o, lse = oc.attend(q[..., :], k, v[:, :, :8], mask, 0.4, sinks, mode)
            probs[..., :8] = o
            probs[..., 8] = oc.attend(q, k, v[:, :, 1:], mask, 0.4, sinks, mode)[0][..., 7]
        w = oc.key_weights(q, k, lse, mask, 0.4, sinks, mode)
        assert np.allclose(w[0], probs[:, :2].sum((0, 1))) and np.allclose(w[1], probs[:, 2:].sum((0, 1)))


def test_key_weights_refusals(lib):
    def call(paged, **over):
        a = dict(q=A, k=A, lse=A, w=A, slots_n=1, stride=64, slots=None, acc=1, cu_q=A, cu_k=A)
        if paged:
            a.update(bt=A, block=16, max_blocks=4, blocks=8)
        a.update(ctx=None, reqs=1, total_q=4)
        if not paged:
            a.update(total_k=64)
        a.update(max_q=4, max_k=64, ndec=-1, hq=4, hkv=2, d=128, table=None, covered=None, causal=1, wl=-1, wr=-1,
                 first=0, sinks=None, mode=0, scale=0.1, ws=None, wsb=0, stream=None)
        a.update(over)
        return (lib.mvp_attn_key_weights_paged if paged else lib.mvp_attn_key_weights_varlen)(*a.values())

    for paged in (False, True):
        for name in ("q", "k", "lse", "w", "cu_q", "cu_k") + (("bt",) if paged else ()):
            assert call(paged, **{name: None}) == mvp.MVP_ERR_ARG, name
        for over in (dict(reqs=0), dict(total_q=-1), dict(hq=3), dict(hkv=0), dict(mode=3), dict(mode=1), dict(wl=-2),
                     dict(first=-1), dict(causal=2), dict(acc=2), dict(ndec=2), dict(scale=0.0),
                     dict(scale=float("nan")), dict(stride=63), dict(slots_n=0), dict(max_k=0), dict(max_q=0),
                     dict(total_q=0, acc=0)):
            assert call(paged, **over) == mvp.MVP_ERR_ARG, over
        for over in (dict(d=96), dict(hq=258), dict(scale=1e-31), dict(q=A + 8), dict(k=A + 4), dict(table=A + 4)):
            assert call(paged, **over) == mvp.MVP_ERR_UNSUPPORTED, over
        assert call(paged, total_q=0) == mvp.MVP_OK
    for over in (dict(block=8), dict(block=24), dict(blocks=0), dict(max_blocks=3)):
        assert call(True, **over) == mvp.MVP_ERR_ARG, over
    assert mvp.key_weights_workspace_size(0, 1, 1, 1) == 0
    assert mvp.key_weights_workspace_size(4, 8, 1, 10000) == 0  # single tokens need none


# ------------------------------------------------------------------ caches of four dimensions
def test_caches_are_written_where_they_are():
    """[num_blocks, block_size, Hkv, D] caches are viewed as rows, never
    copied: what a call writes there would be lost with the copy."""
    import torch

    from masked_varlen_prefill_gb300._cache import _caches

    k, v = torch.zeros(4, 16, 2, 64), torch.zeros(4, 16, 2, 64)
    a, b, blocks = _caches(k, v, 16)
    assert blocks == 4 and a.shape == (64, 2, 64)
    assert a.data_ptr() == k.data_ptr() and b.data_ptr() == v.data_ptr()
    both = torch.zeros(4, 2, 16, 2, 64)  # K and V of a block next to each other
    for pair in ((both[:, 0], both[:, 1]), (k, both[:, 1]), (both[:, 0], v), (k.transpose(1, 2), v.transpose(1, 2))):
        with pytest.raises(ValueError):
            _caches(*pair, 16)
    two = torch.zeros(2, 4, 16, 2, 64)  # one tensor, K and V apart
    a, b, _ = _caches(two[0], two[1], 16)
    assert a.data_ptr() == two.data_ptr() and b.data_ptr() == two[1].data_ptr()


def test_block_size_of_a_cache_of_four_dimensions():
    import torch

    from masked_varlen_prefill_gb300._cache import _caches

    k = torch.zeros(4, 32, 2, 64)
    for block in (16, 64, 0):
        with pytest.raises(ValueError):
            _caches(k, k, block)
    assert _caches(k, k, 32)[2] == 4
