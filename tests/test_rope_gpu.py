"""Rotary positions written into a paged cache (GPU), against the float64
oracle.

Tolerance per element, derived: the fp32 rotation is off by at most 1e-6 of
the pair's length (the turn is exact to 2^-32 and rounded to fp32, an angle
error of pi * 2^-25 < 1e-7; sincospi a few 2^-24; four roundings of products
and sum of at most 2^-24 each), and one rounding to bf16 adds half a step,
2^-8 of the value.  Copied elements of bf16 inputs are equal.
"""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _case(q_lens, k_lens, hq, hkv, d, rot, axes, block, src, adjacent, seed, pos_top=1000, pad=0, fused=True):
    rng = np.random.RandomState(seed)
    dev = torch.device("cuda", torch.cuda.current_device())
    total = sum(q_lens) + pad
    g = torch.Generator(device=dev).manual_seed(seed)
    if fused:
        qkv = torch.randn((total, hq + 2 * hkv, d), generator=g, device=dev, dtype=src)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = (torch.randn((total, h, d), generator=g, device=dev, dtype=src) for h in (hq, hkv, hkv))
    need = [-(-n // block) for n in k_lens]
    blocks = sum(need) + 3
    ids = rng.permutation(blocks)
    bt = np.full((len(k_lens), max(max(need), 1)), -9, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    pairs = rot // 2
    inv = 10000.0 ** (-np.arange(pairs) / pairs)
    ax = rng.randint(0, axes, pairs)
    ax[0] = axes - 1
    pos = rng.randint(-50, pos_top, (axes, total)).astype(np.int32)
    k0 = torch.randn((blocks * block, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
    v0 = torch.randn((blocks * block, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    t32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    return dict(q=q, k=k, v=v, k0=k0, v0=v0, pos=pos, inv=inv, ax=ax, bt=bt, cu=cu, q_lens=q_lens, k_lens=k_lens,
                block=block, adjacent=adjacent, args=(t32(pos), mvp.rope_table(inv, ax, num_axes=axes), t32(cu),
                                                      t32(k_lens), t32(bt), block))


def _run(c, q_out=None, stream=None):
    kc, vc = c["k0"].clone(), c["v0"].clone()
    if q_out is None:
        q_out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device=kc.device)
    mvp.rope_append_paged(c["q"], c["k"], c["v"], q_out, kc, vc, *c["args"], adjacent=c["adjacent"], stream=stream)
    return q_out, kc, vc


def _close(got, ref, src):
    """got within the derived bound of the rotation ref of src (same shape)."""
    pair = np.sqrt((np.asarray(src) ** 2).sum(-1, keepdims=True))  # at least any pair's length
    tol = 2.0 ** -8 * np.abs(ref) + 1e-6 * pair
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"off by {err.max()} where {tol.flat[err.argmax()]} is allowed"


def _check(c, q_out, kc, vc):
    n = int(c["cu"][-1])
    f64 = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    q, k = f64(c["q"])[:n], f64(c["k"])[:n]
    _close(f64(q_out)[:n], oc.rotate(q, c["pos"][:, :n], c["inv"], c["ax"], c["adjacent"]), q)
    assert (f64(q_out)[n:] == 7.0).all(), "rows past the batch were written"
    rk = oc.rotate(k, c["pos"][:, :n], c["inv"], c["ax"], c["adjacent"])
    rows = []
    for b, (ql, kl) in enumerate(zip(c["q_lens"], c["k_lens"])):
        rows += [c["bt"][b, j // c["block"]] * c["block"] + j % c["block"] for j in range(kl - ql, kl)]
    rows = np.array(rows, dtype=np.int64)
    _close(f64(kc)[rows], rk, k)
    assert torch.equal(vc[rows], c["v"][:n].bfloat16())
    rest = np.setdiff1d(np.arange(kc.shape[0]), rows)
    assert torch.equal(kc[rest], c["k0"][rest]) and torch.equal(vc[rest], c["v0"][rest]), "other cache rows changed"


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (256, 256), (256, 64), (512, 512),
                                   (80, 48), (40, 32)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
def test_head_dims(d, rot, adjacent, src):
    c = _case([5, 1, 0, 33], [5, 70, 20, 300], 6, 2, d, rot, 3, 32, src, adjacent, seed=d + rot, pad=3)
    q_out, kc, vc = _run(c)
    torch.cuda.synchronize()
    _check(c, q_out, kc, vc)


@pytest.mark.parametrize("axes,block", [(1, 16), (2, 64), (4, 128), (3, 256)])
def test_axes_and_far_positions(axes, block):
    c = _case([1] * 70 + [130], list(range(1, 71)) + [131], 8, 8, 128, 128, axes, block, torch.bfloat16, False,
              seed=axes, pos_top=2 ** 31 - 1)
    q_out, kc, vc = _run(c)
    torch.cuda.synchronize()
    _check(c, q_out, kc, vc)


def test_one_token_and_one_head():
    c = _case([1], [1], 1, 1, 64, 64, 1, 16, torch.bfloat16, True, seed=9, fused=False)
    _check(c, *_run(c))


def test_many_requests():
    rng = np.random.RandomState(4)
    q = [int(x) for x in rng.randint(0, 4, 1500)]
    c = _case(q, [a + int(x) for a, x in zip(q, rng.randint(0, 40, 1500))], 2, 1, 64, 32, 2, 16, torch.float32, False,
              seed=5)
    _check(c, *_run(c))


def test_queries_in_place():
    c = _case([40, 3], [60, 3], 4, 2, 128, 128, 2, 16, torch.bfloat16, False, seed=11, fused=False)
    before = c["q"].clone()
    q_out, kc, vc = _run(c, q_out=c["q"])
    torch.cuda.synchronize()
    c["q"] = before
    _check(c, q_out, kc, vc)


def test_keys_without_a_row_are_skipped():
    """Ids outside the cache, a key below 0 and a key past the table: the
    queries are rotated, nothing else is written."""
    c = _case([4, 4, 4], [4, 2, 4], 2, 2, 64, 64, 1, 16, torch.bfloat16, False, seed=12)
    pos, table, cu, sl, bt, block = c["args"]
    bt = bt.clone()
    bt[0, 0], bt[2, 0] = -1, 1 << 30
    sl = sl.clone()
    c["args"] = (pos, table, cu, sl, bt, block)
    q_out, kc, vc = _run(c)
    torch.cuda.synchronize()
    n = 12
    q = c["q"].double().cpu().numpy()
    _close(q_out.double().cpu().numpy(), oc.rotate(q, c["pos"], c["inv"], c["ax"], False), q)
    rows = [int(bt[1, 0]) * 16 + j for j in range(2)]  # request 1: keys -2 .. 1
    rest = np.setdiff1d(np.arange(kc.shape[0]), rows)
    assert torch.equal(kc[rest], c["k0"][rest]) and torch.equal(vc[rest], c["v0"][rest])
    assert torch.equal(vc[rows], c["v"][6:8]) and n == 12
    assert mvp.get_last_device_error() == 0


def test_stream_graph_and_checked_build():
    c = _case([17, 64], [90, 64], 4, 2, 128, 64, 3, 16, torch.bfloat16, False, seed=13)
    ref = _run(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _run(c)
    explicit = _run(c, stream=None)
    torch.cuda.synchronize()
    for r, a, b in zip(ref, got, explicit):
        assert torch.equal(r, a) and torch.equal(r, b)
    kc, vc = c["k0"].clone(), c["v0"].clone()
    q_out = torch.zeros_like(ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mvp.rope_append_paged(c["q"], c["k"], c["v"], q_out, kc, vc, *c["args"])
    for _ in range(2):
        q_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, ref[0]) and torch.equal(kc, ref[1]) and torch.equal(vc, ref[2])
    with mvp.bounds_checked():
        dbg = _run(c)
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == mvp.MVP_OK
    for r, a in zip(ref, dbg):
        assert torch.equal(r, a)


@pytest.mark.parametrize("rows", [2500, 5003])
@pytest.mark.parametrize("hq,hkv,d,rot", [(2, 1, 64, 16), (4, 1, 64, 64), (8, 2, 64, 32)])
def test_several_tokens_per_cta(rows, hq, hkv, d, rot):
    """Many small rows: a CTA takes several, of one request or of several, and
    the last CTA fewer."""
    c = _case([rows - 400, 1, 0, 399], [rows, 9, 3, 450], hq, hkv, d, rot, 2, 16, torch.bfloat16, rows % 2 == 1,
              seed=rows + rot, pad=3)
    _check(c, *_run(c))


def test_far_rows_of_a_large_cache():
    """Cache rows past 2^32 bytes."""
    c = _case([70, 1], [300, 20], 2, 8, 128, 64, 2, 256, torch.bfloat16, False, seed=21)
    ref = _run(c)
    blocks = 5 * (1 << 30) // (8 * 128 * 2 * 256)
    shift = blocks - c["k0"].shape[0] // 256
    big = torch.zeros((blocks * 256, 8, 128), dtype=torch.bfloat16, device="cuda")
    big[shift * 256:] = c["k0"]
    vc, q_out = big.clone(), torch.zeros_like(ref[0])
    vc[shift * 256:] = c["v0"]
    pos, table, cu, sl, bt, block = c["args"]
    mvp.rope_append_paged(c["q"], c["k"], c["v"], q_out, big, vc, pos, table, cu, sl, (bt + shift).int(), block)
    torch.cuda.synchronize()
    assert torch.equal(q_out, ref[0]) and torch.equal(big[shift * 256:], ref[1]) and torch.equal(vc[shift * 256:], ref[2])
    assert not big[:shift * 256].any()


def test_caches_of_four_dimensions():
    c = _case([40, 3], [60, 3], 4, 2, 64, 64, 2, 16, torch.bfloat16, False, seed=21)
    ref = _run(c)
    _check(c, *ref)
    shape = (-1, 16, 2, 64)
    kc, vc = c["k0"].clone(), c["v0"].clone()
    q_out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device=kc.device)
    mvp.rope_append_paged(c["q"], c["k"], c["v"], q_out, kc.view(shape), vc.view(shape), *c["args"])
    assert torch.equal(kc, ref[1]) and torch.equal(vc, ref[2])
    both = torch.stack([c["k0"].view(shape), c["v0"].view(shape)], 1)  # K and V of a block next to each other
    with pytest.raises(ValueError):
        mvp.rope_append_paged(c["q"], c["k"], c["v"], q_out, both[:, 0], both[:, 1], *c["args"])


@pytest.mark.parametrize("rows,hq,d,rot", [(50, 40, 256, 64), (50, 64, 128, 128), (4000, 2, 64, 32)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_queries_in_place_of_many_heads(rows, hq, d, rot, adjacent):
    """A thread takes several pieces of a row in turn, some after others of
    that row were written, and (4000 rows) a CTA several rows."""
    c = _case([rows - 3, 3], [rows, 30], hq, 2, d, rot, 2, 16, torch.bfloat16, adjacent, seed=rows + hq, fused=False)
    before = c["q"].clone()
    ref = _run(c)
    q_out, kc, vc = _run(c, q_out=c["q"])
    torch.cuda.synchronize()
    assert torch.equal(q_out, ref[0]) and torch.equal(kc, ref[1]) and torch.equal(vc, ref[2])
    c["q"] = before
    _check(c, q_out, kc, vc)
