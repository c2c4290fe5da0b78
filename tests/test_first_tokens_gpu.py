"""Attention under a sliding window that leaves the first tokens visible
(GPU), packed and paged, against the float64 oracle, with the tolerances of
the other attention tests (``gpu_helpers.compare``: 1e-2 or two bf16 half
steps of the value, lse 1e-3 relative)."""

import sys

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import workloads
from oracle import cache as oc

from . import gpu_helpers as gh

pytestmark = pytest.mark.gpu


def _ws(w, n_dec=-1):
    n = mvp.attn_workspace_size(w.num_reqs if n_dec < 0 else n_dec, w.num_heads_q, w.head_dim, max(w.k_lens))
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _packed(w, x, first, table=None, ctx=None, n_dec=-1, ws=True, want_lse=True, **kw):
    q, k, v, sinks = x
    cu_q, cu_k = gh.device_meta(w, q.device)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((w.num_heads_q, w.total_q), float("nan"), device=q.device) if want_lse else None
    mvp.attn_fwd_varlen(q, k, v, out, cu_q, cu_k, max(w.q_lens), max(w.k_lens), lse=lse, context_lens=ctx,
                        range_table=table, causal=w.causal, window_left=w.window_left, window_right=w.window_right,
                        sinks=sinks, sink_mode=w.sink_mode, scale=w.scale, workspace=_ws(w, n_dec) if ws else None,
                        num_decode_reqs=n_dec, first_tokens=first, **kw)
    torch.cuda.synchronize()
    assert mvp.get_last_device_error() == 0
    return out, lse


def _paged(w, x, first, block, table=None, ctx=None, n_dec=-1, ws=True):
    q, k, v, sinks = x
    kc, vc, bt, sl = workloads.to_paged(k, v, w.k_lens, block, seed=w.seed, table_fill=-5)
    cu_q, _ = gh.device_meta(w, q.device)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((w.num_heads_q, w.total_q), float("nan"), device=q.device)
    mvp.attn_fwd_paged(q, kc, vc, out, cu_q, sl, bt, block, max(w.q_lens), max(w.k_lens), lse=lse, context_lens=ctx,
                       range_table=table, causal=w.causal, window_left=w.window_left, window_right=w.window_right,
                       sinks=sinks, sink_mode=w.sink_mode, scale=w.scale, workspace=_ws(w, n_dec) if ws else None,
                       num_decode_reqs=n_dec, first_tokens=first)
    torch.cuda.synchronize()
    assert mvp.get_last_device_error() == 0
    return out, lse


def _oracle(w, x, first, table=None, ctx=None):
    q, k, v, sinks = [None if t is None else t.detach().cpu().double().numpy() for t in x]
    cu_q, cu_k = w.cu_seqlens()
    out, lse = np.zeros(q.shape), np.full((w.num_heads_q, w.total_q), -np.inf)
    for b in range(w.num_reqs):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        c = w.k_lens[b] - w.q_lens[b] if ctx is None else ctx[b]
        mask = oc.mask_first(w.q_lens[b], w.k_lens[b], c, w.causal, w.window_left, w.window_right, first,
                             None if table is None else table[rq])
        out[rq], lse[:, rq] = oc.attend(q[rq], k[rk], v[rk], mask, w.scale, sinks, w.sink_mode)
    return out, lse


def _same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def _check(w, first, block, table=None, ctx=None, n_dec=-1, ws=True):
    """packed against the oracle, paged against packed bit for bit."""
    x = gh.make_inputs(w)
    t = None if table is None else torch.from_numpy(table).to(x[0].device)
    c = None if ctx is None else torch.tensor(ctx, dtype=torch.int32, device=x[0].device)
    a = _packed(w, x, first, t, c, n_dec, ws)
    ref = _oracle(w, x, first, table, ctx)
    gh.compare(*a, *ref, what=f"first={first}", strict=False)
    assert _same(a, _paged(w, x, first, block, t, c, n_dec, ws)), "paged != packed"
    return x, a


def _w(q, k, hq, hkv, d, window, causal=True, right=0, sink=0, ranges=None, seed=1):
    return workloads.Workload("first", seed, q, k, hq, hkv, d, causal, window, right, sink, ranges)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("first", [1, 4, 130, 700])
def test_prefill_head_dims(d, first):
    w = _w([300, 2, 0, 129], [1500, 900, 5, 129], 4, 2, d, 99, sink=2, seed=d + first)
    _check(w, first, [16, 64, 256][first % 3])


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 1), (128, 8, 2), (128, 6, 2), (256, 4, 4), (512, 6, 1), (128, 16, 1)])
@pytest.mark.parametrize("first,window", [(1, 0), (5, 300), (64, 64), (1000, 17), (5000, 2000)])
def test_decode(d, hq, hkv, first, window):
    w = _w([1] * 5, [1, 64, 333, 2049, 9001], hq, hkv, d, window, sink=first % 3, seed=d + first)
    _check(w, first, 32)
    x, a = _check(w, first, 128, ws=False)
    b = _packed(w, x, first, n_dec=5)
    gh.compare(*b, a[0].double().cpu().numpy(), a[1].double().cpu().numpy(), what="split", strict=False)


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 1), (128, 8, 2), (256, 4, 2), (512, 2, 1)])
@pytest.mark.parametrize("first,window", [(4, 1000), (300, 3000), (9000, 5)])
def test_few_rows_in_many_parts(d, hq, hkv, first, window, monkeypatch):
    """A workspace with room for 30 parts of a row, more than keys per 4096."""
    monkeypatch.setattr(sys.modules[__name__], "_ws", lambda w, n_dec=-1: torch.empty(
        mvp.attn_workspace_size(w.num_reqs, hq, d, 30 * 4096), dtype=torch.uint8, device="cuda"))
    _check(_w([1] * 3, [9001, 700, 1], hq, hkv, d, window, sink=first % 3, seed=d + first), first, 64)


@pytest.mark.parametrize("seed", range(10))
def test_random_masks(seed):
    rng = np.random.RandomState(seed)
    n = rng.randint(1, 5)
    q = [int(x) for x in rng.choice([1, 1, 7, 150, 400], n)]
    k = [a + int(x) for a, x in zip(q, rng.randint(0, 900, n))]
    causal = bool(rng.rand() < 0.7)
    w = _w(q, k, 8, int(rng.choice([1, 2, 8])), int(rng.choice([64, 128, 256])), int(rng.randint(0, 500)), causal,
           0 if causal else int(rng.choice([-1, 0, 40])), int(rng.randint(0, 3)), seed=seed)
    table = None
    if causal and seed % 2:
        table = np.full((w.total_q, 2), -1, dtype=np.int32)
        cu, _ = w.cu_seqlens()
        for b in range(n):  # a range that holds each of its rows, some keys past them
            p = k[b] - q[b] + np.arange(q[b])
            s, e = int(p[0]) + q[b] // 3, int(p[0]) + q[b] // 3 + 200
            table[cu[b]:cu[b + 1]][(p >= s) & (p <= e)] = (s, e)
    _check(w, int(rng.choice([1, 3, 64, 128, 129, 600])), int(rng.choice([16, 32, 64, 128, 256])), table)


def test_only_first_tokens_are_visible():
    """Positions far past the keys: the window holds no key of the request,
    the first tokens are all the row sees; and a request that sees nothing
    because the causal rule bounds the first tokens too."""
    w = _w([3, 1, 2, 1], [40, 200, 6, 300], 4, 2, 128, 5, sink=0)
    for first in (1, 33, 150):
        _check(w, first, 16, ctx=[500, 5000, -4, -2])  # requests 2 and 3: positions below 0
    w = _w([3, 1], [40, 200], 4, 2, 64, 5, sink=2)
    _check(w, 7, 16, ctx=[500, 5000])


def test_nothing_to_add_is_the_plain_call():
    w = _w([200, 1, 64], [900, 700, 64], 8, 2, 128, 100, sink=1)
    x = gh.make_inputs(w)
    plain = _packed(w, x, 0)
    assert not torch.equal(plain[0], _packed(w, x, 1)[0])
    wide = _w([200, 1, 64], [900, 700, 64], 8, 2, 128, -1, sink=1)
    assert _same(_packed(wide, x, 0), _packed(wide, x, 9))
    # a window that reaches key 0 from every row: the same visible keys
    covers = _w([200, 1, 64], [900, 700, 64], 8, 2, 128, 1000, sink=1)
    a, b = _packed(covers, x, 0), _packed(covers, x, 9)
    gh.compare(*b, a[0].double().cpu().numpy(), a[1].double().cpu().numpy(), strict=False)


def test_without_lse_and_side_by_side():
    """No LSE buffer gives the same output; decode rows beside prefill rows."""
    w = _w([1] * 40 + [500, 300], [3000 + 37 * i for i in range(40)] + [2500, 300], 16, 4, 128, 256, sink=2)
    x, a = _check(w, 20, 64, n_dec=40)
    assert torch.equal(_packed(w, x, 20, want_lse=False, n_dec=40)[0], a[0])
    assert torch.equal(_packed(w, x, 20, want_lse=False)[0][40:], a[0][40:])


def test_masked_keys_may_hold_anything():
    """NaN and infinite keys (and huge values) between the first tokens' tile
    and the window's are never read; NaN keys inside a visited tile are
    masked."""
    w = _w([1, 130], [3000, 2600], 4, 2, 128, 200)
    x = gh.make_inputs(w)
    a = _packed(w, x, 4)
    q, k, v, s = x
    _, cu_k = w.cu_seqlens()
    k, v = k.clone(), v.clone()
    for b, lo in ((0, 2799), (1, 2470 - 200)):
        k0 = int(cu_k[b])
        k[k0 + 4:k0 + lo] = float("nan")
        k[k0 + 600:k0 + 700] = float("inf")
        v[k0 + 128:k0 + lo // 128 * 128] = float("nan")
    assert _same(a, _packed(w, (q, k, v, s), 4))


def test_captured_and_bounds_checked():
    w = _w([150, 1, 1, 40], [800, 900, 4200, 40], 8, 4, 256, 77, sink=1)
    x = gh.make_inputs(w)
    ref = _packed(w, x, 30)
    with mvp.bounds_checked():
        assert _same(ref, _packed(w, x, 30)) and _same(ref, _paged(w, x, 30, 16))
    q, k, v, sinks = x
    cu_q, cu_k = gh.device_meta(w, q.device)
    out, lse, ws = torch.zeros_like(q), torch.zeros((8, w.total_q), device=q.device), _ws(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mvp.attn_fwd_varlen(q, k, v, out, cu_q, cu_k, 150, 4200, lse=lse, window_left=77, sinks=sinks, sink_mode=1,
                            scale=w.scale, workspace=ws, first_tokens=30)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(ref, (out, lse))


def test_refused_combinations():
    w = _w([4], [9], 2, 2, 64, 3)
    x = gh.make_inputs(w)
    with pytest.raises(ValueError):
        _packed(w, x, 2, wait_limit_us=5)
    with pytest.raises(mvp.MvpError):
        _packed(w, x, -1)
    with pytest.raises(mvp.MvpError):
        _paged(w, x, -1, 16)
