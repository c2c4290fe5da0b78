"""The attention weight each key received (GPU) against the float64 oracle.

The tolerance of a key's weight, a sum of positive terms exp(x) with
x = scale q.k - lse, is derived for each case (relative):
  * x is off by the tensor core's fp32 accumulation of D products, at most
    2^-23 (D / 16 + 16) sum |q_d k_d| scale, and by three fp32 roundings of
    values up to |x|, |lse| and the score: 2^-22 of the largest;
  * ex2.approx is off by 2^-22, and each of n additions by 2^-24 of the sum.
"""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import workloads
from oracle import cache as oc

from . import gpu_helpers as gh

pytestmark = pytest.mark.gpu


def _w(q, k, hq, hkv, d, window=-1, causal=True, right=0, sink=0, seed=1):
    return workloads.Workload("weights", seed, q, k, hq, hkv, d, causal, window, right, sink, None)


def _table(w, seed):
    """A range table: ranges that hold their rows and reach keys past them."""
    rng = np.random.RandomState(seed)
    table = np.full((w.total_q, 2), -1, dtype=np.int32)
    cu, _ = w.cu_seqlens()
    for b, (ql, kl) in enumerate(zip(w.q_lens, w.k_lens)):
        p = kl - ql + np.arange(ql)
        at = kl - ql - 5
        while at < kl:
            s, e = at + rng.randint(0, 60), 0
            e = s + rng.randint(2, 300)
            table[cu[b]:cu[b + 1]][(p >= s) & (p <= e)] = (s, e)
            at = e + 2
    return table


class Case:
    def __init__(self, w, first=0, table=None, ctx=None, slots=False):
        self.w, self.first, self.table, self.ctx = w, first, table, ctx
        self.x = gh.make_inputs(w)
        self.dev = self.x[0].device
        q, k, v, sinks = [None if t is None else t.detach().cpu().double().numpy() for t in self.x]
        self.cu_q, self.cu_k = w.cu_seqlens()
        self.lse = np.full((w.num_heads_q, w.total_q), -np.inf, dtype=np.float32)
        self.max_k = max(w.k_lens)
        n = w.num_reqs + (3 if slots else 0)
        rng = np.random.RandomState(w.seed)
        self.slots = rng.permutation(n)[:w.num_reqs].astype(np.int32) if slots else None
        self.w0 = rng.rand(n, w.num_heads_kv, self.max_k + 5).astype(np.float32)
        self.add = np.zeros(self.w0.shape)
        self.rel = 0.0
        g = w.num_heads_q // w.num_heads_kv
        for b in range(w.num_reqs):
            rq, rk = slice(self.cu_q[b], self.cu_q[b + 1]), slice(self.cu_k[b], self.cu_k[b + 1])
            c = w.k_lens[b] - w.q_lens[b] if ctx is None else ctx[b]
            mask = oc.mask_first(w.q_lens[b], w.k_lens[b], c, w.causal, w.window_left, w.window_right, first,
                                 None if table is None else table[rq])
            self.lse[:, rq] = oc.attend(q[rq], k[rk], v[rk], mask, w.scale, sinks, w.sink_mode)[1]
            s = b if self.slots is None else self.slots[b]
            self.add[s, :, :w.k_lens[b]] = oc.key_weights(q[rq], k[rk], self.lse[:, rq], mask, w.scale, sinks, w.sink_mode)
            if w.q_lens[b] and w.k_lens[b]:
                norm = w.scale * np.abs(q[rq]).sum(-1).max() * np.abs(k[rk]).max()  # >= scale sum |q_d k_d|
                big = max(norm, np.abs(self.lse[:, rq][np.isfinite(self.lse[:, rq])]).max(initial=0), 1.0)
                self.rel = max(self.rel, 2.0 ** -23 * (w.head_dim / 16 + 16) * norm + 2.0 ** -22 * big + 2.0 ** -22
                               + 2.0 ** -24 * (w.q_lens[b] * g + 8))

    def t32(self, a):
        return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device=self.dev)

    def run(self, block=0, accumulate=True, ws=True, n_dec=-1, weights=None, k=None, **kw):
        w, (q, k0, v, sinks) = self.w, self.x
        k = k0 if k is None else k
        out = torch.tensor(self.w0, device=self.dev) if weights is None else weights
        lse = torch.tensor(self.lse, device=self.dev)
        size = mvp.key_weights_workspace_size(w.num_reqs, w.num_heads_kv, max(w.q_lens), self.max_k)
        args = dict(slots=self.t32(self.slots), context_lens=self.t32(self.ctx), range_table=self.t32(self.table),
                    causal=w.causal, window_left=w.window_left, window_right=w.window_right, first_tokens=self.first,
                    sinks=sinks, sink_mode=w.sink_mode, scale=w.scale, accumulate=accumulate, num_decode_reqs=n_dec,
                    workspace=torch.empty(size, dtype=torch.uint8, device=self.dev) if ws and size else None, **kw)
        if block:
            kc, _, bt, sl = workloads.to_paged(k, v, w.k_lens, block, seed=w.seed, table_fill=-5)
            mvp.attn_key_weights_paged(q, kc, lse, out, self.t32(self.cu_q), sl, bt, block, max(w.q_lens), self.max_k,
                                       **args)
        else:
            mvp.attn_key_weights_varlen(q, k, lse, out, self.t32(self.cu_q), self.t32(self.cu_k), max(w.q_lens),
                                        self.max_k, **args)
        return out

    def check(self, out, accumulate=True):
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        got = out.double().cpu().numpy()
        for b, n in enumerate(self.w.k_lens):
            s = b if self.slots is None else self.slots[b]
            old = self.w0[s, :, :n].astype(np.float64) if accumulate else 0.0
            ref = self.add[s, :, :n] + old
            tol = self.rel * self.add[s, :, :n] + (2.0 ** -23 * ref if accumulate else 0.0)
            err = np.abs(got[s, :, :n] - ref)
            assert (err <= tol + 1e-30).all(), (b, np.unravel_index((err - tol).argmax(), err.shape), err.max())
            assert np.array_equal(got[s, :, n:], self.w0[s, :, n:]), "entries past the request's keys changed"
        used = range(self.w.num_reqs) if self.slots is None else self.slots
        rest = np.setdiff1d(np.arange(self.w0.shape[0]), used)
        assert np.array_equal(got[rest], self.w0[rest])

    def check_all(self, block, n_dec=-1):
        a = self.run(n_dec=n_dec)
        self.check(a)
        self.check(self.run(accumulate=False, n_dec=n_dec), accumulate=False)
        assert torch.equal(a, self.run(block=block, n_dec=n_dec)), "paged != packed"
        return a


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 8, 8), (128, 6, 2), (256, 4, 2), (512, 4, 1), (128, 16, 1),
                                      (64, 40, 1), (64, 128, 1), (64, 5, 1)])
@pytest.mark.parametrize("window,first", [(-1, 0), (70, 3)])
def test_prefill_heads(d, hq, hkv, window, first):
    w = _w([130, 2, 0, 257], [400, 3, 60, 257], hq, hkv, d, window, sink=2, seed=d + hq)
    Case(w, first).check_all([16, 64, 256][hq % 3])


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 32, 8), (128, 6, 2), (256, 4, 4), (512, 17, 1), (64, 128, 1)])
@pytest.mark.parametrize("window,first", [(-1, 0), (0, 1), (900, 130), (70, 5000)])
def test_single_tokens(d, hq, hkv, window, first):
    w = _w([1] * 6, [1, 127, 128, 2049, 700, 4500], hq, hkv, d, window, sink=1, seed=d + hq)
    a = Case(w, first).check_all([16, 32, 128][hq % 3])
    assert torch.equal(a, Case(w, first).run(n_dec=6))


@pytest.mark.parametrize("d,hq,hkv,q", [(64, 4, 4, [3, 64, 0, 17]), (128, 8, 1, [8, 1, 5, 2]), (256, 12, 4, [21, 20, 1, 0]),
                                        (512, 32, 1, [2, 1, 2, 0]), (64, 6, 2, [22, 3, 1, 1]),
                                        (128, 4, 4, [128, 1, 39, 2]), (512, 8, 2, [24, 2, 0, 1]), (64, 3, 1, [43, 43, 1, 9])])
@pytest.mark.parametrize("window,first,ranges", [(-1, 0, False), (60, 9, False), (900, 0, True), (3, 200, True)])
def test_few_rows(d, hq, hkv, q, window, first, ranges):
    """Up to 128 columns (rows x heads of a KV head; 96 at D = 512) go through the single
    tokens' kernel, and the next size through the other one."""
    w = _w(q, [2300, 64, 40, 900], hq, hkv, d, window, sink=1, seed=d + hq)
    Case(w, first, _table(w, d) if ranges else None).check_all(32, n_dec=0 if ranges else -1)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("q,k", [([130, 300], [400, 301]), ([1, 1], [300, 2])])
def test_key0_sinks_far_apart(d, q, k, monkeypatch):
    """A sink that closes key 0, one that takes nearly all of the weight, and
    small ones, in one tile."""
    inputs = gh.make_inputs

    def far(w):
        x = inputs(w)
        x[3].copy_(torch.tensor([-np.inf, 40.0, -7.5, 0.0]))
        return x

    monkeypatch.setattr(gh, "make_inputs", far)
    Case(_w(q, k, 4, 1, d, -1, sink=1, seed=d)).check_all(16)


@pytest.mark.parametrize("seed", range(12))
def test_random_masks(seed):
    rng = np.random.RandomState(seed)
    n = rng.randint(1, 5)
    q = [int(x) for x in rng.choice([0, 1, 1, 9, 200, 500], n)]
    q[0] = max(q[0], 1)
    k = [a + int(x) for a, x in zip(q, rng.randint(0, 700, n))]
    causal = bool(rng.rand() < 0.7)
    w = _w(q, k, 8, int(rng.choice([1, 2, 8])), int(rng.choice([64, 128, 256])), int(rng.choice([-1, 0, 33, 400])),
           causal, 0 if causal else int(rng.choice([-1, 0, 40])), int(rng.randint(0, 3)), seed=seed)
    table = _table(w, seed) if causal and seed % 2 else None
    c = Case(w, int(rng.choice([0, 1, 64, 200])), table, slots=seed % 3 == 0)
    c.check_all(int(rng.choice([16, 32, 64, 128, 256])))
    c.check(c.run(ws=False))


def test_ranges_reach_far_ahead_and_behind():
    w = _w([900, 700], [1000, 2200], 4, 2, 128, 150, seed=3)
    table = np.full((1600, 2), -1, dtype=np.int32)
    table[0:800] = (90, 950)       # early rows see keys of later tiles
    table[900 + 300:900 + 310] = (1805, 2190)
    Case(w, 2, table).check_all(64)


def test_explicit_contexts_and_rows_that_see_nothing():
    w = _w([3, 1, 200, 1], [40, 300, 250, 600], 4, 2, 128, 9)
    Case(w, 5, ctx=[-2, 5000, 700, -3]).check_all(16)


@pytest.mark.parametrize("q,k", [([700], [700]), ([2000], [2000]), ([1500, 40], [2100, 300])])
def test_rows_shared_by_splits(q, k):
    """Few key blocks: the workspace lets several CTAs share a block's rows."""
    w = _w(q, k, 16, 2, 64, seed=q[0])
    c = Case(w)
    assert mvp.key_weights_workspace_size(len(q), 2, q[0], k[0]) > 0
    a = c.check_all(64)
    b = c.run(ws=False)
    c.check(b)
    assert torch.equal(a, c.run())  # the same in every run


def test_weights_sum_to_the_rows():
    w = _w([333, 1], [800, 900], 8, 2, 128, 200, seed=6)
    c = Case(w, 4)
    out = c.run(accumulate=False).double().cpu().numpy()
    for b in range(2):  # each row and head spreads a weight of 1 (fp32 sums: 1e-4 is far above the bound)
        total = out[b, :, :w.k_lens[b]].sum(1)
        assert np.allclose(total, 4 * w.q_lens[b], rtol=max(1e-5, c.rel))


def test_masked_keys_may_hold_anything():
    w = _w([300, 1], [700, 900], 4, 2, 128, 50, seed=8)
    c = Case(w, 3)
    a = c.run(accumulate=False)
    k = c.x[1].clone()
    k[3:340] = float("nan")          # request 0: keys behind every row's window
    k[700 + 3:700 + 840] = float("inf")
    assert torch.equal(a, c.run(accumulate=False, k=k))


def test_streams_graph_and_checked_build():
    w = _w([150, 1, 600], [800, 3000, 600], 8, 2, 128, 300, sink=1, seed=4)
    c = Case(w, 20, _table(w, 4))
    ref = c.run()
    c.check(ref)
    with mvp.bounds_checked():
        got = c.run(), c.run(block=32)
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == mvp.MVP_OK
    assert torch.equal(ref, got[0]) and torch.equal(ref, got[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    torch.cuda.synchronize()
    assert torch.equal(ref, got)
    q, k, _, sinks = c.x
    lse, cu_q, cu_k, tb = torch.tensor(c.lse, device=c.dev), c.t32(c.cu_q), c.t32(c.cu_k), c.t32(c.table)
    out = torch.tensor(c.w0, device=c.dev)
    ws = torch.empty(max(16, mvp.key_weights_workspace_size(3, 2, 600, 3000)), dtype=torch.uint8, device=c.dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mvp.attn_key_weights_varlen(q, k, lse, out, cu_q, cu_k, 600, 3000, range_table=tb, window_left=300,
                                    first_tokens=20, sinks=sinks, sink_mode=1, scale=w.scale, workspace=ws)
    for _ in range(2):
        out.copy_(torch.tensor(c.w0, device=c.dev))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref, out)


def test_padded_batches():
    """Rows past the last request (a batch padded to a capacity): with total_q
    so large that every request could have several rows, single-token ones are
    the prefill kernel's; whatever the rows hold, nothing changes."""
    w = _w([1, 5, 0, 3], [300, 40, 17, 700], 4, 2, 64, 90, sink=1, seed=12)
    c = Case(w, 3)
    ref = c.run()
    for pad in (1, 30):
        q = torch.full((w.total_q + pad, 4, 64), float("nan"), dtype=torch.bfloat16, device=c.dev)
        q[:w.total_q] = c.x[0]
        lse = torch.full((4, w.total_q + pad), float("nan"), device=c.dev)
        lse[:, :w.total_q] = torch.tensor(c.lse, device=c.dev)
        out = torch.tensor(c.w0, device=c.dev)
        mvp.attn_key_weights_varlen(q, c.x[1], lse, out, c.t32(c.cu_q), c.t32(c.cu_k), 5, c.max_k, window_left=90,
                                    first_tokens=3, sinks=c.x[3], sink_mode=1, scale=w.scale)
        c.check(out)
        if pad == 1:
            assert torch.equal(ref, out)


def test_far_rows_of_a_large_cache():
    """Cache rows past 2^32 bytes: the last blocks of a 5 GB cache."""
    d, hkv, block = 128, 8, 256
    blocks = 5 * (1 << 30) // (d * hkv * 2 * block)
    kc = torch.zeros((blocks * block, hkv, d), dtype=torch.bfloat16, device="cuda")
    w = _w([40, 1], [600, 500], 16, hkv, d, seed=13)
    c = Case(w)
    small, _, bt, sl = workloads.to_paged(c.x[1], c.x[2], w.k_lens, block, seed=3)
    shift = blocks - small.shape[0] // block
    kc[shift * block:] = small
    out = torch.tensor(c.w0, device=c.dev)
    bt = torch.where(bt < 0, bt, bt + shift).int()
    mvp.attn_key_weights_paged(c.x[0], kc, torch.tensor(c.lse, device=c.dev), out, c.t32(c.cu_q), sl, bt, block, 40,
                               c.max_k, scale=w.scale)
    c.check(out)
    # ... evicted there, in place
    new, kept = torch.zeros_like(sl), torch.zeros((2, hkv, 100), dtype=torch.int32, device="cuda")
    ws = torch.empty(mvp.kv_evict_workspace_size(2, hkv, 100), dtype=torch.uint8, device="cuda")
    weights = out.cpu().numpy()
    mvp.kv_evict_paged(kc, kc, out, sl, bt, block, 100, new, kept, ws, c.max_k)
    torch.cuda.synchronize()
    for b in range(2):
        keep = oc.evict(weights[b, 5], w.k_lens[b], 100, 0, 0)
        assert kept[b, 5].tolist() == keep.tolist()
        row = lambda j: (int(bt[b, j // block]) - shift) * block + j % block  # noqa: E731
        src = torch.tensor([row(int(j)) for j in keep], device="cuda")
        dst = torch.tensor([row(j) for j in range(100)], device="cuda") + shift * block
        assert torch.equal(kc[dst, 5], small[src, 5])


def test_refused_in_python():
    c = Case(_w([4], [9], 2, 2, 64))
    for kw in (dict(weights=torch.zeros((1, 2, 8), device="cuda")),):  # rows shorter than max_k_len
        with pytest.raises(mvp.MvpError):
            c.run(**kw)
    for kw in (dict(weights=torch.zeros((1, 3, 9), device="cuda")), dict(weights=torch.zeros((2, 9), device="cuda")),
               dict(weights=torch.zeros((1, 2, 9), dtype=torch.float64, device="cuda"))):
        with pytest.raises(ValueError):
            c.run(**kw)


@pytest.mark.parametrize("q,k", [([1] * 5, [300, 40, 17, 2700, 1]), ([1, 0, 1, 0], [300, 40, 17, 5])])
@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("block", [0, 16])
def test_padded_single_tokens(q, k, accumulate, block):
    """A decode step of fewer requests than its rows have room for."""
    w = _w(q, k, 4, 2, 128, 90, seed=len(q))
    c = Case(w, 3)
    rows = 8
    qp = torch.full((rows, 4, 128), float("nan"), dtype=torch.bfloat16, device=c.dev)
    qp[:w.total_q] = c.x[0]
    lse = torch.full((4, rows), float("nan"), device=c.dev)
    lse[:, :w.total_q] = torch.tensor(c.lse, device=c.dev)
    out = torch.tensor(c.w0, device=c.dev)
    kw = dict(window_left=90, first_tokens=3, scale=w.scale, accumulate=accumulate)
    if block:
        kc, _, bt, sl = workloads.to_paged(c.x[1], c.x[2], k, block, seed=1, table_fill=-5)
        mvp.attn_key_weights_paged(qp, kc, lse, out, c.t32(c.cu_q), sl, bt, block, 1, c.max_k, **kw)
    else:
        mvp.attn_key_weights_varlen(qp, c.x[1], lse, out, c.t32(c.cu_q), c.t32(c.cu_k), 1, c.max_k, **kw)
    assert mvp.last_launch_count() > 0
    c.check(out, accumulate)


def test_caches_of_four_dimensions():
    c = Case(_w([40, 1], [60, 300], 4, 2, 64, seed=5))
    kc, _, bt, sl = workloads.to_paged(c.x[1], c.x[2], c.w.k_lens, 16, seed=2, table_fill=-5)
    lse = torch.tensor(c.lse, device=c.dev)

    def call(cache):
        out = torch.tensor(c.w0, device=c.dev)
        mvp.attn_key_weights_paged(c.x[0], cache, lse, out, c.t32(c.cu_q), sl, bt, 16, 40, c.max_k, scale=c.w.scale)
        return out

    a = call(kc)
    c.check(a)
    blocks = kc.view(-1, 16, 2, 64)
    assert torch.equal(a, call(blocks))
    # K next to V in each block: read from a copy, as the attention call does, on the call's stream
    both = torch.stack([blocks, torch.full_like(blocks, 3.0)], 1)
    assert torch.equal(a, call(both[:, 0]))
    side = torch.cuda.Stream()
    torch.full((2, *kc.shape), 5.0, dtype=torch.bfloat16, device=c.dev)
    out = torch.tensor(c.w0, device=c.dev)
    args = (lse, out, c.t32(c.cu_q), sl, bt, 16, 40, c.max_k)
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # the current stream is busy, the side stream is not
    mvp.attn_key_weights_paged(c.x[0], both[:, 0], *args, scale=c.w.scale, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, out)
    with pytest.raises(ValueError):
        call(kc.view(-1, 32, 2, 64))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q,k", [([1, 1], [1, 40]), ([130, 300], [130, 300]), ([3, 5], [3, 7])])
def test_rows_whose_only_key_a_sink_closes(q, k, d, monkeypatch):
    """A key-0 sink of -inf and a row that sees no other key: its scores are
    all -inf, its lse too, and it gives key 0 nothing."""
    inputs = gh.make_inputs

    def closed(w):
        x = inputs(w)
        x[3].copy_(torch.tensor([-np.inf, 0.5, -np.inf, -1.0]))
        return x

    monkeypatch.setattr(gh, "make_inputs", closed)
    w = _w(q, k, 4, 2, d, sink=1, seed=d)
    c = Case(w)
    assert np.isneginf(c.lse[[0, 2], 0]).all() and np.isfinite(c.add).all()
    c.check_all(16)
    # ... as the attention call leaves it
    lse = torch.empty((4, w.total_q), device=c.dev)
    out = torch.empty_like(c.x[0])
    mvp.attn_fwd_varlen(c.x[0], c.x[1], c.x[2], out, c.t32(c.cu_q), c.t32(c.cu_k), max(q), max(k), lse=lse,
                        sinks=c.x[3], sink_mode=1, scale=w.scale)
    assert torch.isneginf(lse[[0, 2], 0]).all() and (out[0, [0, 2]] == 0).all()
