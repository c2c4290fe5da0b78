"""The bounded cache's steps run together (GPU), as a serving loop uses them:
rotate and append, attend under a window with first tokens, add up the weights,
evict when a request is over its budget, and go on.  Every step's result is
compared with the float64 oracle on the inputs the step really had (the caches,
lse and weights read back before it), with the tolerances of the single
operators' tests.  The decode steps are replays of one captured graph."""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from oracle import cache as oc

from . import gpu_helpers as gh

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCK, MAX_BLOCKS = 8, 2, 128, 16, 20
BUDGET, FIRST, RECENT, WINDOW = 150, 4, 40, 120
INV = 10000.0 ** (-np.arange(48) / 48)  # 96 of 128 dims rotate
AXES = np.arange(48) % 3


class Loop:
    def __init__(self, reqs):
        self.n, dev = reqs, torch.device("cuda", torch.cuda.current_device())
        self.dev = dev
        rng = np.random.RandomState(3)
        self.bt = torch.tensor(rng.permutation(reqs * MAX_BLOCKS).reshape(reqs, MAX_BLOCKS), dtype=torch.int32, device=dev)
        rows = reqs * MAX_BLOCKS * BLOCK
        self.k = torch.zeros((rows, HKV, D), dtype=torch.bfloat16, device=dev)
        self.v = torch.zeros_like(self.k)
        self.w = torch.zeros((reqs, HKV, MAX_BLOCKS * BLOCK), device=dev)
        self.lens = torch.zeros(reqs, dtype=torch.int32, device=dev)   # keys in the cache
        self.seen = np.zeros(reqs, dtype=np.int64)                     # tokens so far: the positions
        self.table = mvp.rope_table(INV, AXES, num_axes=3)
        self.new_lens = torch.zeros_like(self.lens)
        self.kept = torch.zeros((reqs, HKV, BUDGET), dtype=torch.int32, device=dev)
        self.ev_ws = torch.empty(mvp.kv_evict_workspace_size(reqs, HKV, BUDGET), dtype=torch.uint8, device=dev)
        self.max_k = MAX_BLOCKS * BLOCK
        self.gen = torch.Generator(device=dev).manual_seed(5)

    def inputs(self, q_lens):
        total = sum(q_lens)
        self.qkv = torch.randn((total, HQ + 2 * HKV, D), generator=self.gen, device=self.dev).bfloat16()
        self.q = torch.empty((total, HQ, D), dtype=torch.bfloat16, device=self.dev)
        self.out, self.lse = torch.empty_like(self.q), torch.empty((HQ, total), device=self.dev)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device=self.dev)
        self.pos = torch.zeros((3, total), dtype=torch.int32, device=self.dev)
        ws = max(mvp.attn_workspace_size(self.n, HQ, D, self.max_k),
                 mvp.key_weights_workspace_size(self.n, HKV, max(q_lens), self.max_k), 256)
        self.ws = torch.empty(ws, dtype=torch.uint8, device=self.dev)
        self.q_lens, self.max_q = list(q_lens), max(q_lens)

    def step(self):
        x = self.qkv
        mvp.rope_append_paged(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.q, self.k, self.v, self.pos, self.table,
                              self.cu, self.lens, self.bt, BLOCK)
        kw = dict(window_left=WINDOW, first_tokens=FIRST, workspace=self.ws)
        mvp.attn_fwd_paged(self.q, self.k, self.v, self.out, self.cu, self.lens, self.bt, BLOCK, self.max_q, self.max_k,
                           lse=self.lse, **kw)
        mvp.attn_key_weights_paged(self.q, self.k, self.lse, self.w, self.cu, self.lens, self.bt, BLOCK, self.max_q,
                                   self.max_k, **kw)

    def advance(self):
        """New tokens: positions, and cache lengths that count them."""
        pos, at = np.zeros((3, sum(self.q_lens)), dtype=np.int32), 0
        for b, n in enumerate(self.q_lens):
            t = self.seen[b] + np.arange(n)
            pos[:, at:at + n] = [t, t % 7, t % 11]
            at += n
        self.seen += self.q_lens
        self.pos.copy_(torch.tensor(pos))
        self.lens += torch.tensor(self.q_lens, dtype=torch.int32, device=self.dev)
        self.before = self.k.clone(), self.v.clone(), self.w.clone()

    def rows(self, b, n):
        j = np.arange(n)
        return self.bt[b].cpu().numpy().astype(np.int64)[j // BLOCK] * BLOCK + j % BLOCK

    def check(self, what):
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        x, lens, cu, pos = f64(self.qkv), self.lens.tolist(), self.cu.tolist(), self.pos.cpu().numpy()
        rq, rk = (oc.rotate(x[:, s], pos, INV, AXES, False) for s in (slice(0, HQ), slice(HQ, HQ + HKV)))
        out, lse = np.zeros(rq.shape), np.zeros((HQ, rq.shape[0]))
        w0, w1 = f64(self.before[2]), f64(self.w)
        assert np.abs(f64(self.q) - rq).max() <= 2.0 ** -8 * np.abs(rq).max() + 1e-4
        touched = np.zeros(self.k.shape[0], dtype=bool)
        for b in range(self.n):
            a, e, n = cu[b], cu[b + 1], lens[b]
            rows = self.rows(b, n)
            new = rows[n - (e - a):]
            touched[new] = True
            assert np.abs(f64(self.k)[new] - rk[a:e]).max(initial=0) <= 2.0 ** -8 * np.abs(rk[a:e]).max(initial=0) + 1e-4
            assert np.array_equal(f64(self.v)[new], x[a:e, HQ + HKV:])
            k, v, q = f64(self.k)[rows], f64(self.v)[rows], f64(self.q)[a:e]
            mask = oc.mask_first(e - a, n, n - (e - a), True, WINDOW, 0, FIRST)
            out[a:e], lse[:, a:e] = oc.attend(q, k, v, mask, D ** -0.5)
            add = oc.key_weights(q, k, f64(self.lse)[:, a:e], mask, D ** -0.5)
            # (fp32 sums of at most a few hundred terms, scores of |x| < 30: 1e-4 is above the operator's own bound)
            assert np.allclose(w1[b, :, :n], w0[b, :, :n] + add, rtol=1e-4, atol=1e-30)
            assert np.array_equal(w1[b, :, n:], w0[b, :, n:])
        assert torch.equal(self.k[~touched], self.before[0][~touched]), "other cache rows changed"
        gh.compare(self.out, self.lse, out, lse, what=what, strict=False)

    def evict(self):
        k0, v0, w0, lens = self.k.clone(), self.v.clone(), self.w.cpu().numpy(), self.lens.tolist()
        mvp.kv_evict_paged(self.k, self.v, self.w, self.lens, self.bt, BLOCK, BUDGET, self.new_lens, self.kept, self.ev_ws,
                           self.max_k, first_tokens=FIRST, recent_tokens=RECENT)
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        for b, n in enumerate(lens):
            m = min(n, BUDGET)
            assert int(self.new_lens[b]) == m
            for h in range(HKV):
                keep = oc.evict(w0[b, h], n, BUDGET, FIRST, RECENT)
                src, dst = torch.tensor(self.rows(b, n)[keep]), torch.tensor(self.rows(b, m))
                assert torch.equal(self.k[dst, h], k0[src, h]) and torch.equal(self.v[dst, h], v0[src, h])
                assert np.array_equal(self.w[b, h, :m].cpu().numpy(), w0[b, h, keep])
                assert not self.w[b, h, m:].any()
        self.lens.copy_(self.new_lens)


def test_generation_under_a_budget():
    loop = Loop(3)
    for chunk in ([130, 1, 0], [70, 200, 33]):  # prompts in chunks
        loop.inputs(chunk)
        loop.advance()
        loop.step()
        loop.check(f"chunk {chunk}")
    loop.evict()  # requests 0 and 1 are over the budget
    assert loop.lens.tolist() == [150, 150, 33]
    loop.inputs([1, 1, 1])
    loop.advance()
    loop.step()
    loop.check("first decode step")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    for i in range(4):
        loop.qkv.copy_(torch.randn(loop.qkv.shape, generator=loop.gen, device=loop.dev))
        loop.advance()
        graph.replay()
        loop.check(f"replayed decode step {i}")
        if i == 1:
            loop.evict()
            assert loop.lens.tolist() == [150, 150, 36]
    loop.inputs([25, 1, 40])  # a second prompt on the cut-down caches
    loop.advance()
    loop.step()
    loop.check("second prompt")
