"""A pool's steps and capped, biased attention run together (GPU), as a serving
loop uses them: prompts take pages and are written, samples share them, decode
steps grow the samples (as replays of one graph), beams are picked, drafts are
cut back, requests end, and the pool is compacted, in two layers that go by one
block table.  After every step each sample's keys and values are its own
history bit for bit, and attention over them is the float64 oracle's, with the
tolerances of the single operators' tests."""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from oracle import attention as oatt
from oracle import pages as op
from oracle import scores as osc

from . import gpu_helpers as gh

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCK, WIDTH, BLOCKS, LAYERS = 8, 2, 128, 16, 14, 70, 2
CAP, INV = 20.0, 10000.0 ** (-np.arange(64) / 64)


class Loop:
    def __init__(self, reqs):
        self.dev = torch.device("cuda", torch.cuda.current_device())
        self.gen = torch.Generator(device=self.dev).manual_seed(7)
        shape = (BLOCKS, BLOCK, HKV, D)
        self.caches = [torch.full(shape, float(i), dtype=torch.bfloat16, device=self.dev) for i in range(2 * LAYERS)]
        self.pool = mvp.kv_caches(self.caches, BLOCK)
        self.refs = self.i32([0] * BLOCKS)
        self.missing = self.i32([7])
        self.slopes = torch.tensor(0.5 * 2.0 ** -np.arange(1, HQ + 1), dtype=torch.float32, device=self.dev)
        self.table = mvp.rope_table(INV)
        self.tables(reqs)
        self.lens = self.i32([0] * reqs)
        # the same in lists: holders, pages, lengths, and per request and cache the rows written so far
        self.o_refs, self.rows, self.o_lens = [0] * BLOCKS, [[] for _ in range(reqs)], [0] * reqs
        self.history = [[torch.zeros((0, HKV, D), dtype=torch.bfloat16) for _ in self.caches] for _ in range(reqs)]

    def i32(self, x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=self.dev)

    def tables(self, reqs):
        self.bt = torch.full((reqs, WIDTH), -1, dtype=torch.int32, device=self.dev)

    def inputs(self, add):
        """Fixed arrays for steps of these lengths."""
        self.add_list, n = list(add), sum(add)
        self.add = self.i32(add)
        self.cu = self.i32(np.concatenate([[0], np.cumsum(add)]))
        self.qkv = torch.empty((LAYERS, n, HQ + 2 * HKV, D), dtype=torch.bfloat16, device=self.dev)
        self.pos = torch.empty((1, n), dtype=torch.int32, device=self.dev)
        self.q = torch.empty((LAYERS, n, HQ, D), dtype=torch.bfloat16, device=self.dev)
        self.out, self.lse = torch.empty_like(self.q), torch.empty((LAYERS, HQ, n), device=self.dev)
        size = max(mvp.kv_extend_workspace_size(len(add)), 16)
        self.ws = torch.empty(size, dtype=torch.uint8, device=self.dev)
        size = mvp.attn_workspace_size(len(add), HQ, D, WIDTH * BLOCK)
        self.attn_ws = torch.empty(size, dtype=torch.uint8, device=self.dev)

    def step(self):
        mvp.kv_extend_paged(self.pool, self.refs, self.bt, self.lens, self.add, self.lens, self.missing, self.ws)
        for i in range(LAYERS):
            k, v, x = self.caches[2 * i], self.caches[2 * i + 1], self.qkv[i]
            mvp.rope_append_paged(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.q[i], k, v, self.pos, self.table,
                                  self.cu, self.lens, self.bt, BLOCK)
            mvp.attn_fwd_paged(self.q[i], k, v, self.out[i], self.cu, self.lens, self.bt, BLOCK, max(self.add_list),
                               WIDTH * BLOCK, lse=self.lse[i], softcap=CAP, distance_slopes=self.slopes,
                               workspace=self.attn_ws)

    def fresh(self):
        """New tokens' projections and positions."""
        self.qkv.copy_(2 * torch.randn(self.qkv.shape, generator=self.gen, device=self.dev))
        p = np.concatenate([n + np.arange(a) for n, a in zip(self.o_lens, self.add_list)])
        self.pos.copy_(torch.tensor(p[None]))

    def gathered(self, cache, b):
        ids = torch.tensor(self.rows[b], dtype=torch.long, device=self.dev)
        return cache[ids].reshape(-1, HKV, D)[:self.o_lens[b]].cpu()

    def state(self, what):
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        assert self.refs.tolist() == self.o_refs, what
        assert self.lens.tolist() == self.o_lens, what
        bt = self.bt.cpu().numpy()
        for b, row in enumerate(self.rows):
            assert bt[b, :len(row)].tolist() == row, what

    def check(self, what):
        """After step(): the pool, every request's history, and the attention."""
        missing, _ = op.extend(self.o_refs, self.rows, self.o_lens, self.add_list, BLOCK, WIDTH)
        assert int(self.missing) == missing == 0, what
        self.state(what)
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        cu = self.cu.tolist()
        for b, a in enumerate(self.add_list):
            for i, cache in enumerate(self.caches):
                now = self.gathered(cache, b)
                assert torch.equal(now[:self.o_lens[b] - a], self.history[b][i]), f"{what}: request {b} lost its past"
                self.history[b][i] = now
        for i in range(LAYERS):
            x, out, lse = f64(self.qkv[i]), np.zeros(self.out[i].shape), np.zeros(self.lse[i].shape)
            for b, a in enumerate(self.add_list):
                r, n = slice(cu[b], cu[b + 1]), self.o_lens[b]
                k, v = (h.double().numpy() for h in self.history[b][2 * i:2 * i + 2])
                assert np.array_equal(v[n - a:], x[r, HQ + HKV:]), what
                mask = oatt.visible_mask(np.arange(a), n, n - a, True, -1, 0)
                out[r], lse[:, r] = osc.attend(f64(self.q[i])[r], k, v, n - a + np.arange(a), mask, D ** -0.5, CAP,
                                               self.slopes.cpu().numpy())
            gh.compare(self.out[i], self.lse[i], out, lse, what=what, strict=False)

    def fork(self, parents):
        old, lens = self.bt, self.lens
        self.tables(len(parents))
        self.lens = self.i32([-1] * len(parents))
        mvp.kv_fork_paged(self.refs, old, lens, self.i32(parents), self.bt, self.lens, BLOCK)
        self.rows, self.o_lens = op.fork(self.o_refs, self.rows, self.o_lens, parents)
        self.history = [list(self.history[p]) for p in parents]
        self.state("fork")

    def trim(self, keep):
        mvp.kv_trim_paged(self.refs, self.bt, self.lens, self.i32(keep), BLOCK)
        op.trim(self.o_refs, self.rows, self.o_lens, keep, BLOCK)
        self.history = [[h[:n] for h in hs] for hs, n in zip(self.history, self.o_lens)]
        self.state("trim")

    def compact(self):
        ws = torch.empty(mvp.kv_compact_workspace_size(BLOCKS), dtype=torch.uint8, device=self.dev)
        new, live = torch.empty_like(self.refs), self.i32([0])
        mvp.kv_compact_paged(self.pool, self.refs, self.bt, self.lens, new, live, ws)
        want, _, n = op.compact(self.o_refs, self.rows)
        assert int(live) == n and new.tolist() == want
        self.state("compact")


def test_samples_of_shared_prompts():
    loop = Loop(3)
    loop.inputs([50, 33, 0])
    loop.fresh()
    loop.step()
    loop.check("prompts")
    loop.inputs([0, 40, 16])  # a second chunk, and a prompt of one page
    loop.fresh()
    loop.step()
    loop.check("second chunk")

    loop.fork([0, 0, 0, 1, 1, 2, 2])  # samples; 50 and 73 tokens end inside pages, 16 does not
    loop.inputs([1] * 7)
    loop.fresh()
    loop.step()
    loop.check("first decode step")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    loop.state("capture")  # (captured, not run)
    for i in range(17):  # over a page's end for every sample
        loop.fresh()
        graph.replay()
        loop.check(f"decode step {i}")
        if i == 4:
            loop.trim([55, 60, 56, 75, 79, 0, 22])  # drafts that were rejected, a sample that ends
        if i == 9:
            for c in loop.caches:  # free pages may hold anything
                free = [p for p, r in enumerate(loop.o_refs) if r <= 0]
                c[torch.tensor(free, device=loop.dev)] = float("nan")
            before = [[loop.gathered(c, b) for c in loop.caches] for b in range(7)]
            loop.compact()
            for b in range(7):
                assert all(torch.equal(x, loop.gathered(c, b)) for x, c in zip(before[b], loop.caches))
            for c in loop.caches:
                c[sum(r > 0 for r in loop.o_refs):] = 0.0  # (V behind a sequence must be finite where its page is read)

    loop.fork([4, 4, 1, 6])  # beams: others end
    loop.inputs([1, 2, 1, 30])
    loop.fresh()
    loop.step()
    loop.check("beams")
    loop.trim([0] * 4)
    assert not loop.refs.any()
