"""Eviction from a paged cache by accumulated weights (GPU): the kept keys,
the moved K, V and weights are equal to the oracle's, bit for bit."""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _weights(kind, rng, shape):
    if kind == "heavy":
        return np.exp(1.5 * rng.randn(*shape)).astype(np.float32)
    if kind == "ties":
        return rng.randint(0, 3, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, dtype=np.float32)
    if kind == "odd":  # signs, zeros of both signs, infinities, denormals, NaN
        x = rng.choice(np.array([0.0, -0.0, 1e-42, -1e-42, np.inf, -np.inf, np.nan, 1.0, -1.0, 3e38], np.float32), shape)
        return x
    return np.nextafter(np.float32(1), np.float32(2)) ** rng.randint(0, 2, shape).astype(np.float32)  # last bit


class Case:
    def __init__(self, lens, hkv, d, block, budget, first=0, recent=0, kind="heavy", seed=0, out="in", slots=False,
                 stride_extra=3):
        rng = np.random.RandomState(seed)
        dev = torch.device("cuda", torch.cuda.current_device())
        self.lens, self.hkv, self.block, self.budget, self.first, self.recent = lens, hkv, block, budget, first, recent
        need = [-(-n // block) for n in lens]
        need_out = [-(-min(n, budget) // block) for n in lens]
        blocks = sum(need) + sum(need_out) + 2
        ids = rng.permutation(blocks)
        self.bt = np.full((len(lens), max(1, max(need))), -3, dtype=np.int32)
        self.bt_out = np.full((len(lens), max(1, max(need_out))), -3, dtype=np.int32)
        at = 0
        for b in range(len(lens)):
            self.bt[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        for b in range(len(lens)):
            self.bt_out[b, :need_out[b]] = ids[at:at + need_out[b]]
            at += need_out[b]
            if out == "mixed":  # every other block stays where it is
                self.bt_out[b, :need_out[b]:2] = self.bt[b, :need_out[b]:2]
        self.out = out
        g = torch.Generator(device=dev).manual_seed(seed)
        self.k0 = torch.randn((blocks * block, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
        self.v0 = torch.randn((blocks * block, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
        n_slots = len(lens) + (2 if slots else 0)
        self.slots = rng.permutation(n_slots)[:len(lens)].astype(np.int32) if slots else None
        self.w0 = _weights(kind, rng, (n_slots, hkv, max(lens) + stride_extra))
        self.max_k = max(lens)
        self.dev = dev

    def run(self, ws=None, stream=None):
        t32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=self.dev)  # noqa: E731
        k, v, w = self.k0.clone(), self.v0.clone(), torch.tensor(self.w0, device=self.dev)
        w_out = None if self.out == "in" else torch.full_like(w, 5.0)
        new = torch.full((len(self.lens),), -9, dtype=torch.int32, device=self.dev)
        kept = torch.full((len(self.lens), self.hkv, self.budget), -9, dtype=torch.int32, device=self.dev)
        if ws is None:
            n = mvp.kv_evict_workspace_size(len(self.lens), self.hkv, self.budget)
            ws = torch.full((n,), 255, dtype=torch.uint8, device=self.dev)
        mvp.kv_evict_paged(k, v, w, t32(self.lens), t32(self.bt), self.block, self.budget, new, kept, ws, self.max_k,
                           first_tokens=self.first, recent_tokens=self.recent,
                           block_table_out=None if self.out == "in" else t32(self.bt_out), weights_out=w_out,
                           slots=t32(self.slots), stream=stream)
        return k, v, (w if w_out is None else w_out), new, kept

    def check(self, got):
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        k, v, w, new, kept = got
        k_ref, v_ref = self.k0.clone(), self.v0.clone()
        w_ref = self.w0.copy() if self.out == "in" else np.full_like(self.w0, 5.0)
        kept_ref = np.full(tuple(kept.shape), -1, dtype=np.int64)
        row = lambda bt, b, j: bt[b, j // self.block].astype(np.int64) * self.block + j % self.block  # noqa: E731
        for b, n in enumerate(self.lens):
            s = b if self.slots is None else self.slots[b]
            m = min(n, self.budget)
            for h in range(self.hkv):
                keep = oc.evict(self.w0[s, h], n, self.budget, self.first, self.recent)
                kept_ref[b, h, :m] = keep
                src = torch.tensor(row(self.bt, b, keep), device=self.dev)
                dst = torch.tensor(row(self.bt if self.out == "in" else self.bt_out, b, np.arange(m)), device=self.dev)
                k_ref[dst, h], v_ref[dst, h] = self.k0[src, h], self.v0[src, h]
                w_ref[s, h, :m], w_ref[s, h, m:n] = self.w0[s, h, keep], 0
        assert new.tolist() == [min(n, self.budget) for n in self.lens]
        assert np.array_equal(kept.cpu().numpy(), kept_ref)
        assert torch.equal(k.view(torch.int16), k_ref.view(torch.int16))
        assert torch.equal(v.view(torch.int16), v_ref.view(torch.int16))
        assert np.array_equal(w.cpu().numpy().view(np.int32), w_ref.view(np.int32))


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "odd", "last"])
@pytest.mark.parametrize("out", ["in", "new", "mixed"])
def test_weights_of_every_kind(kind, out):
    c = Case([700, 256, 257, 0, 1, 1100], 3, 64, 16, 256, 5, 40, kind, seed=len(kind), out=out, slots=out == "new")
    c.check(c.run())


@pytest.mark.parametrize("d,block", [(16, 16), (64, 256), (80, 32), (128, 64), (256, 16), (512, 128)])
@pytest.mark.parametrize("out", ["in", "new"])
def test_head_dims_and_blocks(d, block, out):
    c = Case([1500, 333, 900], 2, d, block, 333, 4, 100, seed=d, out=out)
    c.check(c.run())


@pytest.mark.parametrize("budget,first,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 64, 0), (64, 0, 64), (65, 32, 32),
                                                 (2047, 0, 0), (2049, 1, 2000)])
def test_budgets(budget, first, recent):
    c = Case([2050, 2048, 70, 2051], 2, 64, 32, budget, first, recent, "ties", seed=budget)
    c.check(c.run())


@pytest.mark.parametrize("n,reqs", [(4095, 1), (8193, 1), (33000, 1), (70001, 1), (20000, 3),
                                    (150001, 1)])
@pytest.mark.parametrize("kind", ["heavy", "ties"])
def test_long_requests_shared_by_clusters(n, reqs, kind):
    c = Case([n - 5 * i for i in range(reqs)], 2, 64, 256, n // 3, 4, 128, kind, seed=n)
    c.check(c.run())


def test_every_other_key_of_a_long_batch_in_place():
    """Each kept key moves, so every segment overwrites rows others read."""
    c = Case([9000] * 6, 4, 128, 64, 4500, 0, 0, seed=3)
    c.w0[:] = 0
    c.w0[:, :, 1::2] = 1
    for _ in range(3):
        c.check(c.run())


def test_workspace_reuse_streams_graph_and_checked_build():
    c = Case([1500, 800], 2, 128, 32, 400, 4, 50, "ties", seed=8)
    ref = c.run()
    c.check(ref)
    ws = torch.zeros(mvp.kv_evict_workspace_size(2, 2, 400), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        c.check(c.run(ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    c.check(got)
    with mvp.bounds_checked():
        c.check(c.run())
    k, v, w = c.k0.clone(), c.v0.clone(), torch.tensor(c.w0, device="cuda")
    lens, bt = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.lens, c.bt))
    new, kept = torch.zeros_like(lens), torch.zeros((2, 2, 400), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mvp.kv_evict_paged(k, v, w, lens, bt, 32, 400, new, kept, ws, 1500, first_tokens=4, recent_tokens=50)
    for _ in range(2):
        k.copy_(c.k0), v.copy_(c.v0), w.copy_(torch.tensor(c.w0, device="cuda"))
        graph.replay()
        c.check((k, v, w, new, kept))


def test_rows_outside_the_cache_are_not_moved():
    c = Case([300], 1, 64, 16, 100, 0, 0, "equal", seed=2, out="new")  # equal weights: keys 0 .. 99 stay
    c.bt[0, 1], c.bt_out[0, 3] = -1, 1 << 29
    k, v, w, new, kept = c.run()
    torch.cuda.synchronize()
    assert mvp.get_last_device_error() == 0
    ref = c.k0.clone()
    for j in range(100):
        if j // 16 not in (1, 3):
            ref[c.bt_out[0, j // 16] * 16 + j % 16] = c.k0[c.bt[0, j // 16] * 16 + j % 16]
    assert torch.equal(k.view(torch.int16), ref.view(torch.int16)) and kept[0, 0].tolist() == list(range(100))


def test_refused_in_python():
    c = Case([300], 1, 64, 16, 100)
    c.max_k = 400  # longer than the table and the weights
    with pytest.raises(mvp.MvpError):
        c.run()
    c = Case([300], 1, 64, 16, 100, 60, 50)
    with pytest.raises(mvp.MvpError):
        c.run()
    with pytest.raises(mvp.MvpError):
        Case([300], 1, 64, 16, 100).run(ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))


def test_caches_of_four_dimensions():
    c = Case([300, 70], 2, 64, 16, 64, 4, 10, seed=9)
    ref = c.run()
    c.check(ref)
    t32 = lambda x: torch.tensor(x, dtype=torch.int32, device=c.dev)  # noqa: E731

    def call(k, v):
        w, new = torch.tensor(c.w0, device=c.dev), t32([0, 0])
        kept = torch.zeros((2, 2, 64), dtype=torch.int32, device=c.dev)
        ws = torch.empty(mvp.kv_evict_workspace_size(2, 2, 64), dtype=torch.uint8, device=c.dev)
        mvp.kv_evict_paged(k, v, w, t32(c.lens), t32(c.bt), 16, 64, new, kept, ws, c.max_k, first_tokens=4,
                           recent_tokens=10)
        return w

    shape = (-1, 16, 2, 64)
    k, v = c.k0.clone(), c.v0.clone()
    assert torch.equal(call(k.view(shape), v.view(shape)), ref[2])
    assert torch.equal(k, ref[0]) and torch.equal(v, ref[1])
    both = torch.stack([c.k0.view(shape), c.v0.view(shape)], 1)  # K and V of a block next to each other
    with pytest.raises(ValueError):
        call(both[:, 0], both[:, 1])
