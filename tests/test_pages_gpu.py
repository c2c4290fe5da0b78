"""The pages of a pool, taken, shared, freed and compacted (GPU): refs, tables,
lengths and what the caches hold are equal to the oracle's, bit for bit."""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from oracle import pages as op

pytestmark = pytest.mark.gpu


class Pool:
    """A pool on the device, and the same in lists."""

    def __init__(self, lens, blocks, block, width, hkv=2, d=64, caches=2, dtype=torch.bfloat16, seed=0, share=0.0,
                 odd=False):
        rng = np.random.RandomState(seed)
        self.block, self.blocks, self.width = block, blocks, width
        self.lens = list(lens)
        ids = iter(rng.permutation(blocks).tolist())
        self.refs, self.rows = [0] * blocks, []
        for n in lens:
            m = op.pages_of(n, block)
            row = [next(ids) for _ in range(m)]
            if self.rows and rng.rand() < share:  # a common beginning with another request
                other = self.rows[rng.randint(len(self.rows))]
                c = min(len(other), m)
                row[:c] = other[:c]
            self.rows.append(row)
        for row in self.rows:
            for page in row:
                self.refs[page] += 1
        self.dev = torch.device("cuda", torch.cuda.current_device())
        bt = np.full((len(lens), width), -7, dtype=np.int32)
        for b, row in enumerate(self.rows):
            bt[b, :len(row)] = row
        # (odd: refs at an address that is not a multiple of 16)
        self.d_refs = torch.zeros(blocks + 1, dtype=torch.int32, device=self.dev)[1:] if odd else \
            torch.zeros(blocks, dtype=torch.int32, device=self.dev)
        self.d_refs.copy_(torch.tensor(self.refs))
        self.d_bt, self.d_lens = self.t32(bt), self.t32(self.lens)
        g = torch.Generator(device=self.dev).manual_seed(seed)
        size = (blocks, block, hkv, d)
        self.caches = [torch.randint(-100, 100, size, generator=g, device=self.dev).to(dtype) for _ in range(caches)]
        self.want = [c.clone() for c in self.caches]
        self.handle = mvp.kv_caches(self.caches, block)

    def t32(self, x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=self.dev)

    def extend(self, add, in_place=True, stream=None):
        n = len(self.lens)
        ws = torch.full((mvp.kv_extend_workspace_size(n),), 255, dtype=torch.uint8, device=self.dev)
        new = self.d_lens if in_place else torch.full_like(self.d_lens, -9)
        missing = torch.full((1,), 77, dtype=torch.int32, device=self.dev)
        mvp.kv_extend_paged(self.handle, self.d_refs, self.d_bt, self.d_lens, self.t32(add), new, missing, ws, stream=stream)
        if not in_place:
            assert self.d_lens.tolist() == self.lens
        self.d_lens = new
        want, copies = op.extend(self.refs, self.rows, self.lens, add, self.block, self.width)
        for old, page, rows in copies:
            for c in self.want:
                c[page, :rows] = c[old, :rows]
        assert int(missing) == want
        self.check()
        return want

    def trim(self, keep):
        mvp.kv_trim_paged(self.d_refs, self.d_bt, self.d_lens, self.t32(keep), self.block)
        op.trim(self.refs, self.rows, self.lens, keep, self.block)
        self.check()

    def fork(self, parents, width=None):
        bt = torch.full((len(parents), width or self.width), -3, dtype=torch.int32, device=self.dev)
        lens = torch.full((len(parents),), -4, dtype=torch.int32, device=self.dev)
        mvp.kv_fork_paged(self.d_refs, self.d_bt, self.d_lens, self.t32(parents), bt, lens, self.block)
        self.rows, self.lens = op.fork(self.refs, self.rows, self.lens, parents)
        self.d_bt, self.d_lens, self.width = bt, lens, width or self.width
        self.check()
        for b, row in enumerate(self.rows):
            assert (bt[b, len(row):] == -3).all()

    def compact(self):
        ws = torch.full((mvp.kv_compact_workspace_size(self.blocks),), 255, dtype=torch.uint8, device=self.dev)
        new = torch.full((self.blocks,), -9, dtype=torch.int32, device=self.dev)
        live = torch.full((1,), -9, dtype=torch.int32, device=self.dev)
        mvp.kv_compact_paged(self.handle, self.d_refs, self.d_bt, self.d_lens, new, live, ws)
        want, moves, n = op.compact(self.refs, self.rows)
        if moves:
            src, dst = (torch.tensor(x, device=self.dev) for x in zip(*moves))
            for c in self.want:
                c[dst] = c[src]
        assert int(live) == n and new.tolist() == want
        self.check()

    def check(self):
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        assert self.d_lens.tolist() == self.lens
        assert self.d_refs.tolist() == self.refs
        bt = self.d_bt.cpu().numpy()
        for b, row in enumerate(self.rows):
            assert bt[b, :len(row)].tolist() == row, f"request {b}"
        for c, w in zip(self.caches, self.want):
            assert torch.equal(c.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("block", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("seed", range(3))
def test_extend(block, seed):
    rng = np.random.RandomState(seed)
    lens = rng.randint(0, 5 * block, 40).tolist() + [0, block, block - 1, 4 * block]
    pool = Pool(lens, 700, block, 12, seed=seed, share=0.5, odd=seed == 1)
    for step in range(4):
        add = rng.choice([0, 0, 1, 1, 2, block - 1, block, block + 1], len(lens)).tolist()
        assert pool.extend(add, in_place=step % 2 == 0) == 0


def test_extend_of_shared_last_pages():
    """All holders of a page append in one call; some; one; its only holder."""
    pool = Pool([40, 40, 70], 60, 16, 8, seed=1)
    pool.fork([0, 0, 0, 2, 1, 2, 2])
    assert pool.extend([1, 3, 0, 20, 1, 0, 5]) == 0
    assert pool.extend([1, 1, 1, 1, 1, 1, 1]) == 0
    pool = Pool([40, 33], 60, 16, 8, seed=2)
    pool.fork([0, 0, 0, 1])
    old = pool.rows[0][2]
    assert pool.extend([1, 1, 1, 1]) == 0  # three copies, and the old page is free
    assert pool.refs[old] == 0
    assert pool.extend([16, 16, 16, 0]) == 0  # and taken again


def test_extend_takes_the_last_page_and_no_more():
    pool = Pool([16, 16, 16], 6, 16, 4, seed=3)
    assert pool.extend([16, 16, 17]) == 1  # four pages wanted, three there
    assert pool.extend([16, 16, 16]) == 0
    assert pool.extend([1, 0, 0]) == 1
    assert pool.extend([0, 0, 0]) == 0
    pool.trim([0, 32, 3])
    assert pool.extend([0, 1, 13]) == 0


def test_extend_refuses_lengths_the_table_cannot_hold():
    pool = Pool([16, 5], 40, 16, 3, seed=4)
    assert pool.extend([33, 1]) == -1
    assert pool.extend([32, -1]) == -1
    assert pool.extend([2 ** 31 - 1, 0]) == -1
    assert pool.extend([32, 43]) == 0


@pytest.mark.parametrize("reqs,blocks", [(1, 1), (1, 5000), (1023, 9000), (1025, 20000), (3000, 70001), (7, 262144)])
def test_extend_of_every_size(reqs, blocks):
    """More requests than the planning CTA has threads; pools of one CTA's part and of eight's."""
    rng = np.random.RandomState(reqs)
    lens = rng.randint(0, 60, reqs).tolist() if reqs > 1 else [0]
    pool = Pool(lens, blocks, 16, 8, hkv=1, d=8, caches=1, seed=reqs, share=0.3, odd=blocks == 70001)
    assert pool.extend(rng.randint(0, 40, reqs).tolist() if blocks > 1 else [16]) == 0
    if blocks > 1:
        assert pool.extend([1] * reqs) == 0


def test_extend_starts_past_full_parts():
    """The free pages are in the last part of the pool, or spread one to a part."""
    for free in ([39990, 39991, 39999], [5, 8000, 16000, 25000, 39000]):
        pool = Pool([0] * len(free), 40000, 16, 3, hkv=1, d=8, caches=1)
        pool.refs = [1] * 40000
        for i in free:
            pool.refs[i] = 0
        pool.d_refs.copy_(torch.tensor(pool.refs))
        assert pool.extend([1] * (len(free) - 1) + [17]) == 1
        assert pool.extend([1] * len(free)) == 0
        assert [row[0] for row in pool.rows] == free


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn])
def test_caches_of_any_type(dtype):
    pool = Pool([20, 20], 30, 16, 6, hkv=3, d=48, caches=3, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype)
    if dtype == torch.float8_e4m3fn:
        pool.caches = [c.to(dtype) for c in pool.caches]
        pool.want = [c.clone() for c in pool.caches]
        pool.handle = mvp.kv_caches(pool.caches, 16)
        pool.want = [w.view(torch.uint8) for w in pool.want]
        pool.caches = [c.view(torch.uint8) for c in pool.caches]
    pool.fork([0, 0, 1, 1])
    assert pool.extend([1, 1, 1, 0]) == 0
    pool.trim([0, 21, 0, 20])
    pool.compact()


def test_many_caches():
    pool = Pool([40, 70, 9], 64, 32, 6, hkv=2, d=512, caches=256, seed=5)
    pool.fork([0, 1, 1, 2, 0])
    assert pool.extend([1] * 5) == 0
    pool.trim([0, 0, 71, 10, 41])
    pool.compact()


@pytest.mark.parametrize("seed", range(4))
def test_fork(seed):
    rng = np.random.RandomState(seed)
    n = [1, 6, 40, 300][seed]
    pool = Pool(rng.randint(0, 200, n).tolist(), 16 * n + 3, 16, 14, hkv=1, d=8, caches=1, seed=seed, share=0.4)
    pool.fork(rng.randint(-2, n + 2, rng.randint(1, 2 * n + 1)).tolist())  # some of no parent
    pool.fork(list(range(len(pool.rows)))[::-1], width=20)  # in another order, into a wider table
    pool.fork([0] * 33)
    pool.fork([-1] * 5)
    assert not any(pool.refs)


def test_fork_to_and_from_nothing():
    pool = Pool([33, 20], 20, 16, 4)
    before = pool.d_refs.clone()
    none = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    no_lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    mvp.kv_fork_paged(pool.d_refs, pool.d_bt, pool.d_lens, no_lens, none, no_lens, 16)  # everything ends
    assert not pool.d_refs.any()
    pool.d_refs.copy_(before)
    out, lens = torch.full((2, 4), 5, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    mvp.kv_fork_paged(pool.d_refs, none, no_lens, pool.t32([0, 1]), out, lens, 16)  # nothing to continue
    assert lens.tolist() == [0, 0] and (out == 5).all() and torch.equal(pool.d_refs, before)


def test_trim():
    pool = Pool([100, 64, 16, 1, 0, 90], 60, 16, 7, seed=6, share=0.6)
    pool.trim([100, 65, 15, 0, 0, 33])
    pool.trim([-1, 0, 16, 3, 5, 32])
    pool.trim([0] * 6)
    assert not any(pool.refs)


def test_ids_outside_the_pool_are_left_out():
    """Table entries that name no page: held by nobody, never read or written as pages."""
    pool = Pool([40, 40], 20, 16, 6)
    pool.rows[0][1], pool.rows[1][2] = -5, 1000
    pool.refs = [0] * 20
    for row in pool.rows:
        for page in row:
            if 0 <= page < 20:
                pool.refs[page] += 1
    pool.d_refs.copy_(torch.tensor(pool.refs))
    pool.d_bt[0, 1], pool.d_bt[1, 2] = -5, 1000
    assert pool.extend([1, 1]) == 0
    pool.fork([0, 1, 1])
    pool.compact()
    pool.trim([0, 3, 0])


@pytest.mark.parametrize("blocks,block,hkv,d", [(1, 16, 1, 8), (37, 256, 2, 128), (4097, 16, 1, 16), (33333, 16, 1, 8)])
@pytest.mark.parametrize("share", [0.0, 0.02, 0.5, 0.97, 1.0])
def test_compact(blocks, block, hkv, d, share):
    """Pools from empty to full, scattered; holders outside the tables."""
    rng = np.random.RandomState(blocks)
    total = int(share * blocks)
    lens, left = [], total
    while left > 0:
        m = min(left, rng.randint(1, 30))
        lens.append(m * block - rng.randint(0, block))
        left -= m
    pool = Pool(lens or [0], blocks, block, 30, hkv=hkv, d=d, seed=blocks)
    held = rng.permutation(total)[:total // 5]  # a prefix cache holds some pages too, and some alone
    for page in held:
        pool.refs[page] += 1
    pool.d_refs.copy_(torch.tensor(pool.refs))
    pool.compact()
    pool.compact()  # nothing left to do
    pool.trim([0] * len(pool.lens))
    pool.compact()


def test_compact_without_requests():
    pool = Pool([50, 20], 40, 16, 4, seed=8)
    pool.trim([0, 0])
    pool.refs[31], pool.refs[7], pool.refs[39] = 2, 1, 5
    pool.d_refs.copy_(torch.tensor(pool.refs))
    pool.d_bt, pool.d_lens = pool.d_bt[:0], pool.d_lens[:0]
    pool.rows, pool.lens = [], []
    pool.compact()  # 7 and 31 and 39 are live: they become 0, 1 and 2
    assert pool.refs[:4] == [1, 2, 5, 0]


def test_negative_refs_are_free():
    pool = Pool([20], 12, 16, 4)
    free = pool.refs.index(0)
    pool.refs[free] = -3
    pool.d_refs.copy_(torch.tensor(pool.refs))
    assert pool.extend([16]) == 0
    assert pool.refs[free] == 1
    last = max(i for i, r in enumerate(pool.refs) if r == 0)
    pool.refs[last] = -1
    pool.d_refs.copy_(torch.tensor(pool.refs))
    pool.compact()


def test_a_captured_step_replays():
    """Extend in a graph: every replay grows the same arrays."""
    pool = Pool([15, 3, 40], 60, 16, 12, seed=9)
    pool.fork([0, 0, 1, 2, 2])
    add, missing = pool.t32([1, 2, 0, 16, 1]), torch.zeros(1, dtype=torch.int32, device=pool.dev)
    ws = torch.empty(mvp.kv_extend_workspace_size(5), dtype=torch.uint8, device=pool.dev)
    graph = torch.cuda.CUDAGraph()
    state = pool.d_refs.clone(), pool.d_bt.clone(), pool.d_lens.clone()
    with torch.cuda.graph(graph):
        mvp.kv_extend_paged(pool.handle, pool.d_refs, pool.d_bt, pool.d_lens, add, pool.d_lens, missing, ws)
    for a, b in zip((pool.d_refs, pool.d_bt, pool.d_lens), state):
        assert torch.equal(a, b)  # captured, not run
    for grow in ([1, 2, 0, 16, 1], [1, 1, 1, 1, 1], [0, 0, 17, 0, 3]):
        add.copy_(torch.tensor(grow))
        graph.replay()
        want, copies = op.extend(pool.refs, pool.rows, pool.lens, grow, 16, 12)
        for old, page, rows in copies:
            for c in pool.want:
                c[page, :rows] = c[old, :rows]
        assert int(missing) == want == 0
        pool.check()


def test_on_another_stream():
    pool = Pool([20, 35], 40, 16, 6, seed=10)
    pool.fork([0, 0, 1])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert pool.extend([1, 1, 1], stream=s) == 0


def test_pages_past_two_to_the_32nd_byte():
    """A cache of more than 4 GiB: copies and moves between its ends."""
    pool = Pool([200], 4, 256, 4, hkv=1, d=8, caches=1)
    big = torch.zeros((70000, 256, 2, 64), dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    refs = torch.ones(70000, dtype=torch.int32, device="cuda")
    refs[69999], refs[3] = 2, 0
    big[69999] = 3.0
    table, lens = pool.t32([[69999, 0], [69999, 0]]), pool.t32([100, 50])
    handle = mvp.kv_caches([big], 256)
    ws = torch.empty(max(mvp.kv_compact_workspace_size(70000), 4096), dtype=torch.uint8, device="cuda")
    missing = torch.zeros(1, dtype=torch.int32, device="cuda")
    mvp.kv_extend_paged(handle, refs, table, lens, pool.t32([1, 0]), lens, missing, ws)
    assert int(missing) == 0 and table[:, 0].tolist() == [3, 69999] and refs[69999] == 1
    assert (big[3, :100] == 3).all() and not big[3, 100:].any() and not big[4].any()
    refs[5] = 0
    table[0, 0] = 0
    new = torch.empty_like(refs)
    mvp.kv_compact_paged(handle, refs, table, lens, new, missing, ws)
    assert int(missing) == 69999 and table[1, 0] == 5 and new[69999] == 5
    assert (big[5] == 3).all() and not big[6].any()


def test_bounds_checked_build():
    with mvp.bounds_checked():
        pool = Pool([20, 35, 3], 40, 16, 6, seed=11)
        pool.fork([0, 0, 1, 2])
        assert pool.extend([1, 1, 1, 30]) == 0
        pool.trim([0, 21, 0, 33])
        pool.compact()


def test_without_requests_nothing_lacks():
    pool = Pool([20], 12, 16, 4)
    missing = torch.full((1,), 5, dtype=torch.int32, device=pool.dev)
    none = pool.d_lens[:0]
    before = pool.d_refs.clone()
    mvp.kv_extend_paged(pool.handle, pool.d_refs, pool.d_bt[:0], none, none, none, missing,
                        torch.empty(0, dtype=torch.uint8, device=pool.dev))
    mvp.kv_trim_paged(pool.d_refs, pool.d_bt[:0], none, none, 16)
    assert int(missing) == 0 and torch.equal(before, pool.d_refs)


def test_a_captured_batch_change_replays():
    """Trim, fork and compact in one graph: the same pool, put back as it was, gives the same again."""
    pool = Pool([40, 17, 100, 5], 60, 16, 8, hkv=1, d=32, seed=12)
    keep, parents = pool.t32([33, 0, 100, 5]), pool.t32([2, 0, 0, 3, -1])
    bt, lens = torch.zeros((5, 8), dtype=torch.int32, device=pool.dev), torch.zeros(5, dtype=torch.int32, device=pool.dev)
    new, live = torch.zeros(60, dtype=torch.int32, device=pool.dev), torch.zeros(1, dtype=torch.int32, device=pool.dev)
    ws = torch.empty(mvp.kv_compact_workspace_size(60), dtype=torch.uint8, device=pool.dev)
    state = [t.clone() for t in (pool.d_refs, pool.d_lens, *pool.caches)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mvp.kv_trim_paged(pool.d_refs, pool.d_bt, pool.d_lens, keep, 16)
        mvp.kv_fork_paged(pool.d_refs, pool.d_bt, pool.d_lens, parents, bt, lens, 16)
        mvp.kv_compact_paged(pool.handle, pool.d_refs, bt, lens, new, live, ws)
    op.trim(pool.refs, pool.rows, pool.lens, keep.tolist(), 16)
    rows, want = op.fork(pool.refs, pool.rows, pool.lens, parents.tolist())
    new_want, moves, n = op.compact(pool.refs, rows)
    src, dst = (torch.tensor(x, device=pool.dev) for x in zip(*moves))
    for c in pool.want:
        c[dst] = c[src]
    for _ in range(2):
        for t, x in zip((pool.d_refs, pool.d_lens, *pool.caches), state):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == want and int(live) == n and new.tolist() == new_want and pool.d_refs.tolist() == pool.refs
        assert all(bt[b, :len(row)].tolist() == row for b, row in enumerate(rows))
        assert all(torch.equal(c, w) for c, w in zip(pool.caches, pool.want))


def test_every_step_on_another_stream():
    """Each step on a stream that waits for nothing but its own inputs, with the current stream kept busy."""
    pool = Pool([40, 17, 100, 5], 60, 16, 8, seed=13)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn((4096, 4096), device=pool.dev)
    for _ in range(20):
        busy = busy @ busy * 1e-3
    bt, lens = torch.zeros((2, 8), dtype=torch.int32, device=pool.dev), torch.zeros(2, dtype=torch.int32, device=pool.dev)
    parents, keep = pool.t32([2, 2]), pool.t32([0, 90])
    new, live = torch.zeros(60, dtype=torch.int32, device=pool.dev), torch.zeros(1, dtype=torch.int32, device=pool.dev)
    ws = torch.empty(mvp.kv_compact_workspace_size(60), dtype=torch.uint8, device=pool.dev)
    s.wait_stream(torch.cuda.current_stream())
    mvp.kv_fork_paged(pool.d_refs, pool.d_bt, pool.d_lens, parents, bt, lens, 16, stream=s)
    mvp.kv_trim_paged(pool.d_refs, bt, lens, keep, 16, stream=s)
    mvp.kv_compact_paged(pool.handle, pool.d_refs, bt, lens, new, live, ws, stream=s)
    s.synchronize()
    rows, n = op.fork(pool.refs, pool.rows, pool.lens, [2, 2])
    op.trim(pool.refs, rows, n, [0, 90], 16)
    _, _, want = op.compact(pool.refs, rows)
    assert int(live) == want and lens.tolist() == n and pool.d_refs.tolist() == pool.refs
    assert bt[1, :len(rows[1])].tolist() == rows[1]
