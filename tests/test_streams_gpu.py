"""Calls given a stream run on that stream (GPU): the current stream is still at
other work when they have ended, and what they wrote is read on theirs."""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import workloads
from oracle import pages as op
from oracle import scores as osc

from . import gpu_helpers as gh
from .test_pages_gpu import Pool
from .test_scored_gpu import Case, _slopes

pytestmark = pytest.mark.gpu


class Elsewhere:
    """``stream``, which has waited for everything before it, with the current
    stream kept at work; ``read`` copies tensors to the host on it."""

    def __enter__(self):
        self.stream = torch.cuda.Stream()
        busy = torch.zeros((8192, 8192), device="cuda")
        to = torch.empty_like(busy)
        torch.mm(busy, busy, out=to)
        torch.cuda.synchronize()
        for _ in range(40):  # (at 70 TFLOP/s some 16 ms each)
            torch.mm(busy, busy, out=to)
        self.end = torch.cuda.Event()
        self.end.record()
        return self

    def read(self, *tensors):
        host = [torch.empty(t.shape, dtype=t.dtype, pin_memory=True) for t in tensors]
        with torch.cuda.stream(self.stream):
            for h, t in zip(host, tensors):
                h.copy_(t, non_blocking=True)
        self.stream.synchronize()
        assert not self.end.query(), "the current stream has ended its work: nothing is shown"
        return host

    def __exit__(self, *_):
        torch.cuda.synchronize()


def _pinned(*shapes):
    """Memory that the reads take, held once before: allocating it may wait for the device."""
    held = [torch.empty(s, dtype=dt, pin_memory=True) for s, dt in shapes]
    del held


def test_the_pools_steps():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731

    def arguments():
        pool = Pool([40, 17, 100, 5], 60, 16, 9, seed=13)
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda")
              for n in (mvp.kv_extend_workspace_size(3), mvp.kv_compact_workspace_size(60))]
        return (pool, i32(3, 9), i32(3), i32(60), i32(1), i32(1).fill_(77), pool.t32([2, 2, 0]), pool.t32([1, 30, 0]),
                pool.t32([0, 120, 40]), ws)

    def steps(pool, bt, lens, new, live, missing, parents, add, keep, ws, stream):
        mvp.kv_fork_paged(pool.d_refs, pool.d_bt, pool.d_lens, parents, bt, lens, 16, stream=stream)
        mvp.kv_extend_paged(pool.handle, pool.d_refs, bt, lens, add, lens, missing, ws[0], stream=stream)
        mvp.kv_trim_paged(pool.d_refs, bt, lens, keep, 16, stream=stream)
        mvp.kv_compact_paged(pool.handle, pool.d_refs, bt, lens, new, live, ws[1], stream=stream)

    steps(*arguments(), None)  # (kernels are loaded)
    args = arguments()
    pool, *outs = args[:6]
    outs = (pool.d_refs, *outs, *pool.caches)
    _pinned(*((t.shape, t.dtype) for t in outs))
    with Elsewhere() as other:
        steps(*args, other.stream)
        refs, bt, lens, new, live, missing, *caches = other.read(*outs)
    rows, n = op.fork(pool.refs, pool.rows, pool.lens, [2, 2, 0])
    lack, copies = op.extend(pool.refs, rows, n, [1, 30, 0], 16, 9)
    assert lack == 0 and len(copies) == 2
    for old, page, filled in copies:
        for c in pool.want:
            c[page, :filled] = c[old, :filled]
    op.trim(pool.refs, rows, n, [0, 120, 40], 16)
    new_want, moves, want = op.compact(pool.refs, rows)
    assert moves
    for src, dst in moves:
        for c in pool.want:
            c[dst] = c[src]
    assert int(missing) == 0 and int(live) == want and lens.tolist() == n and refs.tolist() == pool.refs
    assert new.tolist() == new_want and all(bt[b, :len(row)].tolist() == row for b, row in enumerate(rows))
    for c, w in zip(caches, pool.want):
        assert torch.equal(c[:want], w[:want].cpu())


@pytest.mark.parametrize("block", [0, 16])
def test_attention_with_functions_of_the_score(block):
    """The document table and the attention that reads it, prompts and single tokens (two streams inside)."""
    w = workloads.Workload("t", 22, [1, 1, 150], [700, 300, 200], 4, 2, 128, True, -1, 0, workloads.SINK_NONE, None)
    starts = [[5, 600], [], [30, 111]]
    case = Case(w, cap=20.0, slopes=_slopes(4), starts=starts)
    padded = torch.full((3, 2), 2 ** 31 - 1, dtype=torch.int32)
    for b, row in enumerate(starts):
        padded[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    padded, lens = padded.to(case.dev), torch.tensor(w.k_lens, dtype=torch.int32, device=case.dev)
    cu_q, cu_k = gh.device_meta(w, case.dev)
    kw = case.kw()
    docs = kw["doc_table"] = torch.full((w.total_q, 2), -3, dtype=torch.int32, device=case.dev)
    out, lse = torch.zeros_like(case.q), torch.zeros((4, w.total_q), device=case.dev)
    ws = torch.empty(mvp.attn_workspace_size(2, 4, 128, 700), dtype=torch.uint8, device=case.dev)
    kc, vc, bt, sl = workloads.to_paged(case.k, case.v, w.k_lens, 16, seed=1, table_fill=-5)

    def call(stream):
        mvp.fill_query_documents(padded, cu_q, lens, docs, w.total_q, stream=stream)
        more = dict(lse=lse, workspace=ws, num_decode_reqs=2, stream=stream, **kw)
        if block:
            mvp.attn_fwd_paged(case.q, kc, vc, out, cu_q, sl, bt, block, 150, 700, **more)
        else:
            mvp.attn_fwd_varlen(case.q, case.k, case.v, out, cu_q, cu_k, 150, 700, **more)

    call(None)  # (kernels are loaded)
    torch.cuda.synchronize()
    for t in (docs, out, lse):
        t.zero_()
    _pinned(*((t.shape, t.dtype) for t in (docs, out, lse)))
    with Elsewhere() as other:
        call(other.stream)
        got_docs, got, got_lse = other.read(docs, out, lse)
    assert np.array_equal(got_docs.numpy(), case.doc)
    assert np.array_equal(case.doc, np.concatenate([osc.documents(s, p) for s, p in zip(starts, case.positions)]))
    gh.compare(got, got_lse, *case.oracle(), strict=False)
