"""Attention with functions of the score (a tanh cap, a distance bias) and
documents that do not see each other (GPU), packed and paged, against the
float64 oracle, with the tolerances of the other attention tests
(``gpu_helpers.compare``: 1e-2 or two bf16 half steps of the value, lse 1e-3
relative).  A capped score is off by some 9e-7 of itself and a biased one by half
an fp32 unit of the bias, 1e-4 at most here: less than either by far."""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import workloads
from oracle import cache as oc
from oracle import scores as osc

from . import gpu_helpers as gh

pytestmark = pytest.mark.gpu

W = workloads.Workload
NONE, KEY0, NULL = workloads.SINK_NONE, workloads.SINK_KEY0_BIAS, workloads.SINK_NULL_LOGIT


def _slopes(hq, top=1.0):
    return top * 2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)


class Case:
    """A workload's tensors and masks, its run and its oracle."""

    def __init__(self, w, cap=0.0, slopes=None, starts=None, first=0, ctx=None, ranges=None, gain=3.0, doc=None):
        self.w, self.cap, self.first, self.ctx = w, cap, first, ctx
        q, k, v, self.sinks = gh.make_inputs(w)
        self.q, self.k, self.v = (gain * q.float()).bfloat16(), k, v
        self.dev = q.device
        self.slopes = None if slopes is None else np.asarray(slopes, dtype=np.float32)
        cu_q, _ = w.cu_seqlens()
        self.positions = [(w.k_lens[b] - w.q_lens[b] if ctx is None else ctx[b]) + np.arange(w.q_lens[b])
                          for b in range(w.num_reqs)]
        self.doc = doc
        if starts is not None:
            self.doc = np.concatenate([osc.documents(s, p) for s, p in zip(starts, self.positions)])
        self.table = None
        if ranges is not None:  # closed ranges per request; rows outside of them have none
            self.table = np.full((w.total_q, 2), -1, dtype=np.int32)
            for b in range(w.num_reqs):
                for x, y in ranges[b]:
                    inside = (self.positions[b] >= x) & (self.positions[b] <= y)
                    self.table[cu_q[b]:cu_q[b + 1]][inside] = (x, y)

    def kw(self):
        i32 = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device=self.dev)  # noqa: E731
        return dict(causal=self.w.causal, window_left=self.w.window_left, window_right=self.w.window_right,
                    sinks=self.sinks, sink_mode=self.w.sink_mode, scale=self.w.scale, first_tokens=self.first,
                    context_lens=i32(self.ctx), range_table=i32(self.table), softcap=self.cap,
                    distance_slopes=None if self.slopes is None else torch.tensor(self.slopes, device=self.dev),
                    doc_table=i32(self.doc))

    def run(self, block=0, n_dec=-1, ws=True, want_lse=True, stream=None, **over):
        w, kw = self.w, {**self.kw(), **over}
        cu_q, cu_k = gh.device_meta(w, self.dev)
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full((w.num_heads_q, w.total_q), float("nan"), device=self.dev) if want_lse else None
        n = mvp.attn_workspace_size(w.num_reqs if n_dec < 0 else n_dec, w.num_heads_q, w.head_dim, max(w.k_lens))
        space = torch.empty(n, dtype=torch.uint8, device=self.dev) if ws else None
        lens = max(1, max(w.q_lens)), max(w.k_lens)
        if block:
            kc, vc, bt, sl = workloads.to_paged(self.k, self.v, w.k_lens, block, seed=w.seed, table_fill=-5)
            mvp.attn_fwd_paged(self.q, kc, vc, out, cu_q, sl, bt, block, *lens, lse=lse, workspace=space,
                               num_decode_reqs=n_dec, stream=stream, **kw)
        else:
            mvp.attn_fwd_varlen(self.q, self.k, self.v, out, cu_q, cu_k, *lens, lse=lse, workspace=space,
                                num_decode_reqs=n_dec, stream=stream, **kw)
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        return out, lse

    def oracle(self):
        w = self.w
        q, k, v = (t.double().cpu().numpy() for t in (self.q, self.k, self.v))
        sinks = None if self.sinks is None else self.sinks.double().cpu().numpy()
        cu_q, cu_k = w.cu_seqlens()
        out, lse = np.zeros(q.shape), np.full((w.num_heads_q, w.total_q), -np.inf)
        for b in range(w.num_reqs):
            rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
            c = w.k_lens[b] - w.q_lens[b] if self.ctx is None else self.ctx[b]
            mask = oc.mask_first(w.q_lens[b], w.k_lens[b], c, w.causal, w.window_left, w.window_right, self.first,
                                 None if self.table is None else self.table[rq])
            out[rq], lse[:, rq] = osc.attend(q[rq], k[rk], v[rk], self.positions[b], mask, w.scale, self.cap,
                                             self.slopes, None if self.doc is None else self.doc[rq], sinks,
                                             w.sink_mode)
        return out, lse

    def check(self, block=16, n_dec=-1, ws=True, what=""):
        """packed against the oracle, paged against packed bit for bit."""
        a = self.run(n_dec=n_dec, ws=ws)
        gh.compare(*a, *self.oracle(), what=what, strict=False)
        assert same(a, self.run(block, n_dec=n_dec, ws=ws)), "paged != packed"
        return a


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


KINDS = {
    "cap": dict(cap=20.0),
    "slopes": dict(slopes=True),
    "documents": dict(docs=True),
    "cap+slopes": dict(cap=5.0, slopes=True),
    "cap+slopes+documents": dict(cap=30.0, slopes=True, docs=True),
}


def _make(w, kind, seed=0, **kw):
    rng = np.random.RandomState(seed)
    kind = KINDS[kind]
    starts = None
    if kind.get("docs"):  # documents of one token to about the longest request
        starts = [np.sort(rng.choice(max(2, n), min(n, 1 + rng.randint(0, 9)), replace=False)) for n in w.k_lens]
    return Case(w, cap=kind.get("cap", 0.0), slopes=_slopes(w.num_heads_q) if kind.get("slopes") else None,
                starts=starts, **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_head_dims(d, kind):
    """Prompts with and without context, odd lengths, single tokens among them."""
    _make(W("t", 11 + d, [150, 1, 37, 129], [400, 310, 37, 513], 8, 2, d, True, -1, 0, NONE, None), kind).check(what=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (12, 4), (16, 2), (7, 1), (24, 1)])
def test_head_layouts(hq, hkv, kind):
    w = W("t", hq, [70, 1, 1], [300, 275, 90], hq, hkv, 64 if hq > 8 else 128, True, -1, 0, NONE, None)
    _make(w, kind).check(block=64)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sink", [KEY0, NULL])
@pytest.mark.parametrize("causal,wl,wr", [(True, 60, 0), (True, 0, 0), (False, 20, 33), (False, -1, -1), (False, -1, 5)])
def test_masks_and_sinks(causal, wl, wr, sink, kind):
    w = W("t", 5, [200, 1, 5, 1], [200, 333, 5, 1], 4, 2, 128, causal, wl, wr, sink, None)
    _make(w, kind, seed=3).check(block=32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_first_tokens(d, kind):
    """Some first tokens in the row's document, some not; rows whose window starts among them."""
    w = W("t", 6, [260, 1, 1, 40], [700, 690, 20, 45], 4, 2, d, True, 30, 0, KEY0, None)
    for first in (1, 21, 300):
        _make(w, kind, seed=4, first=first).check(what=f"first={first}")


@pytest.mark.parametrize("kind", KINDS)
def test_ranges(kind):
    """Bidirectional ranges: distances of both signs; ranges that reach over a document's end."""
    w = W("t", 7, [300, 140], [450, 140], 8, 4, 128, True, 90, 0, NULL, None)
    _make(w, kind, seed=5, ranges=[[(155, 280), (300, 301), (390, 449)], [(0, 139)]]).check(block=128)


def test_document_prefixes():
    """Packed documents whose first tokens see each other, as prefix masks do."""
    w = W("t", 8, [500, 77], [500, 77], 4, 1, 256, True, -1, 0, NONE, None)
    starts = [[1, 2, 100, 350, 499], [0, 40]]
    ranges = [[(0, 0), (1, 1), (2, 31), (100, 129), (350, 379)], [(0, 29), (40, 69)]]
    Case(w, starts=starts, ranges=ranges).check()


@pytest.mark.parametrize("d", [64, 512])
def test_rows_that_see_nothing(d):
    """Empty documents, documents past the keys, documents that a window leaves behind, requests without rows."""
    w = W("t", 9, [140, 0, 1, 3, 1], [140, 60, 200, 90, 1], 4, 2, d, True, 10, 0, NULL, None)
    doc = np.tile([0, 10 ** 9], (w.total_q, 1))
    doc[::3] = (-1, -1)
    doc[1::7] = (100000, 200000)
    doc[2::5] = (0, 3)
    doc[140] = (5, 4)
    for sink in (NULL, NONE):
        w.sink_mode = sink
        case = Case(w, doc=doc, slopes=_slopes(4))
        out, lse = case.check()
        if sink == NONE:
            blind = torch.isneginf(lse).all(0)
            assert blind.sum() > 50 and not out[blind].any()


def test_nothing_given_is_the_plain_call():
    """Scores without a cap, bias or documents, and those of a document that
    holds every key, are the plain call's bit for bit where its kernels are
    the same (no cap, no bias, whole documents leave every score as it is)."""
    w = W("t", 10, [200, 1, 65], [300, 500, 65], 8, 2, 128, True, 77, 0, KEY0, None)
    case = Case(w)
    plain = case.run()
    assert same(plain, case.run(softcap=0.0, distance_slopes=None, doc_table=None))
    whole = torch.tensor([[0, 2 ** 31 - 1]] * w.total_q, dtype=torch.int32, device=case.dev)
    assert same(plain, case.run(doc_table=whole))


def test_keys_of_other_documents_may_hold_anything():
    """K of keys that no row's document holds: NaN and infinities.  (V of masked
    keys next to visible ones has to be finite, as in every attention call.)"""
    w = W("t", 12, [60, 1], [300, 280], 4, 2, 128, True, -1, 0, NONE, None)
    case = Case(w, cap=15.0, slopes=_slopes(4), doc=np.array([[100, 290]] * 60 + [[270, 279]]))
    case.k[20] = float("nan")
    case.k[99] = float("inf")
    case.k[291:295] = float("-inf")
    case.k[300:560] = float("nan")
    case.check()


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 1.0, 300.0, 1e30])
def test_caps_of_every_size(cap):
    """Scores far past the cap (all equal it), and far below (the plain softmax)."""
    w = W("t", 13, [130, 1], [200, 190], 4, 2, 64, True, -1, 0, NONE, None)
    case = Case(w, cap=cap, gain=20.0)
    case.check()


def test_infinite_scores_are_capped():
    """q.k overflows fp32: +-inf before the cap (all products of a key have its sign), +-cap after it."""
    w = W("t", 14, [40, 1], [40, 30], 2, 1, 64, True, -1, 0, NONE, None)
    case = Case(w, cap=4.0)
    sign = torch.where(torch.arange(70, device=case.dev) % 3 == 0, -1.0, 1.0)[:, None, None]
    case.q, case.k = (1e20 * case.q.float().abs()).bfloat16(), (1e20 * sign * (case.k.float().abs() + 0.1)).bfloat16()
    out, lse = case.run()
    gh.compare(out, lse, *case.oracle(), strict=False)


@pytest.mark.parametrize("slopes", [[0.0, -0.01], [100.0, 1e-6], [-3.0, 0.5]])
def test_slopes_of_every_kind(slopes):
    """No slope, slopes that leave the row's own key alone, slopes towards far keys."""
    w = W("t", 15, [200, 1, 1], [900, 2000, 1], 2, 1, 128, True, -1, 0, NONE, None)
    Case(w, slopes=slopes).check()
    w = W("t", 15, [200, 3], [200, 90], 2, 1, 256, False, -1, -1, NULL, None)
    Case(w, slopes=slopes, cap=9.0).check()


def test_positions_past_two_to_the_24th():
    """Contexts whose earlier keys were dropped: positions far past the keys held.
    Distances are then rounded to fp32, a relative 2^-24: up to 2 in 4e7, times a slope of 1e-6."""
    w = W("t", 16, [100, 1], [300, 250], 4, 2, 64, True, -1, 0, NONE, None)
    case = Case(w, slopes=[1e-6, 1e-7, 0.0, 2e-7], ctx=[40_000_123, 50_000_001])
    case.check()


@pytest.mark.parametrize("n_dec", [-1, 3])
@pytest.mark.parametrize("kind", KINDS)
def test_decode_rows_first_in_a_mixed_batch(kind, n_dec):
    w = W("t", 17, [1, 1, 1, 300, 20], [900, 5000, 1, 1300, 20], 8, 2, 128, True, -1, 0, NULL, None)
    case = _make(w, kind, seed=6)
    case.check(block=256, n_dec=n_dec)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_long_rows_are_split_and_joined(d, kind):
    w = W("t", 18, [1, 1, 1], [20000, 9000, 37], 4, 2, d, True, -1, 0, KEY0, None)
    case = _make(w, kind, seed=7)
    case.check(block=16)
    case.check(block=64, ws=False)


def test_documents_of_long_rows_skip_the_rest():
    """A document's start and end inside tiles, at their borders, and in one split part alone."""
    w = W("t", 19, [1] * 6, [20000] * 6, 4, 1, 128, True, -1, 0, NONE, None)
    doc = np.array([[0, 19999], [8191, 8191], [4096, 12287], [19999, 30000], [63, 64], [12345, 19998]])
    Case(w, doc=doc).check()


def test_without_lse():
    w = W("t", 20, [150, 1], [200, 300], 4, 2, 128, True, -1, 0, NONE, None)
    case = _make(w, "cap+slopes")
    a, b = case.run(), case.run(want_lse=False)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))


def test_a_captured_call_replays():
    """One graph with the document fill and both calls; other documents by its replays."""
    w = W("t", 21, [200, 1], [300, 400], 4, 2, 128, True, -1, 0, NONE, None)
    case = Case(w, cap=20.0, slopes=_slopes(4), starts=[[0], [0]])
    cu_q, cu_k = gh.device_meta(w, case.dev)
    starts = torch.full((2, 4), 2 ** 31 - 1, dtype=torch.int32, device=case.dev)
    lens = torch.tensor(w.k_lens, dtype=torch.int32, device=case.dev)
    kw = case.kw()
    kw["doc_table"] = torch.empty((w.total_q, 2), dtype=torch.int32, device=case.dev)
    out, lse = torch.empty_like(case.q), torch.empty((4, w.total_q), device=case.dev)
    ws = torch.empty(mvp.attn_workspace_size(2, 4, 128, 400), dtype=torch.uint8, device=case.dev)

    def step():
        mvp.fill_query_documents(starts, cu_q, lens, kw["doc_table"], w.total_q)
        mvp.attn_fwd_varlen(case.q, case.k, case.v, out, cu_q, cu_k, 200, 400, lse=lse, workspace=ws, **kw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rows in ([[], []], [[120, 130, 299], [399]], [[250], [10, 11, 12, 13]]):
        starts.fill_(2 ** 31 - 1)
        for b, row in enumerate(rows):
            starts[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        graph.replay()
        torch.cuda.synchronize()
        assert mvp.get_last_device_error() == 0
        case.doc = np.concatenate([osc.documents(s, p) for s, p in zip(rows, case.positions)])
        assert np.array_equal(kw["doc_table"].cpu().numpy(), case.doc)
        gh.compare(out, lse, *case.oracle(), strict=False)


def test_on_another_stream():
    w = W("t", 22, [150, 1], [200, 300], 4, 2, 128, True, -1, 0, NONE, None)
    case = _make(w, "cap+slopes+documents")
    a = case.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert same(a, case.run(stream=s))


def test_bounds_checked_build():
    w = W("t", 23, [150, 1, 40], [200, 300, 90], 4, 2, 128, True, 50, 0, KEY0, None)
    case = _make(w, "cap+slopes+documents", first=3)
    a = case.run()
    with mvp.bounds_checked():
        assert same(a, case.run()) and same(a, case.run(16))


# ------------------------------------------------------------------ the document table
@pytest.mark.parametrize("seed", range(4))
def test_document_table(seed):
    rng = np.random.RandomState(seed)
    reqs = [1, 5, 60, 700][seed]
    k_lens = rng.randint(1, 900, reqs)
    q_lens = np.minimum(k_lens, rng.randint(0, 300, reqs))
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    starts = np.full((reqs, 12), 2 ** 31 - 1, dtype=np.int64)
    for b in range(reqs):
        m = rng.randint(0, 13)
        starts[b, :m] = np.sort(rng.randint(0, 1000, m))  # equal starts among them
    want = np.concatenate([osc.documents(starts[b], k_lens[b] - q_lens[b] + np.arange(q_lens[b])) for b in range(reqs)])
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((cu[-1] + 5, 2), 77, dtype=torch.int32, device="cuda")
    mvp.fill_query_documents(t(starts), t(cu), t(k_lens), out, int(cu[-1]) + 3)
    assert mvp.last_launch_count() == 1
    got = out.cpu().numpy()
    assert np.array_equal(got[:cu[-1]], want)
    assert (got[cu[-1]:cu[-1] + 3] == -1).all() and (got[cu[-1] + 3:] == 77).all()  # a padded batch; rows past it


def test_document_table_without_starts():
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    mvp.fill_query_documents(None, t([0, 4]), t([9]), out, 4)
    assert out.tolist() == [[0, 2 ** 31 - 2]] * 4
    mvp.fill_query_documents(None, t([0, 0]), t([9]), out[:0], 0)
    assert mvp.last_launch_count() == 0
