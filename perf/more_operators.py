"""Cases of attention with functions of the score (a tanh cap, a distance bias,
documents that do not see each other) and of the pages of a paged K/V cache
(grown, shared copy-on-write, freed, compacted).

``listed()`` and ``draw()`` give cases (dicts of plain values), ``prepare()``
makes what a serving engine holds before the call, ``run()`` is one pass: with
``own`` false the plain form in elementary torch operations, with ``own`` true
the framework's calls.  ``exact()`` is the definition in float64, written apart
from the plain form.
"""

import math
import random

import numpy as np
import torch

own = False

NEG = float("-inf")
FAR = 2**31 - 1  # start of a document that is not there


# ------------------------------------------------------------------ cases
def _attn(name, reqs, q_lo, q_hi, ctx_lo, ctx_hi, hq, hkv, d, block, cap=0.0, slope=0.0, docs=0, prefix=0, window=-1,
          first=0, causal=True, sinks=0, gain=1.0, lens=1):
    return {"name": name, "op": "attn", "reqs": reqs, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "hq": hq, "hkv": hkv, "d": d, "block": block, "cap": cap, "slope": slope, "docs": docs, "prefix": prefix,
            "window": window, "first": first, "causal": causal, "sinks": sinks, "gain": gain, "lens": lens}


def _pages(name, op, reqs, n_lo, n_hi, add, fan, hkv, d, block, caches, pool, lens=1):
    return {"name": name, "op": op, "reqs": reqs, "n_lo": n_lo, "n_hi": n_hi, "add": add, "fan": fan, "hkv": hkv,
            "d": d, "block": block, "caches": caches, "pool": pool, "lens": lens}


def listed():
    return [
        # two short non-causal sequences of an encoder with capped scores and key-0 sinks, where latency counts
        _attn("scored_tiny", 2, 5, 37, 0, 0, 4, 2, 64, 0, cap=30.0, window=8, causal=False, sinks=1, gain=3.0, lens=1),
        # a sliding-window layer with capped scores over four whole prompts
        _attn("capped_prefill_4x4096", 4, 4096, 4096, 0, 0, 16, 8, 256, 0, cap=50.0, window=1023, gain=4.0),
        # a layer that knows positions by a distance bias alone, whole prompts
        _attn("biased_prefill_2x8192", 2, 8192, 8192, 0, 0, 32, 8, 128, 0, slope=1.0, gain=2.0),
        # ragged documents packed into long rows, each with a bidirectional prefix
        _attn("packed_documents", 3, 9001, 16383, 0, 0, 16, 8, 128, 0, docs=700, prefix=64, lens=2),
        # prompt chunks of odd lengths over long paged contexts, capped scores and a distance bias
        _attn("scored_chunks", 6, 999, 2048, 0, 16384, 16, 4, 128, 64, cap=30.0, slope=0.25, gain=3.0, lens=3),
        # decode rows over long paged contexts, capped scores, null-logit sinks
        _attn("capped_decode_256", 256, 1, 1, 1024, 32768, 32, 8, 128, 64, cap=50.0, sinks=2, gain=4.0, lens=4),
        # a few single tokens over long contexts: distance bias, only their own document
        _attn("biased_decode_few", 5, 1, 1, 9000, 32768, 12, 4, 64, 16, slope=0.03, docs=20000, lens=5),

        # a decode step's new tokens: 256 requests, most of which stay in their last page
        _pages("pages_step_256", "extend", 256, 100, 4096, 1, 0, 2, 64, 16, 2, 131072, lens=6),
        # eight samples of each of 32 prompts write their first token: shared last pages are copied, 16 layers
        _pages("pages_samples_32x8", "sample", 32, 500, 4000, 1, 8, 8, 128, 64, 32, 3500, lens=7),
        # a beam step: 64 groups of four rows, each row continues one of its group's
        _pages("pages_beams_256", "fork", 256, 4000, 32768, 0, 4, 2, 64, 16, 1, 600000, lens=8),
        # a small pool of two layers after a few requests have ended
        _pages("pages_compact_small", "compact", 9, 30, 700, 0, 0, 4, 64, 16, 4, 700, lens=9),
        # a pool of 8 GB, half of it live and scattered, 8 layers
        _pages("pages_compact_8gb", "compact", 96, 200, 3000, 0, 0, 8, 128, 64, 16, 4096, lens=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    heads = [(4, 2), (8, 8), (8, 2), (16, 8), (32, 8), (12, 4), (6, 1)]
    while True:
        hq, hkv = rng.choice(heads)
        d = rng.choice([64, 128, 128, 256, 256, 512])
        block = rng.choice([16, 32, 64, 128, 256])
        lens = rng.randrange(1, 1 << 30)
        if rng.random() < 0.6:
            if rng.random() < 0.4:  # single tokens
                reqs, q_lo, q_hi = _log_int(rng, 1, 256), 1, 1
            else:
                reqs, q_hi = _log_int(rng, 1, 8), _log_int(rng, 2, 8192)
                q_lo = max(1, q_hi // rng.choice([1, 2, 7]))
            ctx_hi = _log_int(rng, 1, 32768)
            causal = rng.random() < 0.85
            window = -1 if rng.random() < 0.6 else _log_int(rng, 1, 8192)
            kind = rng.choice(["cap", "slope", "docs", "cap slope", "cap docs", "cap slope docs"])
            docs = _log_int(rng, 1, 5000) if "docs" in kind else 0
            case = _attn("", reqs, q_lo, q_hi, ctx_hi // rng.choice([1, 3, 30]), ctx_hi, hq, hkv, d,
                         block if rng.random() < 0.6 else 0, cap=rng.choice([5.0, 20.0, 30.0, 50.0]) if "cap" in kind else 0.0,
                         slope=rng.choice([1.0, 0.25, 0.01]) if "slope" in kind else 0.0, docs=docs,
                         prefix=_log_int(rng, 2, 300) if causal and rng.random() < 0.3 else 0, window=window,
                         first=0 if window < 0 else rng.choice([0, 0, 4, 70]), causal=causal,
                         sinks=rng.choice([0, 0, 1, 2]), gain=rng.choice([1.0, 3.0, 6.0]), lens=lens)
        else:
            op = rng.choice(["extend", "sample", "fork", "compact"])
            fan = {"extend": 0, "sample": rng.randrange(1, 17), "fork": rng.randrange(1, 9), "compact": 0}[op]
            reqs = _log_int(rng, 1, 512 if op in ("extend", "fork") else 64)
            n_hi = _log_int(rng, 1, 16384)
            add = _log_int(rng, 1, 300) if op in ("extend", "sample") else 0
            need = reqs * (n_hi // block + 1) + reqs * max(1, fan) * (add // block + 2)
            case = _pages("", op, reqs, max(1, n_hi // rng.choice([1, 3, 20])), n_hi, add, fan, hkv, d, block,
                          rng.choice([1, 2, 8, 24]), need + _log_int(rng, 1, 20000), lens=lens)
        del case["name"]
        w = work(case)
        if w["bytes"] <= _MOST[0] and w["flops"] <= _MOST[1] and _state_bytes(case) <= 24e9:
            return case


# ------------------------------------------------------------------ lengths and work
def _lengths(case):
    """(query lengths, key lengths) of the case's requests."""
    r = random.Random(case["lens"])
    if case["op"] != "attn":
        n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["reqs"])]
        n[0] = case["n_hi"]
        return None, n
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["reqs"])]
    q[0] = case["q_hi"]
    c = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]
    return q, [a + b for a, b in zip(q, c)]


def _doc_starts(case):
    """Start positions of every request's documents after its first, ascending, FAR where there are no more."""
    _, k = _lengths(case)
    r = random.Random(case["lens"] + 5)
    rows = []
    for n in k:
        at, row = r.randint(1, 2 * case["docs"]), []
        while at < n:
            row.append(at)
            at += r.randint(1, 2 * case["docs"])
        rows.append(row)
    out = np.full((len(rows), max(1, max(len(x) for x in rows))), FAR, dtype=np.int32)
    for b, row in enumerate(rows):
        out[b, :len(row)] = row
    return out


def _row_bounds(case, b, ql, kl, starts):
    """Per query row, closed: document, base interval, bidirectional prefix and first tokens (numpy int64)."""
    p = (kl - ql) + np.arange(ql, dtype=np.int64)
    w = case["window"]
    if starts is None:
        d_lo, d_hi = np.zeros_like(p), np.full_like(p, kl - 1)
    else:
        s = starts[b].astype(np.int64)
        i = np.searchsorted(s, p, side="right")
        d_lo = np.where(i > 0, s[np.maximum(i - 1, 0)], 0)
        d_hi = np.where(i < len(s), s[np.minimum(i, len(s) - 1)] - 1, FAR)
    lo = np.maximum(p - w, 0) if w >= 0 else np.zeros_like(p)
    hi = np.minimum(p if case["causal"] else (p + w if w >= 0 else np.full_like(p, kl - 1)), kl - 1)
    f_lo, f_hi = d_lo, np.minimum(np.minimum(hi, case["first"] - 1), d_hi)
    r_lo, r_hi = np.full_like(p, -1), np.full_like(p, -1)
    if case["prefix"]:
        inside = p - d_lo < case["prefix"]
        r_lo = np.where(inside, d_lo, -1)
        r_hi = np.where(inside, d_lo + case["prefix"] - 1, -1)
    return d_lo, d_hi, lo, hi, r_lo, r_hi, f_lo, f_hi


def _visible(case):
    """(visible (row, key) pairs, keys seen by any row), summed over the requests."""
    q, k = _lengths(case)
    starts = _doc_starts(case) if case["docs"] else None
    pairs = seen = 0
    for b, (ql, kl) in enumerate(zip(q, k)):
        d_lo, d_hi, lo, hi, _, r_hi, f_lo, f_hi = _row_bounds(case, b, ql, kl, starts)
        # a prefix holds its row's position, so it continues the base interval
        top = np.minimum(np.minimum(np.maximum(hi, r_hi), d_hi), kl - 1)
        low = np.maximum(lo, d_lo)
        n = np.maximum(top - low + 1, 0) + np.maximum(np.minimum(f_hi, low - 1) - f_lo + 1, 0)
        pairs += int(n.sum())
        seen += int(max(0, top.max() - low.min() + 1)) + int(max(0, (np.minimum(f_hi, low.min() - 1) - f_lo + 1).max()))
    return pairs, seen


def _page_counts(case):
    _, n = _lengths(case)
    return n, [-(-x // case["block"]) for x in n]


def work(case):
    if case["op"] == "attn":
        q, k = _lengths(case)
        pairs, seen = _visible(case)
        rows, hq, d = sum(q), case["hq"], case["d"]
        return {"bytes": 2 * 2 * rows * hq * d + 4 * rows * hq + 2 * 2 * seen * case["hkv"] * d,
                "flops": 4 * d * hq * pairs}
    n, pages = _page_counts(case)
    block, row = case["block"], case["hkv"] * case["d"] * 2
    if case["op"] == "extend":
        new = sum(-(-(x + case["add"]) // block) - y for x, y in zip(n, pages))
        return {"bytes": 4 * case["pool"] + 12 * len(n) + 12 * new, "flops": 0}
    if case["op"] == "fork":
        return {"bytes": 4 * (2 * sum(pages) + sum(pages[i] for i in _parents(case))) + 12 * len(n), "flops": 0}
    if case["op"] == "sample":
        kept = case["fan"] * sum(x % block for x in n)
        new = case["fan"] * sum(-(-(x + case["add"]) // block) - x // block for x in n)
        return {"bytes": 2 * kept * row * case["caches"] + 4 * (case["pool"] + 2 * (case["fan"] + 1) * sum(pages) + 2 * new),
                "flops": 0}
    moved = int((_live_pages(case) >= sum(pages)).sum())
    return {"bytes": 2 * moved * block * row * case["caches"] + 8 * case["pool"] + 8 * sum(pages), "flops": 0}


def _state_bytes(case):
    q, k = _lengths(case)
    if case["op"] == "attn":
        return 4 * case["hkv"] * case["d"] * sum(k) + 12 * case["hq"] * case["d"] * sum(q)
    return 2 * case["caches"] * case["pool"] * case["block"] * case["hkv"] * case["d"] + 40 * case["pool"]


# ------------------------------------------------------------------ states
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 31))


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _tables(need, width, ids):
    """A block table [len(need), width] that takes `ids` in order."""
    bt = np.zeros((len(need), width), dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt


def _live_pages(case, seed=0):
    """Pages that the requests hold, in the order of their tables."""
    _, pages = _page_counts(case)
    return np.random.RandomState(case["lens"] % 1000 + seed % 100000).permutation(case["pool"])[:sum(pages)]


def _parents(case):
    """The row that each row of the next step continues: one of its group's."""
    r = random.Random(case["lens"] + 3)
    fan = case["fan"]
    return [i // fan * fan + r.randrange(min(fan, case["reqs"] - i // fan * fan)) for i in range(case["reqs"])]


_MOST = [max(work(c)["bytes"] for c in listed()), max(work(c)["flops"] for c in listed())]


def prepare(case, seed):
    return _prepare_attn(case, seed) if case["op"] == "attn" else _prepare_pages(case, seed)


def _prepare_attn(case, seed):
    g = _gen(seed)
    s = dict(case)
    s["q_lens"], s["k_lens"] = q_lens, k_lens = _lengths(case)
    hq, hkv, d, rows = case["hq"], case["hkv"], case["d"], sum(q_lens)
    s["cu_q"], s["cu_q_host"] = _int32(_cu(q_lens)), _cu(q_lens)
    s["seq_lens"], s["max_q"], s["max_k"] = _int32(k_lens), max(q_lens), max(k_lens)
    if case["block"]:
        need = [-(-n // case["block"]) for n in k_lens]
        s["bt"] = _int32(_tables(need, max(need), np.random.RandomState(seed % 100000).permutation(sum(need))))
        key_rows = sum(need) * case["block"]
    else:
        s["cu_k"], s["cu_k_host"], key_rows = _int32(_cu(k_lens)), _cu(k_lens), sum(k_lens)
    s["q"] = (case["gain"] * _randn(g, rows, hq, d, dtype=torch.float32)).bfloat16()
    s["k"], s["v"] = _randn(g, key_rows, hkv, d), _randn(g, key_rows, hkv, d)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((hq, rows), dtype=torch.float32, device="cuda")
    s["sink_values"] = _randn(g, hq, dtype=torch.float32) if case["sinks"] else None
    # slopes that halve every hq / 8 heads
    s["slopes"] = (case["slope"] * 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)).float() if case["slope"] else None
    starts = _doc_starts(case) if case["docs"] else None
    s["doc_starts"] = None if starts is None else _int32(starts)
    s["doc_table"] = None if starts is None else torch.empty((rows, 2), dtype=torch.int32, device="cuda")
    s["range_table"] = None
    if case["prefix"]:
        t = np.concatenate([np.stack(_row_bounds(case, b, ql, kl, starts)[4:6], 1)
                            for b, (ql, kl) in enumerate(zip(q_lens, k_lens))])
        s["range_table"] = _int32(t)
    if own:
        import masked_varlen_prefill_gb300 as mvp

        s["n_dec"] = len(q_lens) if case["q_hi"] == 1 else -1
        s["ws"] = torch.empty(max(mvp.attn_workspace_size(len(q_lens), hq, d, max(k_lens)), 16), dtype=torch.uint8,
                              device="cuda")
    return s


def _prepare_pages(case, seed):
    g = _gen(seed)
    s = dict(case)
    n, pages = _page_counts(case)
    block, pool, reqs, fan = case["block"], case["pool"], case["reqs"], case["fan"]
    ids = _live_pages(case, seed)
    width = max(pages) + case["add"] // block + 2
    bt = _tables(pages, width, ids)
    refs = np.zeros(pool, dtype=np.int32)
    refs[ids] = 1
    s["caches"] = [_randn(g, pool, block, case["hkv"], case["d"]) for _ in range(case["caches"])]
    s["refs0"], s["bt0"], s["lens0"] = _int32(refs), _int32(bt), _int32(n)
    s["refs"], s["bt"] = s["refs0"].clone(), s["bt0"].clone()
    s["missing"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["max_new"] = case["add"] // block + 2
    if case["op"] == "extend":
        s["add_lens"], s["new_lens"] = _int32([case["add"]] * reqs), _int32([0] * reqs)
    elif case["op"] == "sample":
        rows = reqs * (fan + 1)  # the prompts stay, each with `fan` samples
        s["parents"] = _int32(list(range(reqs)) + [i // fan for i in range(reqs * fan)])
        s["bt_out"] = torch.zeros((rows, width), dtype=torch.int32, device="cuda")
        s["add_lens"] = _int32([0] * reqs + [case["add"]] * (reqs * fan))
        s["lens_out"], s["new_lens"] = _int32([0] * rows), _int32([0] * rows)
        s["end_lens"] = _int32(n + [0] * (reqs * fan))
    elif case["op"] == "fork":
        s["parents"] = _int32(_parents(case))
        s["bt_out"], s["lens_out"] = torch.zeros_like(s["bt"]), torch.zeros_like(s["lens0"])
    else:
        s["map"] = torch.empty(pool, dtype=torch.int32, device="cuda")
        s["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import masked_varlen_prefill_gb300 as mvp

        s["handle"] = mvp.kv_caches(s["caches"], block)
        rows = reqs * (fan + 1) if case["op"] == "sample" else reqs
        size = mvp.kv_compact_workspace_size(pool) if case["op"] == "compact" else mvp.kv_extend_workspace_size(rows)
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _own_attn(s):
    import masked_varlen_prefill_gb300 as mvp

    if s["docs"]:
        mvp.fill_query_documents(s["doc_starts"], s["cu_q"], s["seq_lens"], s["doc_table"], s["q"].shape[0])
    kw = dict(lse=s["lse"], range_table=s["range_table"], causal=s["causal"], window_left=s["window"],
              window_right=0 if s["causal"] else s["window"], first_tokens=s["first"], sinks=s["sink_values"],
              sink_mode=s["sinks"], scale=s["d"] ** -0.5, workspace=s["ws"], num_decode_reqs=s["n_dec"],
              softcap=s["cap"], distance_slopes=s["slopes"], doc_table=s["doc_table"])
    if s["block"]:
        mvp.attn_fwd_paged(s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["seq_lens"], s["bt"], s["block"], s["max_q"],
                           s["max_k"], **kw)
    else:
        mvp.attn_fwd_varlen(s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], **kw)
    return {"out": s["out"], "lse": s["lse"]}


def _own_extend(s):
    """A step's new tokens, none of which are kept (a rejected draft): the pool ends as it began."""
    import masked_varlen_prefill_gb300 as mvp

    mvp.kv_extend_paged(s["handle"], s["refs"], s["bt"], s["lens0"], s["add_lens"], s["new_lens"], s["missing"], s["ws"])
    mvp.kv_trim_paged(s["refs"], s["bt"], s["new_lens"], s["lens0"], s["block"])
    return _page_outputs(s, table=s["bt"], lens=s["new_lens"])


def _own_sample(s):
    """Prompts are shared by their samples, the samples take their first tokens, and end."""
    import masked_varlen_prefill_gb300 as mvp

    mvp.kv_fork_paged(s["refs"], s["bt"], s["lens0"], s["parents"], s["bt_out"], s["lens_out"], s["block"])
    mvp.kv_extend_paged(s["handle"], s["refs"], s["bt_out"], s["lens_out"], s["add_lens"], s["new_lens"], s["missing"],
                        s["ws"])
    mvp.kv_trim_paged(s["refs"], s["bt_out"], s["new_lens"], s["end_lens"], s["block"])
    return _page_outputs(s, table=s["bt_out"], lens=s["lens_out"])


def _own_fork(s):
    import masked_varlen_prefill_gb300 as mvp

    s["refs"].copy_(s["refs0"])  # the pool as the step finds it
    mvp.kv_fork_paged(s["refs"], s["bt"], s["lens0"], s["parents"], s["bt_out"], s["lens_out"], s["block"])
    return _page_outputs(s, table=s["bt_out"], lens=s["lens_out"])


def _own_compact(s):
    import masked_varlen_prefill_gb300 as mvp

    s["refs"].copy_(s["refs0"])  # the pool as the step finds it
    s["bt"].copy_(s["bt0"])
    mvp.kv_compact_paged(s["handle"], s["refs"], s["bt"], s["lens0"], s["map"], s["live"], s["ws"])
    return _page_outputs(s, table=s["bt"], lens=s["live"])


def _page_outputs(s, table, lens):
    out = {"refs": s["refs"], "table": table, "lens": lens, "missing": s["missing"]}
    if s["op"] != "fork":
        out["caches"] = [c.view(torch.int16) for c in s["caches"]]  # moved bit for bit
    if s["op"] == "compact":
        out["map"] = s["map"]
    return out


# The plain forms: 32-bit elementary operations, rounded once.
def _plain_docs(s):
    """The closed key interval of every row's document."""
    rows = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"], rows, right=True) - 1
    p = s["seq_lens"][b].long() - s["cu_q"][b + 1] + rows
    # one ascending list of (request, start), a request's own range of numbers each
    n, m = s["doc_starts"].shape
    zero = torch.zeros((n, 1), dtype=torch.long, device="cuda")
    starts = torch.cat([zero, s["doc_starts"].long()], 1) + (torch.arange(n, device="cuda") << 32)[:, None]
    i = torch.searchsorted(starts.flatten(), (b << 32) + p, right=True)  # (FAR lies past every position)
    hi = torch.where(i < (b + 1) * (m + 1), starts.flatten()[i.clamp(max=n * (m + 1) - 1)] - (b << 32), FAR)
    return torch.stack([starts.flatten()[i - 1] - (b << 32), hi - 1], 1)


def _plain_pieces(s, most=1 << 28):
    """Row pieces of every request: (first row, rows, q [hkv, g, rows, d], p [rows, 1], keys, keys' rows, mask)."""
    hq, hkv, d, w, first = s["hq"], s["hkv"], s["d"], s["window"], s["first"]
    docs = _plain_docs(s) if s["docs"] else None
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["k_lens"])):
        step = max(1, min(ql, most // (hq * kl)))
        for r0 in range(0, ql, step):
            n = min(step, ql - r0)
            at = int(s["cu_q_host"][b]) + r0
            p = torch.arange(kl - ql + r0, kl - ql + r0 + n, device="cuda")[:, None]
            j = torch.arange(0, kl, device="cuda")
            if w >= 0 and kl - ql + r0 - w > first:  # keys that no row of the piece sees are left out
                j = torch.cat([j[:first], j[kl - ql + r0 - w:]])
            right = j <= p if s["causal"] else (j <= p + w if w >= 0 else j >= 0)
            see = right & ((j >= p - w) | (j < first)) if w >= 0 else right & (p >= 0)
            if s["range_table"] is not None:
                t = s["range_table"][at:at + n]
                see = see | ((j >= t[:, :1]) & (j <= t[:, 1:]) & ((j >= p - w) if w >= 0 else True))
            if docs is not None:
                see = see & (j >= docs[at:at + n, :1]) & (j <= docs[at:at + n, 1:])
            rows = s["bt"][b][j // s["block"]].long() * s["block"] + j % s["block"] if s["block"] else j + int(s["cu_k_host"][b])
            q = s["q"][at:at + n].float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            yield at, n, q, p, j, rows, see


def _plain_attn(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    g = hq // hkv
    for at, n, q, p, j, rows, see in _plain_pieces(s):
        x = torch.matmul(q.reshape(hkv, g * n, d), s["k"][rows].float().permute(1, 2, 0)).view(hkv, g, n, -1) * d ** -0.5
        if s["cap"]:
            x = s["cap"] * torch.tanh(x / s["cap"])
        if s["slopes"] is not None:
            x = x - s["slopes"].view(hkv, g, 1, 1) * (p - j).abs()
        if s["sinks"] == 1:
            x = x + s["sink_values"].view(hkv, g, 1, 1) * (j == 0)
        x = x.masked_fill(~see, NEG)
        top = x.amax(-1, keepdim=True)
        if s["sinks"] == 2:
            sink = s["sink_values"].view(hkv, g, 1, 1)
            top = torch.maximum(top, sink)
        top = torch.where(top == NEG, 0.0, top)
        x = torch.exp(x - top)
        z = x.sum(-1, keepdim=True)
        if s["sinks"] == 2:
            z = z + torch.exp(sink - top)
        o = torch.matmul(x.view(hkv, g * n, -1), s["v"][rows].float().permute(1, 0, 2)).view(hkv, g, n, d)
        o = torch.where(z > 0, o / z, 0.0)
        s["out"][at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, d).bfloat16()
        s["lse"][:, at:at + n] = (top + torch.log(z)).view(hq, n)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_grow(s, bt, lens):
    """bt and new_lens for lens + add_lens: pages are taken lowest first, requests in order; a partly filled page that
    others hold too is copied.  (The pools of the cases have the pages; missing is 0.)"""
    refs, block = s["refs"], s["block"]
    n, a = lens.long(), s["add_lens"].long()
    last = n // block
    old = torch.gather(bt.long(), 1, last[:, None])[:, 0]
    shared = (a > 0) & (n % block > 0) & (refs[old] > 1)
    start = torch.where(shared, last, (n + block - 1) // block)
    count = (n + a + block - 1) // block - start
    s["missing"].copy_(torch.clamp(count.sum() - (refs <= 0).sum(), min=0))
    free = torch.sort((refs > 0).int(), stable=True).indices
    b, k = torch.nonzero(torch.arange(s["max_new"], device="cuda") < count[:, None], as_tuple=True)
    page = free[(torch.cumsum(count, 0) - count)[b] + k]
    bt[b, start[b] + k] = page.int()
    refs[page] = 1
    i = torch.nonzero(shared)[:, 0]
    at, row = torch.nonzero(torch.arange(block, device="cuda") < (n % block)[i][:, None], as_tuple=True)
    new = bt[i, last[i]].long()
    for c in s["caches"]:
        c[new[at], row] = c[old[i][at], row]
    refs.index_add_(0, old[i], torch.full_like(i, -1, dtype=torch.int32))
    s["new_lens"].copy_(n + a)


def _plain_cut(s, bt, lens, keep):
    """lens cut to keep: the pages past it lose a holder."""
    block = s["block"]
    col = torch.arange(bt.shape[1], device="cuda")
    gone = (col >= (keep[:, None] + block - 1) // block) & (col < (lens[:, None] + block - 1) // block)
    page = bt[gone].long()
    s["refs"].index_add_(0, page, torch.full_like(page, -1, dtype=torch.int32))
    lens.copy_(torch.minimum(lens, keep))


def _plain_share(s):
    """bt_out and lens_out: the parents' rows; a page gains a holder for every row more that names it."""
    block, bt, n, parents = s["block"], s["bt"], s["lens0"], s["parents"].long()
    held = torch.arange(bt.shape[1], device="cuda") < (n[:, None] + block - 1) // block
    more = torch.full_like(n, -1).index_add_(0, parents, torch.ones_like(s["parents"]))
    s["refs"].index_add_(0, bt[held].long(), more[:, None].expand(bt.shape)[held])
    s["bt_out"].copy_(torch.where(held[parents], bt[parents], s["bt_out"]))
    s["lens_out"].copy_(n[parents])


def _plain_extend(s):
    _plain_grow(s, s["bt"], s["lens0"])
    _plain_cut(s, s["bt"], s["new_lens"], s["lens0"])
    return _page_outputs(s, table=s["bt"], lens=s["new_lens"])


def _plain_sample(s):
    _plain_share(s)
    _plain_grow(s, s["bt_out"], s["lens_out"])
    _plain_cut(s, s["bt_out"], s["new_lens"], s["end_lens"])
    return _page_outputs(s, table=s["bt_out"], lens=s["lens_out"])


def _plain_fork(s):
    s["refs"].copy_(s["refs0"])
    _plain_share(s)
    return _page_outputs(s, table=s["bt_out"], lens=s["lens_out"])


def _plain_compact(s):
    s["refs"].copy_(s["refs0"])
    s["bt"].copy_(s["bt0"])
    refs, bt, block = s["refs"], s["bt"], s["block"]
    page, live = torch.arange(s["pool"], device="cuda"), refs > 0
    s["live"].copy_(live.sum())
    src, dst = torch.nonzero(live & (page >= s["live"]))[:, 0], torch.nonzero(~live & (page < s["live"]))[:, 0]
    s["map"].copy_(torch.where(live, page, -1))
    s["map"][src] = dst.int()
    for c in s["caches"]:
        c[dst] = c[src]
    refs[dst] = refs[src]
    refs[src] = 0
    held = torch.arange(bt.shape[1], device="cuda") < (s["lens0"][:, None] + block - 1) // block
    bt[held] = s["map"][bt[held].long()]
    return _page_outputs(s, table=s["bt"], lens=s["live"])


_OWN = {"attn": _own_attn, "extend": _own_extend, "sample": _own_sample, "fork": _own_fork, "compact": _own_compact}
_PLAIN = {"attn": _plain_attn, "extend": _plain_extend, "sample": _plain_sample, "fork": _plain_fork,
          "compact": _plain_compact}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    if case["op"] != "attn":
        return _exact_pages(case, seed)
    if work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    hq, hkv, d, w = s["hq"], s["hkv"], s["d"], s["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["q"].shape[0]), NEG, dtype=torch.float64, device="cuda")
    sinks = None if s["sink_values"] is None else s["sink_values"].double()
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["k_lens"])):
        at = int(s["cu_q_host"][b])
        key = torch.arange(kl, device="cuda")
        if s["block"]:
            ids = s["bt"][b].long()
            where = (ids[:, None] * s["block"] + torch.arange(s["block"], device="cuda")).flatten()[:kl]
        else:
            where = key + int(s["cu_k_host"][b])
        # the number of the document that a position lies in
        doc = torch.zeros_like(key)
        if s["docs"]:
            begins = [x for x in _doc_starts(s)[b].tolist() if x < kl]
            doc[torch.tensor(begins, device="cuda", dtype=torch.long)] = 1
            doc = torch.cumsum(doc, 0)
        step = max(1, (1 << 27) // kl)
        for r0 in range(0, ql, step):
            r1 = min(ql, r0 + step)
            p = torch.arange(r0, r1, device="cuda")[:, None] + (kl - ql)
            dist = p - key
            near = dist <= w if w >= 0 else dist == dist
            ahead = dist >= 0 if s["causal"] else (-dist <= w if w >= 0 else dist == dist)
            see = ahead & (near | (key < s["first"]))
            if s["range_table"] is not None:
                t = s["range_table"][at + r0:at + r1].long()
                see |= near & (t[:, 0:1] <= key) & (key <= t[:, 1:2])
            see &= doc[p] == doc
            cols = torch.nonzero(see.any(0))[:, 0]
            see, dist = see[:, cols], dist[:, cols].abs().double()
            for h in range(hkv):
                kh, vh = s["k"][where[cols], h].double(), s["v"][where[cols], h].double()
                for i in range(h * hq // hkv, (h + 1) * hq // hkv):
                    x = s["q"][at + r0:at + r1, i].double() @ kh.T / math.sqrt(d)
                    if s["cap"]:
                        x = s["cap"] * torch.tanh(x / s["cap"])
                    if s["slopes"] is not None:
                        x = x - dist * s["slopes"][i].double()
                    if s["sinks"] == 1:
                        x[:, cols == 0] += sinks[i]
                    x = torch.where(see, x, torch.full_like(x, NEG))
                    z = torch.logsumexp(torch.cat([x, sinks[i].expand(r1 - r0, 1)], 1) if s["sinks"] == 2 else x, 1)
                    lse[i, at + r0:at + r1] = z
                    out[at + r0:at + r1, i] = torch.exp(x - torch.where(z == NEG, torch.zeros_like(z), z)[:, None]) @ vh
    return {"out": out, "lse": lse}


def _exact_pages(case, seed):
    """Page by page, as a caller with one table after another would do it; what the caches hold is not a computed value."""
    n, pages = _page_counts(case)
    block, fan, reqs = case["block"], case["fan"], case["reqs"]
    ids = _live_pages(case, seed).tolist()
    width = max(pages) + case["add"] // block + 2
    refs, rows, at = [0] * case["pool"], [], 0
    for m in pages:
        rows.append(ids[at:at + m])
        at += m
    for x in ids:
        refs[x] = 1
    lens, missing, extra = list(n), 0, {}
    if case["op"] in ("fork", "sample"):
        parents = _parents(case) if case["op"] == "fork" else list(range(reqs)) + [i // fan for i in range(reqs * fan)]
        for x in ids:
            refs[x] -= 1
        rows, lens = [list(rows[i]) for i in parents], [n[i] for i in parents]
        for row in rows:
            for x in row:
                refs[x] += 1
    table = np.zeros((len(rows), width), dtype=np.int64)
    if case["op"] in ("extend", "sample"):
        grows = range(reqs) if case["op"] == "extend" else range(reqs, len(rows))
        before, free = list(refs), iter([i for i, x in enumerate(refs) if x <= 0])
        for b in grows:
            full = lens[b] // block
            if lens[b] % block and before[rows[b][full]] > 1:
                refs[rows[b][full]] -= 1
                rows[b][full] = next(free)
                refs[rows[b][full]] += 1
            while len(rows[b]) * block < lens[b] + case["add"]:
                rows[b].append(next(free))
                refs[rows[b][-1]] += 1
        held = rows
        for b in grows:  # cut back
            keep = -(-lens[b] // block) if case["op"] == "extend" else 0
            for x in rows[b][keep:]:
                refs[x] -= 1
        rows = held
    if case["op"] == "compact":
        live = [i for i, x in enumerate(refs) if x > 0]
        free = [i for i in range(len(live)) if refs[i] <= 0]
        to = {x: x for x in live if x < len(live)}
        to.update(zip([x for x in live if x >= len(live)], free))
        rows = [[to[x] for x in row] for row in rows]
        refs = [1 if i < len(live) else 0 for i in range(case["pool"])]
        lens = [len(live)]
        extra = {"map": torch.tensor([to.get(i, -1) for i in range(case["pool"])])}
    for b, row in enumerate(rows):
        table[b, :len(row)] = row
    out = {"refs": torch.tensor(refs), "table": torch.tensor(table), "lens": torch.tensor(lens),
           "missing": torch.tensor([missing]), **extra}
    if case["op"] != "fork":
        out["caches"] = [None] * case["caches"]
    return out
