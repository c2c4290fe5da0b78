"""Cases of the bounded-cache operators: rotary positions written into a paged
K/V cache, attention under a sliding window with first tokens that stay
visible, the attention weight each cached key received, and eviction by it.

``listed()`` and ``draw()`` give cases (dicts of plain values), ``prepare()``
makes what a serving engine holds before the call, ``run()`` is one pass:
with ``own`` false the plain form in elementary torch operations, with ``own``
true the framework's call.  ``exact()`` is the definition in float64, written
apart from the plain form.
"""

import math
import random

import numpy as np
import torch

own = False

NEG = float("-inf")


# ------------------------------------------------------------------ cases
def _rope(name, reqs, q_lo, q_hi, ctx_hi, hq, hkv, d, rot, axes, block, adjacent=False, src="bf16", far=False, lens=1):
    return {"name": name, "op": "rope", "reqs": reqs, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": 0, "ctx_hi": ctx_hi,
            "hq": hq, "hkv": hkv, "d": d, "rot": rot, "axes": axes, "block": block, "adjacent": adjacent, "src": src,
            "far": far, "lens": lens}


def _attn(name, op, reqs, q_lo, q_hi, ctx_lo, ctx_hi, hq, hkv, d, window, first, block, causal=True, ranges=0,
          sinks=0, lens=1):
    return {"name": name, "op": op, "reqs": reqs, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "hq": hq, "hkv": hkv, "d": d, "window": window, "first": first, "block": block, "causal": causal,
            "ranges": ranges, "sinks": sinks, "lens": lens}


def _evict(name, reqs, n_lo, n_hi, hkv, d, budget, first, recent, block, lens=1):
    return {"name": name, "op": "evict", "reqs": reqs, "n_lo": n_lo, "n_hi": n_hi, "hkv": hkv, "d": d,
            "budget": budget, "first": first, "recent": recent, "block": block, "lens": lens}


def listed():
    return [
        # a decode step of the mixed serving batch's 256 rows, one text position per axis
        _rope("rope_decode_256", 256, 1, 1, 400, 32, 8, 128, 128, 3, 64),
        # video prompts prefilled in chunks of a few thousand tokens, whole heads rotated
        _rope("rope_video_chunks", 8, 1024, 2048, 3000, 16, 8, 256, 256, 3, 64, lens=2),
        # fp32 projections, a partly rotated head in the adjacent pairing, positions past a million
        _rope("rope_partial_fp32", 3, 77, 1501, 900, 8, 2, 64, 32, 2, 16, adjacent=True, src="fp32", far=True, lens=3),

        # two short non-causal sequences of an encoder, where latency counts
        _attn("first_tiny", "attn", 2, 5, 37, 0, 0, 4, 2, 64, 8, 4, 0, causal=False, lens=4),
        # sliding-window layer over four whole prompts, packed keys
        _attn("first_prefill_4x4096", "attn", 4, 4096, 4096, 0, 0, 16, 8, 256, 1023, 4, 0),
        # the same layer in chunks over long paged contexts, with multimodal ranges
        _attn("first_chunks_ranges", "attn", 8, 2048, 2048, 0, 30000, 16, 8, 256, 4095, 64, 64, ranges=8, lens=5),
        # decode rows over long paged contexts, null-logit sinks
        _attn("first_decode_256", "attn", 256, 1, 1, 1024, 32768, 32, 8, 128, 4095, 16, 64, sinks=2, lens=6),

        # one short prompt's weights, where latency counts
        _attn("weights_short", "weights", 1, 190, 190, 0, 0, 8, 2, 64, -1, 0, 16),
        # prompt chunks over long paged contexts
        _attn("weights_chunks", "weights", 4, 2048, 2048, 0, 16384, 16, 8, 256, -1, 0, 64, lens=7),
        # every decode step adds one row's weights over the whole context
        _attn("weights_decode_256", "weights", 256, 1, 1, 1024, 32768, 32, 8, 128, -1, 0, 64, lens=8),

        # two requests a little over a small budget
        _evict("evict_small", 2, 560, 640, 4, 64, 512, 4, 64, 16),
        # a batch of long contexts cut down to 4096 keys each
        _evict("evict_batch_48", 48, 4096, 32768, 8, 128, 4096, 64, 1024, 64, lens=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    heads = [(4, 2), (8, 8), (8, 2), (16, 8), (32, 8), (12, 4), (6, 1)]
    op = rng.choice(["rope", "attn", "attn", "weights", "weights", "evict"])
    while True:
        hq, hkv = rng.choice(heads)
        d = rng.choice([64, 128, 128, 256, 256, 512])
        block = rng.choice([16, 32, 64, 128, 256])
        lens = rng.randrange(1, 1 << 30)
        if op == "rope":
            reqs = _log_int(rng, 1, 256)
            q_hi = _log_int(rng, 1, 4096)
            case = _rope("", reqs, max(1, q_hi // rng.choice([1, 2, 5])), q_hi, _log_int(rng, 1, 4000), hq, hkv, d,
                         rng.choice([r for r in (32, 64, 96, 128, 256) if r <= d]), rng.choice([1, 2, 3, 3, 4]), block,
                         adjacent=rng.random() < 0.4, src=rng.choice(["bf16", "bf16", "fp32"]),
                         far=rng.random() < 0.3, lens=lens)
        elif op == "evict":
            reqs = _log_int(rng, 1, 64)
            n_hi = _log_int(rng, 300, 65536)
            budget = max(64, min(n_hi, _log_int(rng, 64, 16384)))
            first = rng.choice([0, 1, 4, 16, 64])
            recent = rng.randrange(0, max(1, budget - first) // 2 + 1)
            case = _evict("", reqs, max(1, n_hi // rng.choice([1, 2, 4])), n_hi, hkv, d, budget, first, recent, block,
                          lens=lens)
        else:
            if rng.random() < 0.4:  # decode rows
                reqs, q_lo, q_hi = _log_int(rng, 1, 256), 1, 1
            else:
                reqs, q_hi = _log_int(rng, 1, 8), _log_int(rng, 2, 4096)
                q_lo = max(1, q_hi // rng.choice([1, 2, 7]))
            ctx_hi = _log_int(rng, 1, 32768)
            window = -1 if (op == "weights" and rng.random() < 0.5) else _log_int(rng, 1, 8192)
            first = 0 if window < 0 else _log_int(rng, 1, 300)
            causal = rng.random() < 0.85
            case = _attn("", op, reqs, q_lo, q_hi, ctx_hi // rng.choice([1, 3, 30]), ctx_hi, hq, hkv, d, window, first,
                         block if rng.random() < 0.6 else 0, causal=causal,
                         ranges=rng.choice([0, 0, 3, 9]) if causal and q_hi > 1 else 0, sinks=rng.choice([0, 0, 1, 2]),
                         lens=lens)
        del case["name"]
        w = work(case)
        if w["bytes"] <= _MOST[0] and w["flops"] <= _MOST[1] and _state_bytes(case) <= 24e9:
            return case


# ------------------------------------------------------------------ lengths and work
def _lengths(case):
    """(query lengths, key lengths) of the case's requests."""
    r = random.Random(case["lens"])
    if case["op"] == "evict":
        n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["reqs"])]
        n[0] = case["n_hi"]
        return None, n
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["reqs"])]
    q[0] = case["q_hi"]
    c = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]
    return q, [a + b for a, b in zip(q, c)]


def _ranges(case):
    """Closed, non-overlapping key ranges [reqs, R, 2] of the case (0, 0: unused)."""
    q, k = _lengths(case)
    r = random.Random(case["lens"] + 17)
    out = np.zeros((len(q), case["ranges"], 2), dtype=np.int32)
    for b, (ql, kl) in enumerate(zip(q, k)):
        at = max(0, kl - ql - 40)
        for i in range(case["ranges"]):
            s = at + r.randint(0, max(1, ql // case["ranges"] // 2))
            e = s + r.randint(1, max(2, ql // case["ranges"] // 2))
            if e >= kl + 50:
                break
            out[b, i] = (s, e)
            at = e + 2
    return out


def _row_bounds(case, b, ql, kl, ranges):
    """Per query row: base interval, range interval and first-token interval, closed (numpy int64)."""
    p = (kl - ql) + np.arange(ql, dtype=np.int64)
    w, c = case["window"], case["causal"]
    lo = np.maximum(p - w, 0) if w >= 0 else np.zeros_like(p)
    right = p if c else (p + w if w >= 0 else np.full_like(p, kl - 1))
    hi = np.minimum(right, kl - 1)
    f_hi = np.minimum(hi, case["first"] - 1)
    r_lo, r_hi = np.ones_like(p), np.zeros_like(p)
    for s, e in ([] if ranges is None else ranges[b]):
        if s < e:
            inside = (p >= s) & (p <= e)
            r_lo = np.where(inside, np.maximum(s, lo), r_lo)
            r_hi = np.where(inside, min(e, kl - 1), r_hi)
    return lo, hi, r_lo, r_hi, f_hi


def _visible(case):
    """(visible (row, key) pairs, keys seen by any row), summed over the requests."""
    q, k = _lengths(case)
    rg = _ranges(case) if case["ranges"] else None
    pairs = seen = 0
    for b, (ql, kl) in enumerate(zip(q, k)):
        lo, hi, r_lo, r_hi, f_hi = _row_bounds(case, b, ql, kl, rg)
        # every range interval holds its row's position, so it continues the base interval
        top = np.where(r_lo <= r_hi, np.maximum(hi, r_hi), hi)
        n = np.maximum(top - lo + 1, 0) + np.maximum(np.minimum(f_hi, lo - 1) + 1, 0)
        pairs += int(n.sum())
        cover = int(top.max() - lo.min() + 1)
        seen += cover + int(max(0, min(case["first"], lo.min())))
    return pairs, seen


def work(case):
    d, hkv = case["d"], case["hkv"]
    q, k = _lengths(case)
    if case["op"] == "rope":
        rows, src = sum(q), (4 if case["src"] == "fp32" else 2)
        return {"bytes": rows * (d * (case["hq"] + 2 * hkv) * (src + 2) + 4 * case["axes"]),
                "flops": rows * (case["hq"] + hkv) * case["rot"] * 3}
    if case["op"] == "evict":
        keep = sum(min(n, case["budget"]) for n in k)
        return {"bytes": hkv * (4 * sum(k) + keep * (2 * 2 * 2 * d + 4 + 4) + 4 * (sum(k) - keep)), "flops": 0}
    pairs, seen = _visible(case)
    rows, hq = sum(q), case["hq"]
    if case["op"] == "attn":
        return {"bytes": 2 * 2 * rows * hq * d + 4 * rows * hq + 2 * 2 * seen * hkv * d, "flops": 4 * d * hq * pairs}
    return {"bytes": 2 * rows * hq * d + 4 * rows * hq + 2 * seen * hkv * d + 4 * sum(k) * hkv,
            "flops": 2 * d * hq * pairs}


def _state_bytes(case):
    q, k = _lengths(case)
    if case["op"] == "evict":
        return case["hkv"] * (4 * case["d"] * (sum(k) + case["reqs"] * case["budget"]) + 8 * case["reqs"] * max(k))
    return 4 * case["hkv"] * case["d"] * sum(k) + 12 * case["hq"] * case["d"] * sum(q) + 4 * case["hkv"] * len(k) * max(k)


_MOST = [max(work(c)["bytes"] for c in listed()), max(work(c)["flops"] for c in listed())]


# ------------------------------------------------------------------ states
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 31))


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _tables(lens, block, seed, extra=0):
    """A block table over a pool in random order, and the pool's size in blocks."""
    need = [-(-n // block) for n in lens]
    total = sum(need)
    order = np.random.RandomState(seed).permutation(total) + extra
    bt = np.full((len(lens), max(need)), 0, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    return bt, total


def _inv_freq(case):
    return 10000.0 ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])


def _pair_axes(case):
    pairs, axes = case["rot"] // 2, case["axes"]
    return np.minimum(np.arange(pairs) * axes // pairs, axes - 1).astype(np.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    q_lens, k_lens = _lengths(case)
    s["q_lens"], s["k_lens"] = q_lens, k_lens
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "evict":
        block, budget = case["block"], case["budget"]
        out_lens = [min(n, budget) for n in k_lens]
        # blocks the batch lives in, then the blocks it is cut down into
        bt, blocks = _tables(k_lens, block, seed % 1000)
        bt_out, blocks_out = _tables(out_lens, block, seed % 1000 + 1, extra=blocks)
        rows = (blocks + blocks_out) * block
        s["k_cache"], s["v_cache"] = _randn(g, rows, hkv, d), _randn(g, rows, hkv, d)
        n = torch.tensor(k_lens, device="cuda")
        # accumulated attention weight: heavy-tailed, some keys never seen
        w = torch.exp(1.5 * torch.randn((case["reqs"], hkv, max(k_lens)), generator=g, device="cuda") - 3)
        w = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.05, 0.0, w)
        s["weights"] = torch.where(torch.arange(max(k_lens), device="cuda") < n[:, None, None], w, 0.0).contiguous()
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["seq_lens"], s["bt"], s["bt_out"], s["dst"] = _int32(k_lens), _int32(bt), _int32(bt_out), blocks * block
        s["new_lens"] = torch.zeros(case["reqs"], dtype=torch.int32, device="cuda")
        s["kept"] = torch.full((case["reqs"], hkv, budget), -7, dtype=torch.int32, device="cuda")
        if own:
            import masked_varlen_prefill_gb300 as mvp

            s["ws"] = torch.empty(mvp.kv_evict_workspace_size(case["reqs"], hkv, budget), dtype=torch.uint8,
                                  device="cuda")
        return s
    hq, rows = case["hq"], sum(q_lens)
    s["cu_q"], s["cu_q_host"] = _int32(_cu(q_lens)), _cu(q_lens)
    s["seq_lens"], s["max_q"], s["max_k"] = _int32(k_lens), max(q_lens), max(k_lens)
    if case["block"]:
        bt, blocks = _tables(k_lens, case["block"], seed % 1000)
        s["bt"], key_rows = _int32(bt), blocks * case["block"]
    else:
        s["cu_k"], s["cu_k_host"], key_rows = _int32(_cu(k_lens)), _cu(k_lens), sum(k_lens)
    if case["op"] == "rope":
        src = torch.float32 if case["src"] == "fp32" else torch.bfloat16
        qkv = _randn(g, rows, hq + 2 * hkv, d, dtype=src)  # one fused projection's output
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty((rows, hq, d), dtype=torch.bfloat16, device="cuda")
        s["k_cache"], s["v_cache"] = _randn(g, key_rows, hkv, d), _randn(g, key_rows, hkv, d)
        # time runs with the text; height and width stay within a frame
        top = 4_000_000 if case["far"] else max(k_lens)
        pos = torch.randint(0, 128, (case["axes"], rows), generator=g, device="cuda", dtype=torch.int32)
        pos[0] = torch.randint(0, top + 1, (rows,), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = pos.contiguous()
        s["inv_freq"] = torch.tensor(_inv_freq(case), device="cuda")
        s["pair_axes"] = torch.tensor(_pair_axes(case), device="cuda").long()
        if own:
            import masked_varlen_prefill_gb300 as mvp

            s["table"] = mvp.rope_table(_inv_freq(case), _pair_axes(case))
        return s
    s["q"] = _randn(g, rows, hq, d)
    s["k"] = _randn(g, key_rows, hkv, d)
    if case["op"] == "attn":
        s["v"] = _randn(g, key_rows, hkv, d)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((hq, rows), dtype=torch.float32, device="cuda")
    s["sink_values"] = _randn(g, hq, dtype=torch.float32) if case["sinks"] else None
    s["range_table"] = None
    s["bounds"] = []
    rg = _ranges(case) if case["ranges"] else None
    table = np.full((rows, 2), -1, dtype=np.int32)
    lse = np.zeros(rows, dtype=np.float32)
    for b, (ql, kl) in enumerate(zip(q_lens, k_lens)):
        at = s["cu_q_host"][b]
        lo, hi, r_lo, r_hi, f_hi = _row_bounds(case, b, ql, kl, rg)
        if rg is not None:
            p = (kl - ql) + np.arange(ql)
            for x, y in rg[b]:
                if x < y:
                    table[at:at + ql][(p >= x) & (p <= y)] = (x, y)
        n = np.maximum(hi - lo + 1, 0) + np.maximum(r_hi - hi, 0) * (r_lo <= r_hi) + np.maximum(np.minimum(f_hi, lo - 1) + 1, 0)
        # scores of unit variance: the log of n terms' sum is near ln n + 1/2
        lse[at:at + ql] = np.log(np.maximum(n, 1)) + 0.5
    if rg is not None:
        s["range_table"] = _int32(table)
    if case["op"] == "weights":
        s["lse"] = (torch.tensor(lse, device="cuda") + 0.05 * _randn(g, hq, rows, dtype=torch.float32)).contiguous()
        s["weights"] = torch.zeros((case["reqs"], hkv, max(k_lens)), dtype=torch.float32, device="cuda")
    if own:
        import masked_varlen_prefill_gb300 as mvp

        n_dec = sum(1 for x in q_lens if x == 1) if case["q_hi"] == 1 else 0
        s["n_dec"] = n_dec if n_dec == len(q_lens) else -1
        size = (mvp.attn_workspace_size(len(q_lens), hq, d, max(k_lens)) if case["op"] == "attn" else
                mvp.key_weights_workspace_size(len(q_lens), hkv, max(q_lens), max(k_lens)))
        s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _own_rope(s):
    import masked_varlen_prefill_gb300 as mvp

    mvp.rope_append_paged(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"], s["positions"], s["table"],
                          s["cu_q"], s["seq_lens"], s["bt"], s["block"], adjacent=s["adjacent"])
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _mask_args(s):
    return dict(range_table=s["range_table"], causal=s["causal"], window_left=s["window"],
                window_right=0 if s["causal"] else s["window"], first_tokens=s["first"], sinks=s["sink_values"],
                sink_mode=s["sinks"], scale=s["d"] ** -0.5, workspace=s["ws"], num_decode_reqs=s["n_dec"])


def _own_attn(s):
    import masked_varlen_prefill_gb300 as mvp

    if s["block"]:
        mvp.attn_fwd_paged(s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["seq_lens"], s["bt"], s["block"], s["max_q"],
                           s["max_k"], lse=s["lse"], **_mask_args(s))
    else:
        mvp.attn_fwd_varlen(s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"],
                            lse=s["lse"], **_mask_args(s))
    return {"out": s["out"], "lse": s["lse"]}


def _own_weights(s):
    import masked_varlen_prefill_gb300 as mvp

    if s["block"]:
        mvp.attn_key_weights_paged(s["q"], s["k"], s["lse"], s["weights"], s["cu_q"], s["seq_lens"], s["bt"],
                                   s["block"], s["max_q"], s["max_k"], accumulate=False, **_mask_args(s))
    else:
        mvp.attn_key_weights_varlen(s["q"], s["k"], s["lse"], s["weights"], s["cu_q"], s["cu_k"], s["max_q"],
                                    s["max_k"], accumulate=False, **_mask_args(s))
    return {"weights": s["weights"]}


def _own_evict(s):
    import masked_varlen_prefill_gb300 as mvp

    mvp.kv_evict_paged(s["k_cache"], s["v_cache"], s["weights"], s["seq_lens"], s["bt"], s["block"], s["budget"],
                       s["new_lens"], s["kept"], s["ws"], max(s["k_lens"]), first_tokens=s["first"],
                       recent_tokens=s["recent"], block_table_out=s["bt_out"], weights_out=s["weights_out"])
    return _evict_outputs(s)


def _evict_outputs(s):
    return {"lens": s["new_lens"], "kept": s["kept"], "weights": s["weights_out"], "k": s["k_cache"][s["dst"]:],
            "v": s["v_cache"][s["dst"]:]}


# The plain forms: 32-bit elementary operations (angles in 64), rounded once.
def _cache_rows(bt, block, j):
    return bt[j // block].long() * block + j % block


def _plain_rotate(s, x):
    """x [rows, heads, d] in 32 bits, rotated."""
    half = s["rot"] // 2
    angle = s["positions"].double()[s["pair_axes"]].T * s["inv_freq"]  # [rows, half]
    c, n = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    y = x.clone()
    a, b = (slice(0, s["rot"], 2), slice(1, s["rot"], 2)) if s["adjacent"] else (slice(0, half), slice(half, s["rot"]))
    y[..., a] = x[..., a] * c - x[..., b] * n
    y[..., b] = x[..., a] * n + x[..., b] * c
    return y


def _plain_rope(s):
    s["q_out"].copy_(_plain_rotate(s, s["q"].float()))
    i = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"], i, right=True, out_int32=True).long() - 1
    j = s["seq_lens"][b] - s["cu_q"][b + 1] + i  # a request's new tokens are its last keys
    at = s["bt"][b, j // s["block"]].long() * s["block"] + j % s["block"]
    s["k_cache"][at] = _plain_rotate(s, s["k"].float()).bfloat16()
    s["v_cache"][at] = s["v"].bfloat16()
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _plain_pieces(s, most=1 << 28):
    """Row pieces of every request: (b, first row, rows, q [hkv, g, rows, d], keys' rows, mask [rows, keys])."""
    hq, hkv, d, w, first = s["hq"], s["hkv"], s["d"], s["window"], s["first"]
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["k_lens"])):
        step = max(1, min(ql, most // (hq * kl)))
        for r0 in range(0, ql, step):
            n = min(step, ql - r0)
            at = int(s["cu_q_host"][b]) + r0
            p = torch.arange(kl - ql + r0, kl - ql + r0 + n, device="cuda")[:, None]
            k_lo = max(0, kl - ql + r0 - w) if w >= 0 else 0
            j = torch.arange(k_lo, kl, device="cuda")
            if k_lo > 0 and first > 0:
                j = torch.cat([torch.arange(0, min(first, k_lo), device="cuda"), j])
            right = j <= p if s["causal"] else (j <= p + w if w >= 0 else j >= 0)
            see = right & ((j >= p - w) | (j < first)) if w >= 0 else right & (p >= 0)
            if s["range_table"] is not None:
                t = s["range_table"][at:at + n]
                see = see | ((j >= t[:, :1]) & (j <= t[:, 1:]) & ((j >= p - w) if w >= 0 else True))
            rows = _cache_rows(s["bt"][b], s["block"], j) if s["block"] else j + int(s["cu_k_host"][b])
            q = s["q"][at:at + n].float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            yield b, at, n, q, j, rows, see


def _plain_scores(s, q, j, rows, see):
    k = s["k"][rows].float().permute(1, 2, 0)  # [hkv, d, keys]
    hkv, g, n, d = q.shape
    x = torch.matmul(q.reshape(hkv, g * n, d), k).view(hkv, g, n, -1) * d ** -0.5
    if s["sinks"] == 1:
        x = x + s["sink_values"].view(hkv, g, 1, 1) * (j == 0)
    return x.masked_fill(~see, NEG)


def _plain_attn(s):
    hq = s["hq"]
    for b, at, n, q, j, rows, see in _plain_pieces(s):
        x = _plain_scores(s, q, j, rows, see)
        top = x.amax(-1, keepdim=True)
        if s["sinks"] == 2:
            sink = s["sink_values"].view(*x.shape[:2], 1, 1)
            top = torch.maximum(top, sink)
        top = torch.where(top == NEG, 0.0, top)
        x = torch.exp(x - top)
        z = x.sum(-1, keepdim=True)
        if s["sinks"] == 2:
            z = z + torch.exp(sink - top)
        v = s["v"][rows].float().permute(1, 0, 2)
        o = torch.matmul(x.view(x.shape[0], -1, x.shape[-1]), v).view(*x.shape[:3], -1)
        o = torch.where(z > 0, o / z, 0.0)
        s["out"][at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, -1).bfloat16()
        s["lse"][:, at:at + n] = (top + torch.log(z)).view(hq, n)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weights(s):
    for b, kl in enumerate(s["k_lens"]):
        s["weights"][b, :, :kl] = 0
    for b, at, n, q, j, rows, see in _plain_pieces(s):
        x = _plain_scores(s, q, j, rows, see)
        lse = s["lse"][:, at:at + n].view(x.shape[0], x.shape[1], n, 1)
        x = torch.exp(x - lse).masked_fill(~see, 0.0)
        s["weights"][b].index_add_(1, j, x.sum((1, 2)))
    return {"weights": s["weights"]}


def _plain_evict(s):
    block, budget = s["block"], s["budget"]
    s["kept"].fill_(-1)
    s["new_lens"].copy_(torch.clamp(s["seq_lens"], max=budget))
    for b, n in enumerate(s["k_lens"]):
        m = min(n, budget)
        j = torch.arange(n, device="cuda")
        always = (j < s["first"]) | (j >= n - s["recent"])
        rank = torch.where(always, float("inf"), torch.nan_to_num(s["weights"][b, :, :n], nan=-1.0))
        order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :m]
        kept = torch.sort(order, dim=1).values  # [hkv, m]
        s["kept"][b, :, :m] = kept.int()
        src = _cache_rows(s["bt"][b], block, kept)
        dst = _cache_rows(s["bt_out"][b], block, torch.arange(m, device="cuda"))
        h = torch.arange(s["hkv"], device="cuda")[:, None]
        s["k_cache"][dst[None, :], h] = s["k_cache"][src, h]
        s["v_cache"][dst[None, :], h] = s["v_cache"][src, h]
        s["weights_out"][b, :, :m] = torch.gather(s["weights"][b], 1, kept)
        s["weights_out"][b, :, m:n] = 0
    return _evict_outputs(s)


_OWN = {"rope": _own_rope, "attn": _own_attn, "weights": _own_weights, "evict": _own_evict}
_PLAIN = {"rope": _plain_rope, "attn": _plain_attn, "weights": _plain_weights, "evict": _plain_evict}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "evict":
        return _exact_evict(s)
    return _exact_attention(s)


def _table_rows(s, b, n, table="bt"):
    flat = [int(x) for x in s[table][b].cpu()]
    return torch.tensor([flat[i // s["block"]] * s["block"] + i % s["block"] for i in range(n)], device="cuda")


def _exact_rope(s):
    rot = s["rot"]
    i = np.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if s["adjacent"] else (i, i + rot // 2)
    pos = s["positions"].cpu().numpy().astype(np.float64)
    angle = torch.tensor(np.stack([pos[a] * f for a, f in zip(_pair_axes(s), _inv_freq(s))], 1), device="cuda")
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotated(x):
        x = x.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k, v = s["k_cache"].double(), s["v_cache"].double()
    rk = rotated(s["k"])
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["k_lens"])):
        at = int(s["cu_q_host"][b])
        rows = _table_rows(s, b, kl)[kl - ql:]
        k[rows], v[rows] = rk[at:at + ql], s["v"][at:at + ql].double()
    return {"q": rotated(s["q"]), "k": k, "v": v}


def _exact_attention(s):
    hq, hkv, d, w = s["hq"], s["hkv"], s["d"], s["window"]
    g = hq // hkv
    attn = s["op"] == "attn"
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda") if attn else None
    lse_out = torch.full((hq, s["q"].shape[0]), NEG, dtype=torch.float64, device="cuda")
    weights = None if attn else torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    sinks = None if s["sink_values"] is None else s["sink_values"].double()
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["k_lens"])):
        at = int(s["cu_q_host"][b])
        rows = _table_rows(s, b, kl) if s["block"] else torch.arange(kl, device="cuda") + int(s["cu_k_host"][b])
        key = torch.arange(kl, device="cuda")[None]
        step = max(1, (1 << 27) // kl)
        for r0 in range(0, ql, step):
            r1 = min(ql, r0 + step)
            p = torch.arange(r0, r1, device="cuda")[:, None] + (kl - ql)
            dist = p - key
            ahead = dist >= 0 if s["causal"] else (-dist <= w if w >= 0 else dist == dist)
            near = dist <= w if w >= 0 else dist == dist
            see = ahead & (near | (key < s["first"]))
            if s["range_table"] is not None:
                t = s["range_table"][at + r0:at + r1].long()
                see |= near & (t[:, 0:1] <= key) & (key <= t[:, 1:2])
            cols = torch.nonzero(see.any(0))[:, 0]
            see = see[:, cols]
            for h in range(hkv):
                kh = s["k"][rows[cols], h].double()
                vh = s["v"][rows[cols], h].double() if attn else None
                for i in range(h * g, (h + 1) * g):
                    x = s["q"][at + r0:at + r1, i].double() @ kh.T / math.sqrt(d)
                    if s["sinks"] == 1:
                        x[:, cols == 0] += sinks[i]
                    x = torch.where(see, x, torch.full_like(x, NEG))
                    if not attn:
                        e = torch.exp(x - s["lse"][i, at + r0:at + r1].double()[:, None])
                        weights[b, h, cols] += torch.where(see, e, torch.zeros_like(e)).sum(0)
                        continue
                    z = torch.logsumexp(torch.cat([x, sinks[i].expand(r1 - r0, 1)], 1) if s["sinks"] == 2 else x, 1)
                    lse_out[i, at + r0:at + r1] = z
                    prob = torch.exp(x - torch.where(z == NEG, torch.zeros_like(z), z)[:, None])
                    out[at + r0:at + r1, i] = prob @ vh
    return {"out": out, "lse": lse_out} if attn else {"weights": weights}


def _exact_evict(s):
    kept = np.full(tuple(s["kept"].shape), -1, dtype=np.int64)
    weights = s["weights"].cpu().numpy()
    w_out = s["weights_out"].double().cpu().numpy()
    k, v = s["k_cache"].double(), s["v_cache"].double()
    for b, n in enumerate(s["k_lens"]):
        m = min(n, s["budget"])
        src, dst = _table_rows(s, b, n), _table_rows(s, b, m, "bt_out")
        for h in range(s["hkv"]):
            middle = np.arange(s["first"], max(s["first"], n - s["recent"]))
            middle = middle[middle < n]
            fixed = np.setdiff1d(np.arange(n), middle)
            value = weights[b, h, middle]
            value = np.where(np.isnan(value), -np.inf, value)
            best = middle[np.lexsort((middle, -value))[:max(0, m - len(fixed))]] if n > m else middle
            keep = np.sort(np.concatenate([fixed, best]))
            kept[b, h, :m] = keep
            w_out[b, h, :m], w_out[b, h, m:n] = weights[b, h, keep], 0
            at = torch.tensor(keep, device="cuda")
            k[dst, h], v[dst, h] = s["k_cache"][src[at], h].double(), s["v_cache"][src[at], h].double()
    return {"lens": torch.tensor([min(n, s["budget"]) for n in s["k_lens"]], device="cuda"),
            "kept": torch.tensor(kept, device="cuda"), "weights": torch.tensor(w_out, device="cuda"),
            "k": k[s["dst"]:], "v": v[s["dst"]:]}
