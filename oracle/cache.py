"""Oracle of the bounded paged cache's steps (test infrastructure, float64).

* ``rotate``       -- rotary positions with several axes, from the formula.
* ``attend``       -- attention under a window with first tokens that stay
  visible: key ``j < first`` is exempt from the window's past side, not from
  the causal (or right) bound.  A brute-force softmax over the dense mask.
* ``key_weights``  -- the softmax weight each key received, per KV head.
* ``evict``        -- which keys stay, by sorting.

Written from the definitions; shares no code with the GPU package.
"""

from __future__ import annotations

import numpy as np

from .attention import SINK_KEY0_BIAS, SINK_NULL_LOGIT, visible_mask


def rotate(x, positions, inv_freq, axes, adjacent):
    """x [rows, heads, D] (float64); positions [num_axes, rows] ints."""
    x = np.asarray(x, dtype=np.float64)
    pairs = len(inv_freq)
    out = x.copy()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + pairs)
        # long double keeps the angle of far positions
        angle = np.asarray(positions[axes[i]], dtype=np.longdouble) * np.longdouble(inv_freq[i])
        c = np.cos(angle).astype(np.float64)[:, None]
        s = np.sin(angle).astype(np.float64)[:, None]
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
    return out


def mask_first(q_len, k_len, ctx, causal, window_left, window_right, first, row_ranges=None):
    """Dense mask [q_len, k_len]: the window's mask OR the first tokens."""
    mask = visible_mask(np.arange(q_len), k_len, ctx, causal, window_left, window_right, row_ranges)
    open_past = visible_mask(np.arange(q_len), k_len, ctx, causal, -1, window_right, None)
    return mask | (open_past & (np.arange(k_len)[None, :] < first))


def _scores(q, k, h, group, scale, sinks, sink_mode):
    s = scale * (q[:, h, :] @ k[:, h // group, :].T)
    if sink_mode == SINK_KEY0_BIAS and k.shape[0]:
        s[:, 0] += sinks[h]
    return s


def attend(q, k, v, mask, scale, sinks=None, sink_mode=0):
    """One request: out [q_len, Hq, D] and lse [Hq, q_len]."""
    hq, group = q.shape[1], q.shape[1] // k.shape[1]
    out = np.zeros(q.shape)
    lse = np.full((hq, q.shape[0]), -np.inf)
    for h in range(hq):
        s = np.where(mask, _scores(q, k, h, group, scale, sinks, sink_mode), -np.inf)
        m = s.max(axis=1, initial=-np.inf)
        if sink_mode == SINK_NULL_LOGIT:
            m = np.maximum(m, sinks[h])
        m = np.where(np.isfinite(m), m, 0.0)
        e = np.where(mask, np.exp(s - m[:, None]), 0.0)
        z = e.sum(axis=1) + (np.exp(sinks[h] - m) if sink_mode == SINK_NULL_LOGIT else 0.0)
        ok = z > 0
        out[ok, h] = (e[ok] @ v[:, h // group, :]) / z[ok, None]
        lse[h, ok] = m[ok] + np.log(z[ok])
    return out, lse


def key_weights(q, k, lse, mask, scale, sinks=None, sink_mode=0):
    """One request: w [Hkv, k_len], the sum over the rows that see a key and
    over the query heads of its KV head of exp(score - lse).  A row whose lse
    is -inf has no probabilities (it sees nothing, or only scores of -inf)."""
    hq, hkv = q.shape[1], k.shape[1]
    w = np.zeros((hkv, k.shape[0]))
    for h in range(hq):
        s = _scores(q, k, h, hq // hkv, scale, sinks, sink_mode)
        z = np.asarray(lse, dtype=np.float64)[h][:, None]
        seen = mask & (z > -np.inf)
        e = np.exp(np.where(seen, s - np.where(z > -np.inf, z, 0.0), -np.inf))
        w[h // (hq // hkv)] += np.where(seen, e, 0.0).sum(axis=0)
    return w


def evict(weights, n, budget, first, recent):
    """Kept key indices, ascending, of one KV head's weights [>= n]."""
    if n <= budget:
        return np.arange(n)
    fixed = [j for j in range(n) if j < first or j >= n - recent]
    rest = [j for j in range(n) if not (j < first or j >= n - recent)]
    value = {j: (-np.inf if np.isnan(weights[j]) else float(weights[j])) for j in rest}
    best = sorted(rest, key=lambda j: (-value[j], j))[:budget - len(fixed)]
    return np.array(sorted(fixed + best))
