"""Oracle of attention with functions of the score and documents (test
infrastructure, float64).

* ``documents`` -- the closed key interval of the document that a position lies
  in, by a scan over the documents' start positions.
* ``attend``    -- a dense softmax over ``softcap tanh(scale q.k / softcap) -
  slope |p - j|``, key-0 sink or null logit included, where ``mask`` holds and
  the key lies in the row's document.

Written from the definitions; shares no code with the GPU package.
"""

from __future__ import annotations

import numpy as np

from .attention import SINK_KEY0_BIAS, SINK_NULL_LOGIT

LAST = 2 ** 31 - 1


def documents(starts, positions):
    """[rows, 2] closed intervals; ``starts`` of one request, LAST = padding."""
    out = []
    for p in positions:
        lo, hi = 0, LAST - 1
        for s in starts:
            if s <= p:
                lo = max(lo, int(s))
            else:
                hi = min(hi, int(s) - 1)
        out.append((lo, hi))
    return np.array(out, dtype=np.int64).reshape(-1, 2)


def attend(q, k, v, positions, mask, scale, softcap=0.0, slopes=None, doc=None, sinks=None, sink_mode=0):
    """One request: out [q_len, Hq, D] and lse [Hq, q_len]."""
    rows, hq = q.shape[:2]
    group = hq // k.shape[1]
    j = np.arange(k.shape[0])[None, :]
    mask = np.array(mask, dtype=bool)
    if doc is not None:
        mask &= (np.asarray(doc)[:, :1] <= j) & (j <= np.asarray(doc)[:, 1:])
    dist = np.abs(np.asarray(positions, dtype=np.float64)[:, None] - j)
    out = np.zeros(q.shape)
    lse = np.full((hq, rows), -np.inf)
    for h in range(hq):
        kh = np.where(mask.any(0)[:, None], k[:, h // group], 0.0)  # keys that nothing sees may hold anything
        s = scale * (q[:, h] @ kh.T)
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        if slopes is not None:
            s = s - float(slopes[h]) * dist
        if sink_mode == SINK_KEY0_BIAS:
            s = s + float(sinks[h]) * (j == 0)
        s = np.where(mask, s, -np.inf)
        if sink_mode == SINK_NULL_LOGIT:
            s = np.concatenate([s, np.full((rows, 1), float(sinks[h]))], axis=1)
        m = s.max(axis=1, initial=-np.inf)
        m = np.where(np.isfinite(m), m, 0.0)
        e = np.exp(s - m[:, None])
        z = e.sum(axis=1)
        seen = z > 0
        out[seen, h] = (e[seen, :k.shape[0]] @ v[:, h // group]) / z[seen, None]
        lse[h, seen] = m[seen] + np.log(z[seen])
    return out, lse
