"""Capped scores over the whole range of ``softcap / scale`` (GPU), packed and
paged, prompts and single tokens.

Keys are multiples b of one vector of +-1 and rows multiples a of the same, so that
every score is scale D a b exactly, whatever the order of its sum.  ``top`` is the
largest score over the cap.  The log-sum-exp is then off by what the functions
are: 9e-7 of a score by the cap, some ten roundings of 2^-24 of it (the scale, the
cap's factor, the exponent, the logarithm), in all less than 4e-6 of the largest;
and 1e-4 for a sum of up to 400 approximate powers (400 * 2^-24 + 2 * 2^-22 < 3e-5).
"""

import numpy as np
import pytest
import torch

from masked_varlen_prefill_gb300 import workloads

from . import gpu_helpers as gh
from .test_scored_gpu import Case, same

pytestmark = pytest.mark.gpu

W = workloads.Workload
NONE, KEY0 = workloads.SINK_NONE, workloads.SINK_KEY0_BIAS


def _case(d, cap, scale, top, seed=0, window=-1, sink=NONE, **kw):
    w = W("t", 30 + seed, [130, 1, 37], [300, 290, 37], 4, 2, d, True, window, 0, sink, None, scale)
    case = Case(w, cap=cap, **kw)
    rng = np.random.RandomState(seed)
    sign = rng.choice([-1.0, 1.0], d)
    # the bf16 numbers of four binades, no two keys of a request alike: none comes nearer than 2^-8 to the largest
    levels = np.concatenate([(1 + np.arange(128) / 128) * 2.0 ** e for e in range(-4, 0)])
    b = np.concatenate([rng.permutation(levels)[:n] * rng.choice([-1.0, 1.0, 1.0], n) for n in w.k_lens])
    a = rng.randint(64, 129, (w.total_q, w.num_heads_q)) / 128
    raw = top * cap / scale / d  # the largest product a b
    half = 2.0 ** np.round(np.log2(raw) / 2)
    t = lambda x: torch.tensor(x, device=case.dev).bfloat16()  # noqa: E731
    case.q = t(raw / half * a[:, :, None] * sign)
    case.k = t(np.repeat(half * b[:, None, None] * sign, w.num_heads_kv, axis=1))
    assert abs(case.q).max().isfinite() and abs(case.k).max().isfinite() and (case.q != 0).all() and (case.k != 0).all()
    return case


def _check(case, cap, top, more=0.0):
    """``more``: what else a score may be off by."""
    out, lse = case.run()
    want = case.oracle()
    gh.compare(out, lse, *want, strict=False)
    err = np.abs(lse.double().cpu().numpy() - want[1])
    largest = cap * np.tanh(top) * (1 + 2.0 ** -7)
    assert err.max() <= 4e-6 * largest + 1e-4 + more, (err.max(), largest)
    assert same((out, lse), case.run(16))


RANGES = [
    # factors of s^2 whose powers leave fp32's range below
    (30.0, 1e-4, 0.74), (30.0, 1e-5, 0.49), (30.0, 1e-5, 0.74), (30.0, 1e-6, 0.49), (30.0, 1e-6, 0.74),
    (30.0, 1e-8, 0.27), (30.0, 1e-8, 0.74), (30.0, 1e-10, 0.27), (30.0, 1e-10, 0.49), (30.0, 1e-12, 2.0),
    # squares that leave it above
    (1e20, 0.125, 0.27), (1e25, 0.125, 0.27), (1e25, 0.125, 0.74), (1e30, 0.125, 0.49), (1e30, 1.0, 1e-8),
    (1e30, 1.0, 1e-14), (1e30, 1e-6, 0.01),
    # factors that leave it above
    (1e-3, 1e3, 0.74), (1e-3, 1e3, 0.27), (1e-20, 1e6, 0.49), (1e-2, 1e2, 0.74),
    # and none that does
    (30.0, 0.125, 0.27), (30.0, 0.125, 0.49), (30.0, 0.125, 0.74), (1000.0, 0.05, 0.74), (50.0, 2e-3, 0.74),
]


@pytest.mark.parametrize("cap,scale,top", RANGES)
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_caps_over_scales(d, cap, scale, top):
    _check(_case(d, cap, scale, top), cap, top)


@pytest.mark.parametrize("cap,scale,top", RANGES[:10])
def test_caps_over_scales_with_a_bias(cap, scale, top):
    """(Slopes of cap / 3000: biases of up to a tenth of the cap, each rounding 2^-24 of it.)"""
    case = _case(128, cap, scale, top, seed=1, slopes=cap / 3000 * np.array([1.0, 0.5, -0.25, 0.0]))
    _check(case, cap, top, more=0.1 * cap * 16 * 2.0 ** -24)


@pytest.mark.parametrize("cap,scale,top", RANGES[:17])
def test_caps_over_scales_under_first_tokens(cap, scale, top):
    _check(_case(64, cap, scale, top, seed=2, window=50, first=5), cap, top)


@pytest.mark.parametrize("window", [-1, 50])
@pytest.mark.parametrize("cap,scale,top", RANGES[10:17])
def test_wide_caps_with_a_bias(cap, scale, top, window):
    """(Keys whose sums of score and bias nearly meet: which of them wins is open, their log-sum-exp is not.)"""
    case = _case(128, cap, scale, top, seed=3, window=window, slopes=cap * top / 3000 * np.array([1.0, 0.5, -0.25, 0.0]))
    out, lse = case.run()
    want = case.oracle()[1]
    err = np.abs(lse.double().cpu().numpy() - want)
    assert torch.isfinite(out).all() and (out.abs() <= case.v.abs().amax() * (1 + 2.0 ** -7)).all()
    assert err.max() <= 4e-6 * cap * np.tanh(top) * 1.2, (err.max(), cap)
    assert same((out, lse), case.run(16))
