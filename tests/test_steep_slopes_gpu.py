"""Distance biases of any size (GPU): the log-sum-exp of rows whose keys are
weighed by steep slopes, near and far from them.

A key's bias is off by some 13 roundings of 2^-24 of the bias of the first of its
tile's columns (the slope, its products, the steps between groups of columns, the
sums with the score and with the row's maximum): of a key far behind the row
less than 2^-20 of it.  Where the keys that count are near, 8e-4 in log2 units
under gentle slopes, and each bias is rounded by itself under steep ones; and 1e-4
for a sum of powers.
"""

import numpy as np
import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import workloads

from . import gpu_helpers as gh
from .test_scored_gpu import Case, same

pytestmark = pytest.mark.gpu

W = workloads.Workload
NONE, KEY0, NULL = workloads.SINK_NONE, workloads.SINK_KEY0_BIAS, workloads.SINK_NULL_LOGIT


def _check(case):
    out, lse = case.run()
    want = case.oracle()
    gh.compare(out, lse, *want, strict=False)
    seen = np.isfinite(want[1])
    err, size = np.abs(lse.double().cpu().numpy() - want[1])[seen], np.abs(want[1][seen])
    bound = 2.0 ** -20 * size + 9e-4
    assert (err <= bound).all(), (err.max(), size[np.argmax(err - bound)])
    assert same((out, lse), case.run(32))


SLOPES = [[1e3, 30.0, 3.0, -0.02], [1e4, 1e5, 300.0, 0.0], [1e6, 1e8, 1e10, 1e20], [-1e3, -30.0, 2e3, -0.5]]


@pytest.mark.parametrize("cap", [0.0, 9.0])
@pytest.mark.parametrize("slopes", SLOPES)
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_prompts_and_single_tokens(d, slopes, cap):
    w = W("t", 40, [200, 1, 37], [500, 290, 37], 4, 2, d, True, -1, 0, NULL if slopes[0] > 0 else NONE, None)
    _check(Case(w, cap=cap, slopes=slopes))


@pytest.mark.parametrize("cap", [0.0, 9.0])
@pytest.mark.parametrize("slopes", SLOPES)
def test_keys_ahead(slopes, cap):
    w = W("t", 41, [200, 3], [230, 90], 4, 1, 128, False, 150, 40, NONE, None)
    _check(Case(w, cap=cap, slopes=slopes))


@pytest.mark.parametrize("cap", [0.0, 9.0])
@pytest.mark.parametrize("slopes", SLOPES[:3])
def test_first_tokens(slopes, cap):
    w = W("t", 42, [260, 1], [500, 300], 4, 2, 128, True, 40, 0, NONE, None)
    _check(Case(w, cap=cap, slopes=slopes, first=7))


@pytest.mark.parametrize("slopes", [[1e-3, 2e-3, 0.0, -1e-3], [0.02, 0.05, 0.01, -0.02]])
@pytest.mark.parametrize("d", [64, 512])
def test_keys_far_behind(d, slopes):
    """Positions past the keys held: the nearest key's bias is up to 5e3."""
    w = W("t", 43, [140, 1], [300, 250], 4, 2, d, True, -1, 0, NONE, None)
    _check(Case(w, slopes=slopes, ctx=[100_000, 90_000]))


@pytest.mark.parametrize("cap", [0.0, 9.0])
def test_biases_of_any_size_leave_averages(cap):
    """Slopes times distances of up to 3e7, past where fp32 tells neighbours apart: each output lies between the
    values, the log-sum-exp is the nearest key's (within ln 300 and 2^-20)."""
    w = W("t", 44, [140, 1], [300, 250], 4, 2, 128, True, -1, 0, NONE, None)
    case = Case(w, cap=cap, slopes=[0.03, 0.01, 1e-3, -1e-2], ctx=[1_000_000_000, 70_000_000])
    out, lse = case.run()
    assert mvp.get_last_device_error() == 0 and torch.isfinite(out).all()
    assert (out.abs() <= case.v.abs().amax() * (1 + 2.0 ** -7)).all()
    want = case.oracle()[1]
    err = np.abs(lse.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -20 * np.abs(want) + 6.0).all(), err.max()


def test_large_negative_scores_under_first_tokens():
    """Documents under first tokens, without slopes: a row's largest score may be far below 0."""
    w = W("t", 46, [150, 1], [300, 290], 4, 2, 128, True, 60, 0, NONE, None, 0.125)
    case = Case(w, first=3, starts=[[], []])
    case.k = torch.ones_like(case.k) * (60 + torch.arange(590, device=case.dev) % 67)[:, None, None].bfloat16()
    case.q = torch.full_like(case.q, -(2.0 ** 17))
    out, lse = case.run()
    want = case.oracle()[1]
    err = np.abs(lse.double().cpu().numpy() - want)
    assert want.max() < -1e8 and (err <= 2.0 ** -21 * np.abs(want) + 8.0).all(), err.max()
    assert torch.isfinite(out).all() and same((out, lse), case.run(32))


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_large_scores_under_gentle_slopes(d):
    """Scores of up to 2e8 (multiples of one vector, so that each is exact): the row's largest keeps its weight."""
    w = W("t", 45, [150, 1], [300, 290], 4, 2, d, True, -1, 0, NONE, None, 0.125)
    case = Case(w, slopes=[0.5, 0.01, -0.1, 0.0])
    case.k = torch.ones_like(case.k) * (1 + torch.arange(590, device=case.dev) % 97)[:, None, None].bfloat16()
    case.q = torch.full_like(case.q, 2.0 ** 17 * 128 / d)
    out, lse = case.run()
    want = case.oracle()[1]
    err = np.abs(lse.double().cpu().numpy() - want)
    assert np.abs(want).max() > 1e8 and (err <= 2.0 ** -21 * np.abs(want) + 8.0).all(), err.max()  # (+ ln of equals)
    assert torch.isfinite(out).all() and same((out, lse), case.run(32))
