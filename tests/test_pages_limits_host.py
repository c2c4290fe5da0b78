"""Lengths and batches at the ends of what the pool's steps take, without a GPU."""

import pytest

import masked_varlen_prefill_gb300 as mvp
from oracle import pages as op

P = 1 << 20


def test_the_oracle_refuses_lengths_past_32_bits():
    top = 2 ** 31 - 1
    width = (top >> 8) + 2
    for n, a, want in ((top - 3, 3, 0), (top - 3, 4, -1), (top, 1, -1), (1, top, -1)):
        refs, rows, lens = [1, 0, 0], [[0] * (width - 1)], [n]
        if want == 0:
            assert op.extend(refs, rows, lens, [a], 256, width)[0] == 0 and lens == [top]
        else:
            assert op.extend(refs, rows, lens, [a], 256, width) == (-1, []) and lens == [n]


@pytest.mark.parametrize("reqs,out", [(1 << 24, 1 << 24), (1 << 20, (1 << 20) + 1)])
def test_fork_refuses_batches_whose_product_is_out_of_reach(reqs, out):
    """Each row of the old batch looks for itself among all parents of the new one."""
    st = mvp.load_library().mvp_kv_fork_paged(P, 8, P, P, reqs, 4, P, out, 2 * P, 4, 2 * P, 16, None)
    assert st == mvp.MVP_ERR_UNSUPPORTED
