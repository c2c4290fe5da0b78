"""Lengths at the ends of what the pool's steps take (GPU)."""

import pytest
import torch

import masked_varlen_prefill_gb300 as mvp

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("n,a,missing", [(TOP - 3, 3, 0), (TOP - 3, 4, -1), (TOP - 300, 400, -1), (TOP, TOP, -1),
                                         (7, TOP, -1)])
def test_extend_keeps_lengths_in_32_bits(n, a, missing):
    """A table of more than 2^31 tokens a row: lengths past that are refused, not wrapped, and nothing changes."""
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    width = (TOP >> 8) + 2
    table = torch.zeros((2, width), dtype=torch.int32, device="cuda")
    table[1, 0] = 1
    refs, caches = t(1, 1, 0, 0, 0, 0), torch.zeros((6, 256, 1, 64), dtype=torch.bfloat16, device="cuda")
    lens, lack = t(n, 256), t(77)
    new = torch.zeros_like(lens)
    ws = torch.empty(mvp.kv_extend_workspace_size(2), dtype=torch.uint8, device="cuda")
    mvp.kv_extend_paged(mvp.kv_caches([caches], 256), refs, table, lens, t(a, 1), new, lack, ws)
    assert int(lack) == missing
    if missing == 0:
        assert new.tolist() == [n + a, 257] and refs.tolist() == [1, 1, 1, 0, 0, 0] and int(table[1, 1]) == 2
    else:
        assert new.tolist() == [n, 256] and refs.tolist() == [1, 1, 0, 0, 0, 0] and not table[1, 1:].any()
    assert not table[0].any() and not caches.any()
