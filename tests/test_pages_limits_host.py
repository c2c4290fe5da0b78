"""Lengths and batches at the ends of what the pool's steps take, without a GPU."""

from oracle import pages as op


def test_the_oracle_refuses_lengths_past_32_bits():
    top = 2 ** 31 - 1
    width = (top >> 8) + 2
    for n, a, want in ((top - 3, 3, 0), (top - 3, 4, -1), (top, 1, -1), (1, top, -1)):
        refs, rows, lens = [1, 0, 0], [[0] * (width - 1)], [n]
        if want == 0:
            assert op.extend(refs, rows, lens, [a], 256, width)[0] == 0 and lens == [top]
        else:
            assert op.extend(refs, rows, lens, [a], 256, width) == (-1, []) and lens == [n]
