"""Pins of the kept rows' oracle where pages are missing: those rows stay, all others move."""
import numpy as np
import pytest

from oracle import paged
from oracle.softmax_attention import host64
from tests.paged_cases import cache


@pytest.mark.parametrize("entry", [-1, -2, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_oracle_skips_rows_whose_page_is_missing(entry, at):
    """Rows 1, 2 and 3 of page 0 come from rows 17, 9 and 18, of pages 2, 1 and 2."""
    kc, vc, table = cache(1, 2, 8, 8, [24], seed=1)
    path, source = [0, 17, 9, 18], {1: 17, 2: 9, 3: 18}
    before = host64(kc)
    gone = table.tolist()
    gone[0][at] = entry
    new = paged.keep(kc, vc, gone, (0,), np.array([path]))[0]
    rows, old = paged.rows(new, table.tolist()[0], 24), paged.rows(before, table.tolist()[0], 24)
    moved = [i for i in source if at not in (0, source[i] // 8)]
    for i in range(24):
        assert np.array_equal(rows[:, i], old[:, source[i] if i in moved else i])


def test_oracle_skips_rows_outside_the_table():
    kc, vc, table = cache(1, 1, 8, 8, [24], seed=1)
    old = paged.rows(host64(kc), table.tolist()[0], 24)
    for start, path, moved in ((0, [0, 24, 23], {2: 23}), (-1, [1, 5, 7], {0: 4, 1: 6}), (22, [1, 2], {22: 23})):
        rows = paged.rows(paged.keep(kc, vc, table.tolist(), (start,), np.array([path]))[0], table.tolist()[0], 24)
        for i in range(24):
            assert np.array_equal(rows[:, i], old[:, moved.get(i, i)])
