"""GPU tests of kept rows whose pages are not there: the row is skipped and recorded, whatever the table's
entry is, and every other row moves."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import paged
from oracle.softmax_attention import host64
from tests.paged_cases import cache, ints

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
PAGE, NODES = 8, 40


def check(recorded, entry=None, at=0, start=3, path=(0, 9, 17, 30, 38), rows=None, counts=None, dtype="bf16", d=64):
    """Two sequences, the first with the given table entry; every element against the oracle."""
    kc, vc, table = cache(2, 3, d, PAGE, [3 + NODES, 5 + NODES], dtype=dtype, device=DEV, seed=2)
    if rows is not None:  # a table that ends early
        table = table[:, :rows // PAGE].contiguous()
    if entry is not None:
        table[0, at] = kc.shape[0] if entry == "pages" else entry
    paths = np.array([path, np.arange(len(path))])
    want = paged.keep(kc, vc, table.tolist(), (start, 5), paths, counts)
    lf.cache_keep(kc, vc, table, ints([start, 5], DEV), ints(paths.tolist(), DEV),
                  counts=None if counts is None else ints(counts, DEV))
    torch.cuda.synchronize()
    assert (lf.linformer_debug_read_device_status() != 0) == recorded
    for x, y in zip((kc, vc), want):
        assert np.array_equal(host64(x), y, equal_nan=True)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 64), ("bf16", 5)])
@pytest.mark.parametrize("entry", [-1, -2, -3, -2 ** 31, "pages", 2 ** 31 - 1])
def test_pages_that_are_not_there(entry, dtype, d):
    kw = dict(dtype=dtype, d=d)
    check(True, entry, at=4, **kw)    # the source of row 3 alone (rows 32 to 39)
    check(True, entry, at=0, **kw)    # targets
    check(True, entry, at=1, path=(0, 1, 2, 3, 4, 20), **kw)  # the last target
    check(False, entry, at=3, **kw)   # rows that nothing moves from or to
    check(False, entry, at=0, path=(0, 1, 2, 3), **kw)        # rows in their places
    check(False, entry, at=4, counts=(3, 5), **kw)            # behind the count


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_the_table_does_not_hold(dtype):
    check(True, rows=40, path=(0, 9, 37, 38), dtype=dtype)          # sources behind its end
    check(True, rows=40, path=(0, 9, 2 ** 31 - 1, 12), dtype=dtype)
    check(True, rows=16, start=14, path=(0, 1, 5), dtype=dtype)     # and a target
    check(True, rows=40, start=-2, path=(1, 5, 9, 12), dtype=dtype)  # before its beginning
    check(True, rows=40, start=-2 ** 31, path=(1, 5, 9, 12), dtype=dtype)
    check(False, rows=40, path=(0, 9, 36), dtype=dtype)
