"""Moves whose written rows meet other written rows or any source rows are refused on the host, before
a launch (the addresses are never touched)."""
import ctypes

import pytest

from sparse_attention_lightning_indexer_gb300 import build, ds4idx

P = 1 << 20
ROW = 16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ds4idx.load()


def _move(lib, src_starts, lens, dst_starts, counts, arrays):
    """arrays: (src, dst, src_rows, dst_rows) in rows of 16 bytes, src and dst as rows from P."""
    def i64(v):
        return ctypes.cast((ctypes.c_int64 * len(v))(*v), ctypes.c_void_p)
    a = (ds4idx.RowArray * len(arrays))(*[
        ds4idx.RowArray(src=P + s * ROW, dst=P + d * ROW, src_rows=sr, dst_rows=dr, row_bytes=ROW)
        for s, d, sr, dr in arrays])
    return lib.ds4idx_evict_compact(P, max(counts), len(lens), i64(src_starts), i64(lens),
                                    i64(dst_starts), i64(counts), len(arrays),
                                    ctypes.cast(a, ctypes.c_void_p), None)


@pytest.mark.parametrize("what,args", [
    ("two sequences, one row of overlap",
     ([0, 50], [50, 50], [0, 9], [10, 10], [(0, 1000, 100, 100)])),
    ("two sequences, the later one first",
     ([0, 50], [50, 50], [9, 0], [10, 10], [(0, 1000, 100, 100)])),
    ("two sequences, the same start",
     ([0, 50], [50, 50], [7, 7], [10, 1], [(0, 1000, 100, 100)])),
    ("one inside a longer one, another between",
     ([0, 50, 60], [50, 10, 10], [0, 40, 20], [30, 5, 5], [(0, 1000, 100, 100)])),
    ("two arrays, one destination",
     ([0], [50], [0], [10], [(0, 1000, 100, 100), (200, 1000, 100, 100)])),
    ("a destination over another array's source",
     ([0], [50], [0], [10], [(0, 1000, 100, 100), (1005, 2000, 100, 100)])),
    ("a destination over another array's source, of a sequence that keeps nothing",
     ([0, 50], [50, 50], [0, 0], [10, 0], [(0, 1040, 100, 100), (1000, 2000, 100, 100)])),
    ("a destination over its own array's source",
     ([0], [50], [49], [10], [(0, 0, 100, 100)])),
    ("the source behind it",
     ([60], [40], [55], [6], [(0, 0, 100, 100)])),
])
def test_refused(lib, what, args):
    assert _move(lib, *args) == ds4idx.ERR_INVALID_ARG, what
