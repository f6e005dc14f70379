"""The per-request operators without a GPU: their workspaces and the calls at the ends of
what their entry points take."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

BAD = ctypes.c_size_t(-1).value
COUNTERS = 256 * 1024  # a workspace's first bytes, the GEMMs' arrival counters


@pytest.fixture(scope="module")
def L():
    import spec_verify_amd as svq
    if not os.path.exists(svq.library_path):
        from spec_verify_amd import build
        build.build()
    return svq.lib()


def test_the_parts_of_a_sampled_row_begin_on_cache_lines(L):
    """A part's header and list are read and written in 16-byte pieces: every part of the
    workspace is a whole number of 128-byte lines. (M, V: rows split in 8, 5 and 65 parts.)"""
    for M, V, parts in ((1, 248320, 8), (3, 248320, 8), (51, 248320, 5), (1, 1 << 24, 65)):
        v = L.svq_sample_workspace_bytes(M, V)
        assert v != BAD and v > COUNTERS
        assert (v - COUNTERS) % (M * parts) == 0, (M, V, v)
        assert (v - COUNTERS) // (M * parts) % 128 == 0, (M, V, v)


@pytest.mark.parametrize("ld,columns", [(512, 8), (512, 248), (512, 264), (512, 504), (504, 256), (256, 256), (512, 512 * 3 + 8)])
def test_column_slices_that_share_columns_are_refused(L, ld, columns):
    """out begins `columns` elements behind base, in a matrix of `ld` columns, N = 256: some
    of out's columns are base's."""
    p = [(i + 1) << 40 for i in range(8)]
    for there, back in ((p[0], p[0] + 2 * columns), (p[0] + 2 * columns, p[0])):
        got = L.svq_adapter_add(there, ld, p[1], p[2], p[3], p[4], p[5], back, ld, 5, 256, 512, 16, 4, p[7], 1 << 30, None)
        assert got == 7, (ld, columns, got)
