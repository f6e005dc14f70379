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
