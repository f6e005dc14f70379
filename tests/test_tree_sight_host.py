"""Who sees whom in tree attention, without a GPU: the arithmetic of the masks, compiled for the
host from the kernels' own header, against the definition, token by token."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import tree_reference as ref

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "spec_verify_amd", "csrc")
CHAIN, PATHS, WALK = 0, 1, 2


@pytest.fixture(scope="module")
def sight(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    lib = str(tmp_path_factory.mktemp("sight") / "sight.so")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "sight_host.cpp"), "-o", lib], check=True)
    return ctypes.CDLL(lib).sight


def _tree(rng, n, shape):
    if shape == "chain":
        return np.arange(n, dtype=np.int32) - 1
    if shape == "wild":  # entries that name nothing among them
        return rng.integers(-3, n + 2, n).astype(np.int32)
    return np.array([i - 1 - int(rng.random() ** 2 * i) for i in range(n)], dtype=np.int32)


def _check(sight, how, parents, length, window, first, shift=0):
    """All tiles of one sequence; shift: the first begins at that number (the chunk's rows have tiles of their own
    behind an 8-bit cache, from number `cached` on: -1)."""
    n = len(parents)
    paths = ref.paths(None if how == CHAIN else parents, n)
    depth = np.array([len(p) - 1 for p in paths])
    row_at = length + depth
    own = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(paths):
        own[i, p] = True
    pos = np.arange(length)
    cached = np.ones((n, length), dtype=bool)
    if window > 0:
        cached = (row_at[:, None] - pos < window) | (pos < first)
        own &= (row_at[:, None] - row_at < window) | (row_at < first)
    places = np.full(max(length, 1), -1, dtype=np.int32)
    par = np.ascontiguousarray(parents, dtype=np.int32)

    def masks(begin, tiles):
        words, needs = np.zeros((tiles, n), dtype=np.uint64), np.zeros(tiles, dtype=np.int32)
        p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
        count = sight(how, n, p(par), length, window, first, begin, tiles, p(words), p(needs), p(places))
        bits = np.unpackbits(words.view(np.uint8).reshape(tiles, n, 8), axis=2, bitorder="little").astype(bool)
        return count, bits.transpose(1, 0, 2).reshape(n, tiles * 64), needs
    count, _, _ = masks(0, 0)
    case = (how, n, length, window, first, parents.tolist())
    at = places[:count]
    assert (np.diff(at) > 0).all(), case
    hidden = np.ones(length, dtype=bool)
    hidden[at] = False
    assert not cached[:, hidden].any(), case   # what has no number is seen by no row
    begin = count if shift < 0 else 0
    tiles = (count + n - begin + 63) // 64
    _, bits, needs = masks(begin, tiles)
    want = np.zeros((n, begin + tiles * 64), dtype=bool)
    want[:, :count] = cached[:, at]
    want[:, count:count + n] = own
    want = want[:, begin:]
    wrong = bits != want
    assert not wrong.any(), (case, np.argwhere(wrong)[:5].tolist(), int(wrong.sum()))
    for k in range(tiles):
        assert needs[k] or want[:, 64 * k:64 * k + 64].all(), (case, k)


HOWS = [("chain", CHAIN), ("chain", PATHS), ("tree", PATHS), ("wild", PATHS), ("chain", WALK), ("tree", WALK), ("wild", WALK)]


@pytest.mark.parametrize("first", [0, 1, 4, 70])
@pytest.mark.parametrize("shape,how", HOWS)
def test_every_place_of_a_windows_edge_in_its_tile(sight, shape, how, first):
    """(first + window - 1) % 64 takes every value, with caches around and far behind the window."""
    rng = np.random.default_rng(first)
    for window in list(range(1, 20)) + list(range(60, 130)):
        for n, length in ((16, 5 * 64 + window), (64, 700), (7, window), (33, window + 63), (1, 300), (40, 200)):
            _check(sight, how, _tree(rng, n, shape), length, window, first)


@pytest.mark.parametrize("window,first", [(128, 4), (1024, 4), (4096, 4), (2000, 4), (65, 0), (512, 4), (128, 1), (512, 1),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0), (64, 2 ** 31 - 1), (0, 5), (-3, 9)])
@pytest.mark.parametrize("shape,how", HOWS)
def test_usual_windows_over_long_caches(sight, shape, how, window, first):
    rng = np.random.default_rng(7)
    for n, length in ((16, 6000), (64, 5000), (24, 4103), (5, 1027), (9, 64), (3, 0), (63, 1)):
        _check(sight, how, _tree(rng, n, shape), length, window, first)
        _check(sight, how, _tree(rng, n, shape), length, window, first, shift=-1)


def test_any_tree_window_and_length(sight):
    rng = np.random.default_rng(11)
    for _ in range(4000):
        shape, how = HOWS[rng.integers(len(HOWS))]
        n = int(rng.integers(1, 65))
        length, window = (int(x) for x in np.exp(rng.uniform(0, np.log([3000, 2000]))) - 1)
        _check(sight, how, _tree(rng, n, shape), length, window, int(rng.integers(0, 71)), shift=-int(rng.integers(0, 2)))


@pytest.mark.parametrize("shape", ["chain", "tree", "wild"])
def test_trees_of_more_than_64_nodes(sight, shape):
    rng = np.random.default_rng(13)
    for n in (65, 130, 400):
        for window, first in ((0, 0), (40, 3), (100, 0), (128, 4), (300, 70), (1000, 4)):
            for length in (0, 63, 500):
                _check(sight, WALK, _tree(rng, n, shape), length, window, first, shift=-int(rng.integers(0, 2)))
    _check(sight, CHAIN, np.zeros(400, dtype=np.int32), 500, 100, 4)
