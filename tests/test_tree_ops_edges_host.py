"""The operators of a tree of drafts without a GPU: calls at the ends of what their entry points take."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

from test_tree_ops_host import L, P, _adjust, _attend  # noqa: F401 (L is the library's fixture)

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "spec_verify_amd", "csrc")


def test_columns_of_one_matrix_that_share_none(tmp_path):
    """The check of the entry points, compiled from their header, against sets of elements."""
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    lib = str(tmp_path / "check.so")
    source = ('#include "svq_check.h"\nextern "C" int apart(int64_t a, int64_t na, int64_t b, int64_t nb, int64_t ld) '
              '{ return svq::columns_apart((void *)(2 * a), na, (void *)(2 * b), nb, ld); }\n')
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-x", "c++", "-", "-o", lib],
                   input=source.encode(), check=True)
    apart = ctypes.CDLL(lib).apart
    apart.argtypes = [ctypes.c_int64] * 5
    rows, a = 40, 100
    for ld in (1, 5, 8):
        for na in range(1, ld + 1):
            for nb in range(1, ld + 1):
                ours = {a + i * ld + c for i in range(rows) for c in range(na)}
                for b in range(a - 2 * ld, a + 2 * ld + 1):
                    theirs = {b + i * ld + c for i in range(rows) for c in range(nb)}
                    assert bool(apart(a, na, b, nb, ld)) == ours.isdisjoint(theirs), (ld, na, nb, b - a)


@pytest.mark.parametrize("at,ld", [(1016, 2048), (1032, 2048), (512, 4096), (3600, 4096), (2048, 2048), (8, 1024)])
@pytest.mark.parametrize("side", [1, -1])
def test_out_that_shares_columns_with_q_is_refused(L, at, ld, side):  # noqa: F811
    """1024 columns of q and of out, the one `at` columns behind the other, in a matrix of `ld` columns."""
    q, out = (P[4], P[4] + 2 * at) if side > 0 else (P[4] + 2 * at, P[4])
    assert _attend(L, q=q, ldq=ld, out=out, ldo=ld) == 7


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_strides_and_workspaces_beside_columns(L, name):  # noqa: F811
    """Columns apart, but of rows of other strides, and a workspace among them."""
    p = dict(q=P[4], k=P[5], v=P[6])[name]
    assert _attend(L, out=p + 2 * 1024, ldo=4104, **{name: p, "ld" + name: 4096}) == 7
    assert _attend(L, out=p + 2 * 1024, ldo=4096, ws=p + 512, **{name: p, "ld" + name: 4096}) == 7


@pytest.mark.parametrize("name,at", [("k", 504), ("k", 3600), ("v", 8), ("v", 4088)])
def test_out_that_shares_columns_with_keys_or_values_is_refused(L, name, at):  # noqa: F811
    """out, 1024 columns, begins `at` columns behind k's or v's 512, in a matrix of 4096."""
    p = P[5] if name == "k" else P[6]
    assert _attend(L, out=p + 2 * at, ldo=4096, **{name: p, "ld" + name: 4096}) == 7


@pytest.mark.parametrize("at,ld", [(999, 2000), (1, 2000), (1001, 2000), (2000, 2000), (0, 2008), (500, 1000), (999, 1999)])
@pytest.mark.parametrize("side", [1, -1])
def test_adjusted_logits_that_share_columns_are_refused(L, at, ld, side):  # noqa: F811
    """out's 1000 columns begin `at` behind the logits' 1000, or before: some columns are both's."""
    a, b = (P[13], P[13] + 2 * at) if side > 0 else (P[13] + 2 * at, P[13])
    assert _adjust(L, logits=a, ld=ld, out=b, ldo=ld if at else ld - 8) == 7


@pytest.mark.parametrize("pages,status", [((1 << 24) - 3, 8), ((1 << 24) - 2, 2)])
def test_steps_stay_below_31_bits(L, pages, status):  # noqa: F811
    """128 heads, one row, pages of a tile: 2^24 tiles would be 2^31 steps, one more than are counted. (Without a
    workspace, what is otherwise valid ends with status 8.)"""
    assert _attend(L, ws=None, M=1, S=1, H=128, G=128, D=64, ldq=8192, ldk=8192, ldv=8192, ldo=8192, page_size=64,
                   max_pages=pages, ld_table=pages, k0=1 << 19, k1=8192, k2=64, v0=1 << 19, v1=8192, v2=64) == status
