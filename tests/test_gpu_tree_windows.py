"""GPU: tree attention under a sliding window. Who sees whom by values that count exactly, for
every place of the window's edge in its tile; and infinities and NaN outside the window."""
import os

import numpy as np
import pytest

import tree_reference as ref
from test_gpu_tree_attention import Problem, _count_problem, _say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU (torch.cuda.is_available() is False)")
    import spec_verify_amd as svq
    if not os.path.exists(svq.library_path):
        from spec_verify_amd import build
        build.build()
    svq.lib()
    yield


def _on_device(p):
    names = dict(q=p.q, k=p.k, v=p.v, k_cache=p.caches[0], v_cache=p.caches[1], page_table=p.table, lengths=p.lengths,
                 starts=p.starts, parents=p.parents, k_scale=p.scales[0], v_scale=p.scales[1])
    return {n: x if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()
            for n, x in names.items()}


def _path_trees(p):
    """Every other sequence's explicit tree is a path."""
    for i, (a, n) in enumerate(ref.sequences(p.starts, len(p.q))):
        if i % 2 == 0:
            p.parents[a:a + n] = np.arange(n) - 1


def _shares(p, window, sinks):
    """What a problem of equal weights and unit vectors gives: of every row, the share of each column."""
    out = np.zeros((len(p.q), p.D))
    for s, (a, n) in enumerate(ref.sequences(p.starts, len(p.q))):
        L = int(p.lengths[s])
        paths = ref.paths(None if p.parents is None else p.parents[a:a + n], n)
        depth = np.array([len(x) - 1 for x in paths])
        seen = np.ones((n, L + n), dtype=bool)
        for i, path in enumerate(paths):
            seen[i, L:] = False
            seen[i, [L + j for j in path]] = True
        at = np.concatenate([np.arange(L), L + depth])
        if window > 0:
            seen &= ((L + depth)[:, None] - at < window) | (at < sinks)
        unit = np.eye(p.D)[np.arange(L + n) % p.D]
        out[a:a + n] = seen @ unit / seen.sum(1)[:, None]
    return out


def _check_shares(p, held, window, sinks):
    got = p.svq.tree_attention(**held, window=window, sinks=sinks).double().cpu().numpy()
    want = _shares(p, window, sinks)[:, None]
    # a count over a count: one fp32 reciprocal and product, then bf16
    wrong = np.abs(got - want) > want * (2.0 ** -8 + 2.0 ** -21)
    assert not wrong.any(), (window, sinks, p.H, int(wrong.sum()), np.argwhere(wrong)[:5].tolist())
    assert ((got == 0) == (np.broadcast_to(want, got.shape) == 0)).all(), (window, sinks)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("sinks", [0, 1, 4, 70])
@pytest.mark.parametrize("rows,H", [([16, 40, 64, 7, 33], 1), ([16, 40, 64, 7, 33], 4), ([5, 9, 3], 2)],
                         ids=["blocks-of-32", "blocks-of-128", "blocks-of-16"])
def test_every_place_of_the_edge_in_its_tile(rows, H, sinks, e4m3):
    """(sinks + window - 1) % 64 takes every value, over caches around and far behind the window."""
    _say("edges", rows, H, sinks, e4m3)
    p = _count_problem(rows, [700, 500, 333, 129, 64][:len(rows)], e4m3, H=H, G=1)
    _path_trees(p)
    held = _on_device(p)
    for window in range(65, 129):
        _check_shares(p, held, window, sinks)
    for window in (1, 7, 63, 64, 200, 320):
        _check_shares(p, held, window, sinks)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(128, 4), (1024, 4), (4096, 4), (2000, 4), (65, 0), (512, 4), (128, 1)])
def test_usual_windows_over_long_caches(window, sinks, e4m3):
    _say("window", window, sinks, e4m3)
    p = _count_problem([16, 24, 64], [6000, 4103, 1027], e4m3, H=2, G=1, D=256)
    _path_trees(p)
    _check_shares(p, _on_device(p), window, sinks)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D,H,window,sinks", [(64, 4, 128, 4), (128, 2, 65, 0), (256, 12, 200, 70)])
def test_infinities_and_nan_outside_the_window(D, H, window, sinks, e4m3):
    """Cached tokens that no row's window holds, and the oldest one, which the roots alone see: the other
    rows keep their bits."""
    rows, lengths = [16, 40], [500, 700]
    p = Problem(31, rows, lengths, H=H, G=2, D=D, e4m3=e4m3, window=window, sinks=sinks)
    _path_trees(p)
    held = _on_device(p)
    call = lambda: p.svq.tree_attention(**held, window=window, sinks=sinks).view(torch.int16).cpu()
    clean = call()
    for name, cache in zip(("k_cache", "v_cache"), p.caches):
        for x in [float("nan")] + ([] if e4m3 else [float("inf"), float("-inf")]):
            ugly = cache.clone()
            for s, l in enumerate(lengths):
                for j in range(sinks, l - window + 1):
                    ugly[int(p.table[s, j // p.page]), j % p.page] = x
            _say("outside", name, x)
            held[name] = ugly.cuda()
            assert torch.equal(call(), clean), (name, x)
            for s, l in enumerate(lengths):
                ugly[int(p.table[s, (l - window + 1) // p.page]), (l - window + 1) % p.page] = x
            _say("the oldest", name, x)
            held[name] = ugly.cuda()
            got = call()
            for s, (a, n) in enumerate(ref.sequences(p.starts, sum(rows))):
                for i, path in enumerate(ref.paths(p.parents[a:a + n], n)):
                    same = torch.equal(got[a + i], clean[a + i])
                    assert same == (len(path) > 1), (name, x, s, i)
        held[name] = cache.cuda()
