"""GPU: calls of the operators of a tree of drafts that stand at the ends of what their
documentation allows."""
import os

import numpy as np
import pytest

import tree_reference as ref
import test_gpu_adjust_logits as logits
from test_gpu_tree_attention import Problem, _say

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


def _bits(t):
    return t.contiguous().view(torch.int16).cpu()


@pytest.mark.parametrize("rows,H,D", [([13, 40], 6, 64), ([5], 12, 256), ([64, 30], 4, 128)])
def test_attention_into_other_columns_of_the_projections_matrix(rows, H, D):
    """One matrix holds q, k, v and out side by side."""
    _say("beside", rows, H, D)
    p = Problem(41, rows, [300, 70][:len(rows)], H=H, G=2, D=D)
    want = _bits(p.call())
    M, G = len(p.q), 2
    for order in ("qkvo", "oqkv", "kovq"):
        parts = dict(q=p.q, k=p.k, v=p.v, o=torch.full((M, H, D), 7.0).bfloat16())
        wide = torch.cat([parts[c].reshape(M, -1) for c in order], 1).cuda()
        cols = dict(zip(order, wide.split([parts[c].shape[1] * D for c in order], 1)))
        view = {c: x.view(M, -1, D) for c, x in cols.items()}
        p.call(q=view["q"], k=view["k"], v=view["v"], out=view["o"])
        assert torch.equal(_bits(view["o"]), want), order
        for c in "qkv":
            assert torch.equal(_bits(view[c]), _bits(parts[c])), (order, c)


@pytest.mark.parametrize("V,apart", [(1000, 1000), (1001, 1001), (1001, 1010), (77, 80), (40000, 40001)])
def test_adjusted_logits_into_other_columns_of_their_matrix(V, apart):
    _say("beside", V, apart)
    p = logits.Problem(42, [5, 9], [60, 20], V, biases=10, masks=2)
    want = _bits(p.call())
    M = len(p.logits)
    for first, second in ((0, apart), (apart, 0)):
        wide = torch.full((M, apart + V + 3), 3.0, dtype=torch.bfloat16, device="cuda")
        src, out = wide[:, first:first + V], wide[:, second:second + V]
        src.copy_(p.logits)
        p.call(src, out=out)
        assert torch.equal(_bits(out), want)
        assert torch.equal(_bits(src), _bits(p.logits))
        for c in (src, out):
            c.fill_(3.0)
        assert (wide == 3.0).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_infinities_and_nan_in_q_at_a_scale_of_zero(e4m3):
    """0 times an infinite or undefined product is NaN, and the other rows and heads weigh everything alike."""
    p = Problem(43, [20, 9], [200, 64], H=4, G=2, D=64, e4m3=e4m3)
    p.q[3, 1, 5], p.q[7, 0, 63], p.q[25, 3, 0] = float("inf"), float("-inf"), float("nan")
    hit = np.zeros(p.q.shape[:2], dtype=bool)
    hit[3, 1] = hit[7, 0] = hit[25, 3] = True
    for scale in (0.0, -0.0):
        _say("scale", scale)
        got = p.call(scale=scale).double().cpu().numpy()
        want, bound, _ = p.expected(scale=scale)
        assert np.isnan(want[hit]).all() and np.isnan(got[hit]).all()
        assert (np.abs(got - want) <= bound)[~hit].all()


@pytest.mark.parametrize("scale,by", [(1e-30, 1e-30), (1e-20, 1e-25), (-1e-30, 1e-30), (1e-30, 0.01)])
def test_scales_whose_product_32_bits_do_not_hold(scale, by):
    """The caller's scale times the keys' is 0 in fp32: all that a row sees weighs alike, the rest nothing."""
    p = Problem(44, [20, 9], [200, 64], H=4, G=2, D=64, e4m3=True)
    p.scales[0] = torch.full((2,), by)
    _say("scales", scale, by)
    got = p.call(scale=scale).double().cpu().numpy()
    want, bound, _ = p.expected(scale=scale)
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("rows,length,H,D,tree", [([1], 1500, 2, 64, False), ([5], 20000, 4, 128, False), ([16, 40], 700, 4, 64, True),
                                                  ([24], 2500, 6, 256, True), ([3, 2], 20, 2, 64, True)])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_infinite_and_undefined_values_whatever_their_weight(rows, length, H, D, tree, e4m3):
    """A seen value that is infinite or NaN leaves its column of the row infinite or NaN, though its weight is
    less than fp32 holds or 0, wherever it stands among masked tiles, whole ones and parts; other columns are as
    if it were finite."""
    p = Problem(45, rows, [length] * len(rows), H=H, G=2, D=D, e4m3=e4m3, tree=tree)
    n = len(rows)
    places = sorted({0, 1, length // 3, length // 2, length - 2, length - 1})
    p.q[:] = p.q.abs() + 0.5
    # the token that takes all the weight: the scores of others are hundreds of powers of two below
    for peak in (places[1], places[-2], None):
        keys = p.caches[0].clone()
        for s in range(n):
            if peak is not None:
                keys[p.table[s, peak // p.page], peak % p.page] = 400.0 if e4m3 else 100.0
            elif not e4m3:  # scores of -inf
                for j in places:
                    keys[p.table[s, j // p.page], j % p.page] = float("-inf")
        keep, p.caches[0] = p.caches[0], keys
        want, bound, _ = p.expected()
        p.caches[0] = keep
        odd = [i for i, j in enumerate(places) if j != peak]
        fine = [i for i in range(D) if i not in odd]
        for x in [float("nan")] if e4m3 else [float("inf"), float("-inf"), float("nan")]:
            values = p.caches[1].clone()
            for i in odd:
                j = places[i]
                for s in range(n):
                    values[p.table[s, j // p.page], j % p.page, :, i] = x
            _say("values of", x, "peak", peak, "at", places)
            got = p.call(k_cache=keys.cuda(), v_cache=values.cuda()).double().cpu().numpy()
            assert not np.isfinite(got[:, :, odd]).any()
            assert (np.abs(got - want) <= bound)[:, :, fine].all()


def test_a_row_that_sees_scores_of_minus_infinity_alone():
    """Zero where the values are finite; a column with an infinite or undefined one is not."""
    for rows, length in (([3], 70), ([5], 3000), ([1], 64)):
        p = Problem(46, rows, [length], H=2, G=1, tree=False)
        p.q[:] = p.q.abs() + 0.1
        p.caches[0][:] = float("-inf")
        p.k[:] = float("-inf")
        p.caches[1][p.table[0, 1], 3, 0, 7] = float("inf")
        got = p.call().float().cpu()
        assert not torch.isfinite(got[:, :, 7]).any()
        got[:, :, 7] = 0
        assert (got == 0).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 2)])
def test_a_pool_of_no_pages_and_a_table_of_none(e4m3, window, sinks):
    """Rows see their paths alone, whatever the lengths say; with a table there is nothing that it could name."""
    p = Problem(47, [9, 70, 1], [50, 0, 3], H=4, G=2, D=64, e4m3=e4m3, window=window, sinks=sinks)
    none = [c[:0] for c in p.caches]
    _say("no pages", window, sinks)
    named = p.call(k_cache=none[0].cuda(), v_cache=none[1].cuda())   # lengths count, for a window too
    p.table[:] = -1
    assert torch.equal(_bits(named), _bits(p.call()))
    p.check("a table that names nothing", named, overall=False)
    bare = p.call(k_cache=none[0].cuda(), v_cache=none[1].cuda(), page_table=p.table[:, :0])
    p.lengths[:] = 0
    p.check("no table", bare, overall=False)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows,lengths", [([100, 300], [2000, 130]), ([64, 20], [4000, 90])])
def test_missing_pages_before_wide_trees(rows, lengths, e4m3):
    """Tiles with tokens that are not there, far before the chunk's rows."""
    p = Problem(48, rows, lengths, H=2, G=1, D=64, e4m3=e4m3)
    p.table[0, 3::7] = -1
    p.table[1, 1] = len(p.caches[0])
    p.check(f"missing pages, {rows}")
