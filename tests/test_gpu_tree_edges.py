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
