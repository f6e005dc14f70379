"""GPU: low-rank adapters where a value, a rank or a launch shape is at an end: infinities
beside padded ranks, on both sides of the rule that chooses one launch or two."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU (torch.cuda.is_available() is False)")
    import os
    import spec_verify_amd as svq
    if not os.path.exists(svq.library_path):
        from spec_verify_amd import build
        build.build()
    svq.lib()
    yield


def _say(*a):
    print("[gpu]", *a, flush=True)
    sys.stdout.flush()


def _call(p, **kw):
    import spec_verify_amd as svq
    d = {k: v.cuda() for k, v in p.items()}
    return svq.adapter_add(d["base"], d["x"], d["a"], d["b"], d["rows"], d["scales"], **kw).cpu()


# K of either side of the bound of one launch (16 ranks a tile: 2560, 32: 1280); ranks that
# fill their tiles and that do not
@pytest.mark.parametrize("K,R", [(640, 8), (640, 24), (640, 16), (640, 32), (2560, 8), (2688, 8), (1280, 24), (1408, 24)])
def test_an_infinity_is_a_rows_own_whatever_the_rank(K, R):
    """a, b and scale positive: one +inf or -inf in a row of x makes that row's outputs the
    same infinity, and no padded rank turns it into NaN."""
    _say("adapter infinity", K, R)
    g = torch.Generator().manual_seed(K + R)
    M, N, slots = 5, 48, 2
    pos = lambda *s: (torch.rand(*s, generator=g) + 0.5).bfloat16()
    p = dict(base=torch.randn(M, N, generator=g).bfloat16(), x=pos(M, K), a=pos(slots, R, K), b=pos(slots, N, R),
             rows=torch.tensor([0, 1, 0, -1, 1], dtype=torch.int32), scales=torch.tensor([0.5, 2.0]))
    clean = _call(p)
    assert bool(clean.isfinite().all())
    p["x"][2, 77] = float("inf")
    p["x"][4, K - 1] = -float("inf")
    got = _call(p)
    assert bool((got[2] == float("inf")).all()) and bool((got[4] == -float("inf")).all())
    assert torch.equal(got[[0, 1, 3]], clean[[0, 1, 3]])
