"""GPU: sampling where a count or a launch shape is at an end. Tokens are whole numbers and
have to be equal; the definition is in 64 bits."""
import sys

import numpy as np
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


def test_more_rows_than_one_launch_takes():
    """2^22 and some rows of 1024 threads pass 2^32, which no launch may have. Two tokens:
    the likelier one (the first of two equals) for u W < 1, W = 1 + exp(-difference / T)."""
    import spec_verify_amd as svq
    _say("sample 2^22 rows")
    M = (1 << 22) + 5
    g = torch.Generator("cuda").manual_seed(1)
    l = (torch.randn(M, 2, device="cuda", generator=g) * 2).bfloat16()
    # rows that are counted the long way, one in each launch
    for m in (3, M - 2):
        l[m] = torch.tensor([3e5, 2.5e5], device="cuda").bfloat16()
    u = torch.rand(M, device="cuda", generator=g)
    T = torch.rand(M, device="cuda", generator=g) + 0.5
    tokens, logprobs = svq.sample(l, u, T)
    v = l.double()
    second = (v[:, 1] > v[:, 0]).long()             # of the likelier one
    w = torch.exp(-(v[:, 0] - v[:, 1]).abs() / T.double())
    other = u.double() * (1 + w) >= 1
    assert torch.equal(tokens.long(), second ^ other.long())
    want = torch.where(other, torch.log(w), 0.0) - torch.log1p(w)
    # half a step of fp32, and what two fp64 values differ
    assert bool(((logprobs.double() - want).abs() <= 2.0 ** -24 * want.abs() + 1e-12).all())
