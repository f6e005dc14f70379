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


def _every_bin(copies, keep):
    """(logits, order): `copies` tokens of each of the first `keep` patterns of the magnitudes
    from 2^-16 to 2^16, both signs, shuffled within each copy; order[i, c] is copy c of the i-th
    largest value."""
    rng = np.random.default_rng(copies)
    mags = np.arange(111 << 7, (111 << 7) + 4096)
    bits = np.concatenate([mags[::-1], mags | 0x8000])[:keep]   # descending
    place = np.stack([rng.permutation(keep) + c * keep for c in range(copies)], 1)
    row = np.empty(copies * keep, np.uint16)
    row[place] = bits[:, None]
    return torch.from_numpy(row.view(np.int16)).view(torch.bfloat16), place


@pytest.mark.parametrize("copies,keep,M", [(1, 8192, 8192), (1, 4000, 250), (1, 8192, 100), (5, 8192, 48)])
def test_every_bin_is_reached_by_every_seek(copies, keep, M):
    """One row that holds every value with a bin; each position of its order in turn is the last
    of top-k, the last of top-p and the draw. At T = 2^20 the weights are between 0.88 and 1, so
    a position's share of the mass is far wider than the steps of fp32."""
    import spec_verify_amd as svq
    _say("sample every bin", copies, keep, M)
    row, place = _every_bin(copies, keep)
    l = row.cuda().repeat(M, 1)
    v = np.sort(row.float().numpy().astype(np.float64))[::-1]
    cum = np.cumsum(np.exp((v - v[0]) / 2 ** 20))
    dev = lambda a, t=torch.float32: torch.tensor(a, dtype=t, device="cuda")
    T, last = dev(np.full(M, 2.0 ** 20)), dev(np.full(M, 1 - 2.0 ** -24))
    for i0 in range(0, keep, M):
        i = np.minimum(np.arange(i0, i0 + M), keep - 1)
        at, want = i * copies + i % copies, torch.from_numpy(place[i, i % copies]).int()
        middle = dev((cum[at] - 0.5) / cum[-1])
        assert torch.equal(svq.sample(l, middle, T)[0].cpu(), want), i0
        assert torch.equal(svq.sample(l, last, T, top_k=dev(at + 1, torch.int32))[0].cpu(), want), i0
        assert torch.equal(svq.sample(l, last, T, top_p=middle)[0].cpu(), want), i0


@pytest.mark.parametrize("M,V", [(1, 248320), (7, 50021), (51, 248320)])
def test_a_workspace_need_not_be_cleared(M, V):
    """The caller's workspace, exactly as large as it has to be, full of anything, used by one
    call after another; its neighbours stay as they were."""
    import spec_verify_amd as svq
    _say("sample workspace", M, V)
    g = torch.Generator("cuda").manual_seed(V + M)
    l = (torch.randn(M, V, device="cuda", generator=g) * 2.2).bfloat16()
    l[M - 1, ::3] = -1e9
    u = torch.rand(M, device="cuda", generator=g)
    k = torch.randint(0, 90, (M,), device="cuda", generator=g, dtype=torch.int32)
    want = [svq.sample(l, u), svq.sample(l, u, top_k=k)]
    n = svq.sample_workspace_bytes(M, V)
    assert n > 0
    memory = torch.empty(n + 512, dtype=torch.uint8, device="cuda")
    for fill in (0, 0xFF, 0x7F):
        memory.fill_(fill)
        ws = memory[256:256 + n]
        for w, kw in zip(want, ({}, dict(top_k=k))):
            got = svq.sample(l, u, workspace=ws, **kw)
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
        assert bool((memory[:256] == fill).all()) and bool((memory[256 + n:] == fill).all())
