"""The per-request operators without a GPU: every invalid argument of their C
entry points is refused on the host before anything reaches the HIP runtime, the
workspace queries answer for every valid shape, and the Python binding refuses
what it can see is wrong."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

BAD = ctypes.c_size_t(-1).value
# aligned, far apart and never dereferenced: every call below fails validation first
P = [(i + 1) << 40 for i in range(12)]


@pytest.fixture(scope="module")
def L():
    import spec_verify_amd as svq
    if not os.path.exists(svq.library_path):
        from spec_verify_amd import build
        build.build()
    return svq.lib()


def _adapter(L, base=P[0], ldb=256, x=P[1], a=P[2], b=P[3], rows=P[4], scales=P[5], out=P[6], ldo=256, M=5, N=256,
             K=512, R=16, slots=4, ws=P[7], wsb=1 << 30):
    return L.svq_adapter_add(base, ldb, x, a, b, rows, scales, out, ldo, M, N, K, R, slots, ws, wsb, None)


@pytest.mark.parametrize("status,change", [
    (1, dict(base=None)), (1, dict(x=None)), (1, dict(a=None)), (1, dict(b=None)), (1, dict(rows=None)),
    (1, dict(scales=None)), (1, dict(out=None)),
    (2, dict(M=0)), (2, dict(N=-16)), (2, dict(K=0)), (2, dict(R=0)), (2, dict(R=264)), (2, dict(slots=0)),
    (2, dict(ldb=240)), (2, dict(ldo=255)), (2, dict(M=1 << 20, K=1 << 11)), (2, dict(M=1 << 23, N=256)),
    (2, dict(slots=(1 << 31) - 1, R=256, K=1 << 20)),
    (4, dict(N=250)), (4, dict(K=320)), (4, dict(R=12)), (4, dict(ldb=260)), (4, dict(ldo=257)),
    (6, dict(base=P[0] + 8)), (6, dict(x=P[1] + 8)), (6, dict(a=P[2] + 2)), (6, dict(b=P[3] + 4)),
    (6, dict(rows=P[4] + 2)), (6, dict(scales=P[5] + 1)), (6, dict(out=P[6] + 8)),
    (7, dict(out=P[1])), (7, dict(out=P[2] + 4096)), (7, dict(out=P[3])), (7, dict(out=P[4])), (7, dict(out=P[5])),
    (7, dict(out=P[0] + 16)), (7, dict(out=P[0], ldo=512)), (7, dict(ws=P[0])), (7, dict(ws=P[6])),
    (7, dict(ws=P[2])),
    (8, dict(ws=None)), (8, dict(wsb=64)), (8, dict(ws=P[7] + 16)),
])
def test_adapter_refusals(L, status, change):
    assert _adapter(L, **change) == status


def test_adapter_workspace_query(L):
    assert L.svq_adapter_workspace_bytes(5, 250, 512, 16, 4) == BAD
    assert L.svq_adapter_workspace_bytes(0, 256, 512, 16, 4) == BAD
    assert L.svq_adapter_workspace_bytes(5, 256, 512, 264, 4) == BAD
    for M in (1, 5, 16, 17, 128, 2000, 1 << 16):
        for K in (128, 5120, 16256):
            for R in (8, 16, 24, 64, 256):
                v = L.svq_adapter_workspace_bytes(M, 256, K, R, 8)
                # the fp32 intermediate, at least once and at most once per 128 elements of K,
                # and a row's share of an item
                assert M * R * 4 <= v - 256 * 1024 <= M * R * 4 * (K // 128) + 128 * M, (M, K, R, v)


def _sample(L, logits=P[0], ld=1000, u=P[1], t=P[2], k=P[3], p=P[4], mp=P[5], tok=P[6], lp=P[7], M=4, V=1000,
            ws=P[8], wsb=1 << 40):
    return L.svq_sample(logits, ld, u, t, k, p, mp, tok, lp, M, V, ws, wsb, None)


@pytest.mark.parametrize("status,change", [
    (1, dict(logits=None)), (1, dict(u=None)), (1, dict(tok=None)),
    (2, dict(M=0)), (2, dict(V=0)), (2, dict(V=1001)), (2, dict(V=(1 << 24) + 1, ld=1 << 25)), (2, dict(M=(1 << 24) + 1)),
    (6, dict(logits=P[0] + 1)), (6, dict(u=P[1] + 2)), (6, dict(t=P[2] + 1)), (6, dict(k=P[3] + 2)),
    (6, dict(p=P[4] + 2)), (6, dict(mp=P[5] + 2)), (6, dict(tok=P[6] + 2)), (6, dict(lp=P[7] + 2)),
    (7, dict(tok=P[0] + 64)), (7, dict(tok=P[1])), (7, dict(tok=P[2])), (7, dict(lp=P[6])), (7, dict(lp=P[3] + 4)),
    (7, dict(tok=P[4])), (7, dict(lp=P[5])),
])
def test_sample_refusals(L, status, change):
    assert _sample(L, **change) == status


@pytest.mark.parametrize("status,change", [
    (8, dict(ws=None)), (8, dict(wsb=64)), (8, dict(ws=P[8] + 16)), (7, dict(ws=P[0])), (7, dict(ws=P[6])),
    (7, dict(ws=P[1])),
])
def test_sample_workspace_refusals(L, status, change):
    assert L.svq_sample_workspace_bytes(1, 248320) > 0
    assert _sample(L, M=1, V=248320, ld=248320, **change) == status


def test_sample_workspace_query(L):
    assert L.svq_sample_workspace_bytes(0, 5) == BAD
    assert L.svq_sample_workspace_bytes(5, 0) == BAD
    assert L.svq_sample_workspace_bytes(1, (1 << 24) + 1) == BAD
    for M in (1, 2, 5, 31, 128, 300, 5000, 1 << 24):
        for V in (1, 7, 8, 9, 8191, 8200, 32001, 248320, 1 << 24):
            v = L.svq_sample_workspace_bytes(M, V)
            assert v != BAD and v <= (1 << 30), (M, V, v)


def _accept(L, tok=P[0], inp=P[1], starts=P[2], acc=P[3], nxt=P[4], com=P[5], M=20, S=4):
    return L.svq_accept_drafts(tok, inp, starts, acc, nxt, com, M, S, None)


@pytest.mark.parametrize("status,change", [
    (1, dict(tok=None)), (1, dict(inp=None)), (1, dict(starts=None)), (1, dict(acc=None)), (1, dict(nxt=None)),
    (1, dict(com=None)), (2, dict(M=0)), (2, dict(S=0)), (2, dict(M=(1 << 24) + 1)), (2, dict(S=-1)),
    (6, dict(tok=P[0] + 2)), (6, dict(com=P[5] + 1)),
    (7, dict(com=P[0])), (7, dict(com=P[1] + 76)), (7, dict(acc=P[2] + 16)), (7, dict(nxt=P[3])), (7, dict(com=P[4])),
])
def test_accept_refusals(L, status, change):
    assert _accept(L, **change) == status


def test_binding_refuses_host_tensors_and_bad_shapes():
    import spec_verify_amd as svq
    bf = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        svq.sample(bf, torch.zeros(4))
    with pytest.raises(TypeError, match="logits must be"):
        svq.sample(bf.float(), torch.zeros(4))
    with pytest.raises(ValueError, match="matrix"):
        svq.sample(bf[0], torch.zeros(1))
    with pytest.raises(ValueError, match="device tensor"):
        svq.adapter_add(bf, bf, bf, bf, torch.zeros(4, dtype=torch.int32), torch.zeros(1))
    with pytest.raises(ValueError, match="device tensor"):
        i = torch.zeros(4, dtype=torch.int32)
        svq.accept_drafts(i, i, i)
    with pytest.raises(TypeError, match="int32"):
        svq.accept_drafts(torch.zeros(4), torch.zeros(4), torch.zeros(2))
    with pytest.raises(ValueError, match="S >= 1"):
        i = torch.zeros(4, dtype=torch.int32)
        svq.accept_drafts(i, i, i[:1])
