"""The operators of a tree of drafts without a GPU: every invalid argument of their C entry
points is refused on the host before anything reaches the HIP runtime, the workspace query
answers for every valid shape, and the Python binding refuses what it can see is wrong."""
import ctypes
import os

import numpy as np
import pytest

import tree_reference as ref

torch = pytest.importorskip("torch")

BAD = ctypes.c_size_t(-1).value
# aligned, far apart and never dereferenced: every call below fails validation first
P = [(i + 1) << 42 for i in range(20)]


@pytest.fixture(scope="module")
def L():
    import spec_verify_amd as svq
    if not os.path.exists(svq.library_path):
        from spec_verify_amd import build
        build.build()
    return svq.lib()


CACHE = dict(k=P[0], v=P[1], k0=8192, k1=512, k2=256, v0=8192, v1=512, v2=256, pages=100, page_size=16, type=0, ks=0, vs=0,
             table=P[2], ld_table=50, max_pages=40, lengths=P[3])


def _attend(L, q=P[4], ldq=1024, k=P[5], ldk=512, v=P[6], ldv=512, starts=P[7], parents=P[8], out=P[9], ldo=1024, M=20,
            S=4, H=4, G=2, D=256, ws=P[10], wsb=1 << 40, cache=True, **change):
    import spec_verify_amd as svq
    c = svq._CACHE.pack(*{**CACHE, **change}.values()) if cache else None
    return L.svq_tree_attention(q, ldq, k, ldk, v, ldv, c, starts, parents, 0.1, 0, 0, out, ldo, M, S, H, G, D, ws, wsb,
                                None)


@pytest.mark.parametrize("status,change", [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(cache=False)), (1, dict(starts=None)),
    (1, dict(out=None)), (1, dict(table=0)), (1, dict(lengths=0)),
    (2, dict(M=0)), (2, dict(S=0)), (2, dict(H=0)), (2, dict(G=0)), (2, dict(H=2, G=4)), (2, dict(M=(1 << 24) + 1)),
    (2, dict(M=1 << 20, H=1 << 12)), (2, dict(ldq=1016)), (2, dict(ldk=504)), (2, dict(ldv=504)), (2, dict(ldo=1016)),
    (2, dict(pages=-1)), (2, dict(pages=1 << 32)), (2, dict(page_size=0)), (2, dict(page_size=(1 << 20) + 1)),
    (2, dict(max_pages=-1)), (2, dict(max_pages=1 << 20, page_size=1 << 11, ld_table=1 << 20)), (2, dict(ld_table=39)),
    (2, dict(k0=-8192)), (2, dict(v0=1 << 47)), (2, dict(k0=1 << 44)),
    (4, dict(H=5, ldq=2048, ldo=2048)), (4, dict(ldq=1028)), (4, dict(ldo=1025)),
    (6, dict(q=P[4] + 8)), (6, dict(out=P[9] + 2)), (6, dict(k=P[5] + 4)), (6, dict(v=P[6] + 8)),
    (6, dict(starts=P[7] + 2)), (6, dict(parents=P[8] + 1)), (6, dict(k1=516)), (6, dict(v2=257)),
    (6, dict(type=1, ks=P[11] + 2)), (6, dict(type=1, k2=264)), (6, dict(table=P[2] + 2)),
    (7, dict(out=P[4])), (7, dict(out=P[5] + 64)), (7, dict(out=P[0] + 4096)), (7, dict(out=P[1])), (7, dict(out=P[7])),
    (7, dict(out=P[8])), (7, dict(out=P[2])), (7, dict(out=P[3])), (7, dict(out=P[10] + 4096)), (7, dict(ws=P[4])),
    (7, dict(ws=P[0])), (7, dict(type=1, vs=P[10])),
    (8, dict(ws=None)), (8, dict(wsb=4096)), (8, dict(ws=P[10] + 16)),
    (10, dict(D=96, ldq=1024)), (10, dict(D=512, ldq=4096, ldo=4096)), (10, dict(type=2)), (10, dict(ks=P[11])),
    (10, dict(type=-1)),
])
def test_attention_refusals(L, status, change):
    assert _attend(L, **change) == status


# (without a workspace, what is otherwise valid ends with status 8)
@pytest.mark.parametrize("status,change", [
    (2, dict(k0=1 << 31)), (2, dict(v1=1 << 31)), (2, dict(type=1, k0=1 << 32)), (8, dict(type=1, k0=(1 << 32) - 16)),
    (8, dict(k0=1 << 40, pages=1)), (8, dict(v1=1 << 40, page_size=1)), (8, dict(k0=-5, pages=1)), (8, dict(G=1, k2=3)),
    (2, dict(ldk=1 << 31)), (2, dict(ldv=1 << 31)), (8, dict(ldq=1 << 31, ldo=1 << 31)),
    (8, dict(max_pages=1 << 20, page_size=1 << 10, ld_table=1 << 20)),
    (2, dict(max_pages=1 << 20, page_size=1 << 10, ld_table=1 << 20, M=2000)),
    (2, dict(M=1 << 20)), (8, dict(M=1 << 17)),
    (8, dict(table=0, max_pages=0)), (8, dict(table=0, max_pages=0, ld_table=0)),
    (8, dict(parents=None)), (8, dict(type=1)), (8, dict(type=1, ks=P[11], vs=P[12])),
])
def test_attention_limits(L, status, change):
    assert _attend(L, ws=None, **change) == status


def test_a_pool_without_pages_has_no_address(L):
    import spec_verify_amd as svq
    for pages, status in ((0, 8), (1, 1)):
        c = svq._CACHE.pack(*{**CACHE, "k": 0, "v": 0, "pages": pages}.values())
        assert L.svq_tree_attention(P[4], 1024, P[5], 512, P[6], 512, c, P[7], None, 0.1, 0, 0, P[9], 1024, 20, 4, 4, 2, 256,
                                    None, 0, None) == status


def test_attention_workspace_query(L):
    q = L.svq_tree_attention_workspace_bytes
    for bad in ((0, 1, 4, 2, 64), (5, 0, 4, 2, 64), (5, 1, 4, 3, 64), (5, 1, 4, 2, 80), (5, 1, 2, 4, 64),
                (1 << 22, 1, 1 << 10, 1, 64)):
        assert q(*bad) == BAD, bad
    for M in (1, 5, 128, 2048, 1 << 20):
        for S in (1, 7, 128, 1 << 20):
            for H, G in ((1, 1), (24, 4), (64, 1)):
                for D in (64, 128, 256):
                    v = q(M, S, H, G, D)
                    # the counters' place and at most two blocks of 128 fp32 rows a workgroup
                    assert 256 * 1024 < v <= 256 * 1024 + 4096 * 2 * 128 * (D + 2) * 4, (M, S, H, G, D, v)


ADJ = dict(history=P[0], ld_history=100, max_history=90, lengths=P[1], prompts=P[2], inputs=P[3], parents=P[4], rep=P[5],
           pres=P[6], freq=P[7], bs=P[8], bt=P[9], bv=P[10], biases=30, allowed=P[11], ld_allowed=40, masks=6, mask_rows=P[12])


def _adjust(L, logits=P[13], ld=1000, starts=P[14], out=P[15], ldo=1000, M=20, S=4, V=1000, adjustments=True, **change):
    import spec_verify_amd as svq
    a = svq._ADJUSTMENTS.pack(*{**ADJ, **change}.values()) if adjustments else None
    return L.svq_adjust_logits(logits, ld, starts, a, out, ldo, M, S, V, None)


@pytest.mark.parametrize("status,change", [
    (1, dict(logits=None)), (1, dict(starts=None)), (1, dict(out=None)), (1, dict(adjustments=False)),
    (1, dict(history=0)), (1, dict(lengths=0)), (1, dict(inputs=0)), (1, dict(bs=0)), (1, dict(bt=0)), (1, dict(bv=0)),
    (1, dict(allowed=0)), (1, dict(mask_rows=0)),
    (2, dict(M=0)), (2, dict(S=-1)), (2, dict(V=0)), (2, dict(V=1001)), (2, dict(ld=999)), (2, dict(ldo=999)),
    (2, dict(M=(1 << 24) + 1)), (2, dict(max_history=101)), (2, dict(max_history=-1)),
    (2, dict(max_history=(1 << 29) + 1, ld_history=1 << 30)), (2, dict(biases=-1)), (2, dict(masks=0)),
    (2, dict(ld_allowed=31)),
    (6, dict(logits=P[13] + 1)), (6, dict(out=P[15] + 1)), (6, dict(history=P[0] + 2)), (6, dict(inputs=P[3] + 1)),
    (6, dict(freq=P[7] + 2)), (6, dict(bv=P[10] + 2)), (6, dict(mask_rows=P[12] + 3)), (6, dict(starts=P[14] + 2)),
    (7, dict(out=P[13] + 2)), (7, dict(out=P[13], ldo=1008)), (7, dict(out=P[0])), (7, dict(out=P[1])), (7, dict(out=P[2])),
    (7, dict(out=P[3])), (7, dict(out=P[4])), (7, dict(out=P[5])), (7, dict(out=P[8])), (7, dict(out=P[10])),
    (7, dict(out=P[11] + 64)), (7, dict(out=P[12])), (7, dict(out=P[14])),
])
def test_adjust_refusals(L, status, change):
    assert _adjust(L, **change) == status


def _accept(L, tok=P[0], inp=P[1], par=P[2], starts=P[3], acc=P[4], nxt=P[5], com=P[6], path=P[7], M=20, S=4):
    return L.svq_accept_tree(tok, inp, par, starts, acc, nxt, com, path, M, S, None)


@pytest.mark.parametrize("status,change", [
    (1, dict(tok=None)), (1, dict(inp=None)), (1, dict(par=None)), (1, dict(starts=None)), (1, dict(acc=None)),
    (1, dict(nxt=None)), (1, dict(com=None)), (1, dict(path=None)), (2, dict(M=0)), (2, dict(S=0)),
    (2, dict(M=(1 << 24) + 1)), (6, dict(par=P[2] + 2)), (6, dict(path=P[7] + 1)), (7, dict(com=P[0])), (7, dict(path=P[6])),
    (7, dict(path=P[2] + 76)), (7, dict(acc=P[3] + 16)), (7, dict(nxt=P[4])),
])
def test_accept_refusals(L, status, change):
    assert _accept(L, **change) == status


def test_binding_refuses_host_tensors_and_bad_shapes():
    import spec_verify_amd as svq
    i = torch.zeros(4, dtype=torch.int32)
    bf = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        svq.tree_attention(bf, bf, bf, cache, cache, i.view(1, 4), i[:1], i[:2])
    with pytest.raises(ValueError, match=r"\[M, H, D\]"):
        svq.tree_attention(bf[0], bf, bf, cache, cache, i.view(1, 4), i[:1], i[:2])
    for limits in (dict(window=(1 << 32) + 5), dict(sinks=1 << 31), dict(window=-(1 << 31) - 1)):
        with pytest.raises(ValueError, match="32 bits"):
            svq.tree_attention(bf, bf, bf, cache, cache, i.view(1, 4), i[:1], i[:2], **limits)
    with pytest.raises(ValueError, match="device tensor"):
        svq.adjust_logits(bf[0], i.view(1, 4), i[:1], i[:2], i[:2])
    with pytest.raises(TypeError, match="logits must be"):
        svq.adjust_logits(bf[0].float(), i.view(1, 4), i[:1], i[:2], i[:2])
    with pytest.raises(ValueError, match="device tensor"):
        svq.accept_tree(i, i, i, i)
    with pytest.raises(TypeError, match="int32"):
        svq.accept_tree(i.float(), i, i, i)
    with pytest.raises(ValueError, match="S >= 1"):
        svq.accept_tree(i, i, i, i[:1])


def test_the_reference_walks_and_sees_as_defined():
    """Hand-worked: a tree 0 -> (1, 2), 1 -> 3, 2 -> 4 behind two cached tokens."""
    parents = np.array([-1, 0, 0, 1, 2])
    assert ref.paths(parents, 5) == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4]]
    assert ref.paths(None, 3) == [[0], [0, 1], [0, 1, 2]]
    got = ref.accept(np.array([7, 1, 9, 2, 3]), np.array([5, 8, 7, 1, 9]), parents, np.array([0, 5]))
    assert [x.tolist() for x in got] == [[2], [3], [7, 9, 3, -1, -1], [0, 2, 4, -1, -1]]
    q, k = np.zeros((5, 1, 1)), np.zeros((5, 1, 1))
    v = np.arange(1.0, 6).reshape(5, 1, 1)
    cache = np.array([10.0, 20.0]).reshape(1, 2, 1, 1)
    table, starts = np.zeros((1, 1), dtype=int), [0, 5]
    out, _, _ = ref.attend(q, k, v, cache, cache, table, [2], starts, parents, 1.0)
    assert np.allclose(out.ravel(), [31 / 3, 33 / 4, 34 / 4, 37 / 5, 39 / 5])
    out, _, _ = ref.attend(q, k, v, cache, cache, table, [2], starts, parents, 1.0, window=2, sinks=1)
    # positions 2, 3, 3, 4, 4: the window holds the row and one more, the first token stays
    assert np.allclose(out.ravel(), [31 / 3, 13 / 3, 14 / 3, 16 / 3, 18 / 3])
    x, _, _, plain = ref.adjust(np.array([[2.0, -2.0, 1.0, 0.5]]), np.array([[0, 1, 1]]), [3], np.array([2]), [0, 1],
                                prompt_lengths=[1], repetition=[2.0], presence=[0.25], frequency=[0.5],
                                bias=([0, 2], [3, 3], [1.0, 0.5]), allowed=np.array([[0b1011]], dtype=np.int32),
                                mask_rows=[0])
    assert x.tolist() == [[1.0, -4.0 - 1.0 - 0.25, -np.inf, 2.0]] and not plain.any()
