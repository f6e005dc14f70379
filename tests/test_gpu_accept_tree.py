"""GPU: acceptance along a tree of drafts against a walk in plain Python; whole numbers, so
everything is equal. And one whole step of verifying a tree, operator after operator."""
import os
import sys

import numpy as np
import pytest

import tree_reference as ref

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


def _say(*a):
    print("[gpu]", *a, flush=True)
    sys.stdout.flush()


def _problem(seed, rows, pad=0, hit=0.7, depth=2.0, words=50):
    rng = np.random.default_rng(seed)
    M = sum(rows) + 2 * pad
    starts = np.concatenate([[pad], pad + np.cumsum(rows)]).astype(np.int32)
    parents = np.full(M, -1, dtype=np.int32)
    tokens, inputs = rng.integers(0, words, M).astype(np.int32), rng.integers(0, words, M).astype(np.int32)
    for a, k in ref.sequences(starts, M):
        for i in range(1, k):
            parents[a + i] = i - 1 - int(rng.random() ** depth * i)
            if rng.random() < hit:
                inputs[a + i] = tokens[a + parents[a + i]]
    return tokens, inputs, parents, starts


def _check(label, problem):
    import spec_verify_amd as svq
    _say("accept", label)
    got = svq.accept_tree(*(torch.from_numpy(x).cuda() for x in problem))
    for name, g, w in zip(("accepted", "next", "committed", "path"), got, ref.accept(*problem)):
        assert (g.cpu().numpy() == w).all(), (label, name)


@pytest.mark.parametrize("rows", [[1], [2], [8], [64], [65], [300], [1000], [0, 5, 0, 0, 9, 0], [1 + i % 40 for i in range(500)],
                                  [256, 257, 255, 1]], ids=lambda r: f"{len(r)}x{max(r)}")
@pytest.mark.parametrize("hit", [0.0, 0.5, 0.95, 1.0])
def test_against_a_walk(rows, hit):
    _check(rows[:4], _problem(31 + len(rows), rows, pad=2, hit=hit))


def test_chains_are_as_accept_drafts():
    import spec_verify_amd as svq
    rows = [1, 4, 9, 70, 300]
    tokens, inputs, parents, starts = _problem(5, rows, hit=0.0)
    for a, n in ref.sequences(starts, len(tokens)):
        parents[a:a + n] = np.arange(n) - 1
        inputs[a + 1:a + n] = tokens[a:a + n - 1]
    inputs[starts[3] + 66] += 1
    problem = (tokens, inputs, parents, starts)
    _check("chains", problem)
    dev = [torch.from_numpy(x).cuda() for x in problem]
    tree, drafts = svq.accept_tree(*dev), svq.accept_drafts(dev[0], dev[1], dev[3])
    for t, d in zip(tree, drafts):
        assert torch.equal(t, d)


def test_siblings_with_one_token_and_nothing_to_draw():
    t, i, p, s = _problem(6, [40, 12], hit=1.0, words=2)
    _check("two words", (t, i, p, s))
    t[:] = -1
    i[:] = -1
    _check("nothing to draw", (t, i, p, s))


def test_parents_and_starts_outside():
    t, i, p, s = _problem(7, [9, 9], hit=1.0)
    p[::2] = [3, 100, -5, 2 ** 31 - 1, -2 ** 31, 8, 0, 1, 2]
    i[:], t[:] = 1, 1
    _check("parents", (t, i, p, s))
    s[0], s[2] = -4, 99
    _check("starts", (t, i, p, s))


def test_graph_replays():
    import spec_verify_amd as svq
    problems = [_problem(40 + k, [64, 3, 20], hit=0.8) for k in range(3)]
    dev = [torch.from_numpy(x).cuda() for x in problems[0]]
    svq.accept_tree(*dev)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = svq.accept_tree(*dev)
    for problem in problems + problems[:1]:
        for d, x in zip(dev, problem):
            d.copy_(torch.from_numpy(x))
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, ref.accept(*problem)):
            assert (got.cpu().numpy() == want).all()
        svq.accept_tree(*dev)


def test_a_step_of_verifying_trees():
    """Projections, attention, head, adjustment, sampling and acceptance of two sequences' trees; the accepted rows go
    into the cache. The next step's attention to them equals that of a chunk that was a chain from the start."""
    import spec_verify_amd as svq
    H, G, D, page, V, K = 4, 2, 64, 16, 512, 256
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").bfloat16()
    rows, lengths = [13, 6], [30, 47]
    tokens, inputs, parents, starts = _problem(8, rows, hit=0.0, words=V)
    parents, inputs, starts = (torch.from_numpy(x).cuda() for x in (parents, inputs, starts))
    M = sum(rows)
    width = (H + 2 * G) * D
    weight = torch.randn(width, K, generator=gen, device="cuda").mul(0.06).bfloat16()
    codes, scales = svq.rtn_quantize(weight, bits=4)
    tiled = svq.q4_repack(codes)
    x = normal(M, K)
    fused = svq.w4a16_gemm(x, tiled, scales, width)
    q, k, v = (c.view(M, -1, D) for c in fused.split([H * D, G * D, G * D], 1))
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    caches = [normal(8, page, G, D) for _ in range(2)]
    held = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    attended = svq.tree_attention(q, k, v, *caches, table, held, starts, parents=parents)
    head = torch.randn(V, H * D, generator=gen, device="cuda").mul(0.1).bfloat16()
    head_codes, head_scales = svq.rtn_quantize(head)
    logits = torch.cat([svq.w8a16_gemm(part, head_codes, head_scales) for part in attended.view(M, -1).split(16)])
    history = torch.randint(0, V, (2, 64), generator=gen, device="cuda", dtype=torch.int32)
    rep = torch.full((2,), 1.2, device="cuda")
    adjusted = svq.adjust_logits(logits, history, held, inputs, starts, parents=parents, repetition=rep, out=logits)
    sampled, _ = svq.sample(adjusted, torch.rand(M, generator=gen, device="cuda"))
    # the drafts of every second node are what was sampled at its parent
    first = torch.tensor([0] * rows[0] + [rows[0]] * rows[1], device="cuda")
    follow = torch.where(parents >= 0, sampled[first + parents.clamp(min=0)], inputs)
    accepted, following, committed, path = svq.accept_tree(sampled, follow, parents, starts)
    want = ref.accept(*(t.cpu().numpy() for t in (sampled, follow, parents, starts)))
    for got, w in zip((accepted, following, committed, path), want):
        assert (got.cpu().numpy() == w).all()
    assert int(accepted.max()) > 1
    # the accepted rows become cached tokens
    m = torch.nonzero(path >= 0)[:, 0]
    seq = (m >= rows[0]).long()
    at = held[seq].long() + m - first[m]
    for cache, new in zip(caches, (k, v)):
        cache[table[seq, at // page].long(), at % page] = new[first[m] + path[m].long()]
    now = held + accepted + 1
    one = torch.arange(3, dtype=torch.int32, device="cuda")
    q2, k2, v2 = normal(2, H, D), normal(2, G, D), normal(2, G, D)
    got = svq.tree_attention(q2, k2, v2, *caches, table, now, one)
    host = [c.double().cpu().numpy() for c in (q2, k2, v2, *caches)]
    want, bound, _ = ref.attend(*host, table.cpu().numpy(), now.cpu().numpy(), one.cpu().numpy(), None, D ** -0.5)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
