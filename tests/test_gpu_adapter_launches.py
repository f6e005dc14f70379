"""GPU: the adapter kernels of two launches, which every hidden size above 2560 and every rank
above 32 takes: column slices, infinities and NaN, equal bits, K ranges of several rounds, and
workspaces of the caller's.

Bound on an element's error. The rank-R intermediate t_r is an fp32 sum of exact products: a
wave adds up its tiles of 128 one after another, eight waves meet, then the K ranges; whatever
the order inside a matrix instruction, at most 128 * (a wave's tiles) + 7 + (ranges - 1)
roundings of at most one fp32 step (2^-23 of the sum of magnitudes) reach it. Scaling rounds
once (2^-24). The second sum has three exact parts of each rank, of ranks in steps of 32, and
base: as many roundings as terms. The result is rounded to bf16 once, half a step: 2^-8 of it."""
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


def _ranges(M, K, R):
    """(128-element tiles of a K range, ranges), as the plan of the first launch has them."""
    tiles = 1 if R <= 16 else 2 if R <= 32 else 4
    groups = -(-M // 16) * -(-R // (16 * tiles))
    KT = K // 128
    blocks = max(1, min(-(-KT // 8), 1024 // groups))
    if groups < 64 and blocks > 4:
        blocks = -(-blocks // 8) * 8
    T = -(-KT // blocks)
    if groups >= 64:
        T = -(-T // 8) * 8
    return T, -(-KT // T)


def _problem(seed, M, K, N, R, slots, bare=True):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).bfloat16()
    rows = torch.randint(-1 if bare else 0, slots, (M,), device="cuda", generator=g, dtype=torch.int32)
    return dict(base=n(M, N, std=3.0), x=n(M, K), a=n(slots, R, K, std=K ** -0.5), b=n(slots, N, R, std=R ** -0.5),
                rows=rows, scales=torch.rand(slots, device="cuda", generator=g) * 2 + 0.1)


def _call(d, **kw):
    import spec_verify_amd as svq
    return svq.adapter_add(d["base"], d["x"], d["a"], d["b"], d["rows"], d["scales"], **kw)


def _within(d, out, label):
    M, K = d["x"].shape
    R = d["a"].shape[1]
    T, ranges = _ranges(M, K, R)
    first = 128 * -(-T // 8) + 7 + ranges - 1
    second = 3 * 32 * -(-R // 32) + 1
    for s in range(-1, d["a"].shape[0]):
        m = (d["rows"] == s).nonzero().flatten()
        if s < 0:
            assert torch.equal(out[m].view(torch.int16), d["base"][m].view(torch.int16)), label
            continue
        x, base, sc = d["x"][m].double(), d["base"][m].double(), d["scales"][s].double()
        at, bt = d["a"][s].double().t().contiguous(), d["b"][s].double().t().contiguous()
        t = x @ at
        t_err = first * 2.0 ** -23 * (x.abs() @ at.abs()) + 2.0 ** -24 * t.abs()
        want = base + sc * (t @ bt)
        bound = sc * (t_err @ bt.abs()) + second * 2.0 ** -23 * (base.abs() + sc * ((t.abs() + t_err) @ bt.abs()))
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
        assert bool(((out[m].double() - want).abs() <= bound).all()), (label, s)


ROUNDS = [  # a wave takes several tiles of a range, and the last range is shorter
    (2001, 17408, 48, 16, 3), (2001, 17408, 48, 72, 3), (1999, 17408, 32, 128, 2), (8192, 5120, 16, 16, 4),
]
ONE_ROUND = [(1100, 11136, 528, 24, 5), (5, 17408, 48, 16, 2), (130, 17408, 64, 64, 6), (70, 5120, 96, 16, 5)]


@pytest.mark.parametrize("M,K,N,R,slots", ROUNDS + ONE_ROUND)
def test_k_ranges_of_one_round_and_of_several(M, K, N, R, slots):
    T, ranges = _ranges(M, K, R)
    _say("adapter rounds", M, K, N, R, "tiles", T, "ranges", ranges)
    assert (T > 8) == ((M, K, N, R, slots) in ROUNDS)
    d = _problem(M + R, M, K, N, R, slots)
    _within(d, _call(d), (M, K, N, R))


@pytest.mark.parametrize("M,K,N,R,slots", ROUNDS + ONE_ROUND)
def test_every_product_once(M, K, N, R, slots):
    """Whole numbers: x has 30 entries of -1 or 1 in a row, so |t| <= 30, |out| <= 220, all sums
    exact in fp32 and bf16. A tile left out or taken twice shows."""
    _say("adapter integers", M, K, N, R)
    g = torch.Generator("cuda").manual_seed(M * 3 + R)
    integers = lambda lo, hi, *s: torch.randint(lo, hi, s, device="cuda", generator=g)
    x = torch.zeros(M, K, device="cuda")
    x.scatter_(1, integers(0, K, M, 30), integers(0, 2, M, 30).float() * 2 - 1)
    a = integers(-1, 2, slots, R, K).float()
    b = torch.zeros(slots, N, R, device="cuda")
    b.scatter_(2, integers(0, R, slots, N, 1), 1.0)
    d = dict(base=integers(-100, 101, M, N).bfloat16(), x=x.bfloat16(), a=a.bfloat16(), b=b.bfloat16(),
             rows=integers(-1, slots, M).int(), scales=torch.tensor([1.0, 2.0, 4.0, 0.0, -1.0, 1.0], device="cuda")[:slots])
    out = _call(d).double()
    for s in range(-1, slots):
        m = (d["rows"] == s).nonzero().flatten()
        want = d["base"][m].double()
        if s >= 0:
            want = want + d["scales"][s].double() * ((x[m].double() @ a[s].double().t().contiguous()) @ b[s].double().t().contiguous())
        assert torch.equal(out[m], want), s


TWO = [(21, 5120, 96, 16, 4), (40, 384, 160, 64, 6), (70, 5120, 96, 32, 5)]


@pytest.mark.parametrize("M,K,N,R,slots", TWO)
def test_in_place_and_column_slices(M, K, N, R, slots):
    """One projection's columns of a fused output, in place and not; the other columns and the
    rows' ends stay as they were."""
    _say("adapter slices", M, K, N, R)
    d = _problem(3, M, K, N, R, slots)
    plain = _call(d)
    _within(d, plain, "plain")
    for width, first in ((N, 0), (3 * N, N), (104 + N, 104)):
        wide = torch.full((M, width), 7.0, dtype=torch.bfloat16, device="cuda")
        part = wide[:, first:first + N]
        part.copy_(d["base"])
        assert _call({**d, "base": part}, out=part).data_ptr() == part.data_ptr()
        assert torch.equal(part, plain)
        wide[:, first:first + N] = 7.0
        assert bool((wide == 7.0).all())
    src = torch.zeros(M, N + 32, dtype=torch.bfloat16, device="cuda")
    src[:, 16:16 + N] = d["base"]
    dst = torch.full((M, 2 * N + 48), 5.0, dtype=torch.bfloat16, device="cuda")
    _call({**d, "base": src[:, 16:16 + N]}, out=dst[:, N:2 * N])
    assert torch.equal(dst[:, N:2 * N], plain)
    assert bool((dst[:, :N] == 5.0).all()) and bool((dst[:, 2 * N:] == 5.0).all())


@pytest.mark.parametrize("M,K,N,R,slots", TWO)
def test_rows_and_adapters_do_not_reach_each_other(M, K, N, R, slots):
    """Infinities and NaN in one request's rows and in an adapter that only they use leave
    every other row as it is without them; so does one row among clean ones of its adapter."""
    _say("adapter isolation", M, K, N, R)
    d = _problem(5, M, K, N, R, slots)
    d["rows"] = torch.arange(M, device="cuda", dtype=torch.int32) % slots
    clean = _call(d)
    bad = {k: v.clone() for k, v in d.items()}
    hit = d["rows"] == 2
    bad["a"][2, :, 5] = float("nan")
    bad["b"][2, 7] = float("inf")
    bad["x"][hit] = float("inf")
    bad["base"][hit] = float("nan")
    assert torch.equal(_call(bad)[~hit], clean[~hit])
    bad = {k: v.clone() for k, v in d.items()}
    bad["x"][8, K - 1] = float("nan")
    got = _call(bad)
    keep = torch.arange(M, device="cuda") != 8
    assert torch.equal(got[keep], clean[keep])
    assert bool(got[8].isnan().all())


@pytest.mark.parametrize("M,K,N,R,slots", TWO)
def test_repeated_calls_and_single_rows(M, K, N, R, slots):
    """Equal bits from equal calls; a row by itself meets its bound."""
    _say("adapter repeats", M, K, N, R)
    d = _problem(6, M, K, N, R, slots)
    whole = _call(d)
    for _ in range(3):
        assert torch.equal(_call(d), whole)
    for m in (0, 15, 16, M - 1):
        one = {**d, "base": d["base"][m:m + 1], "x": d["x"][m:m + 1], "rows": d["rows"][m:m + 1]}
        _within(one, _call(one), m)


# of one launch, of two, and of two with items that only some rows fill
@pytest.mark.parametrize("M,K,N,R,slots", TWO + [(37, 640, 1040, 24, 5), (300, 5120, 96, 16, 40)])
def test_a_workspace_need_not_be_cleared(M, K, N, R, slots):
    """The caller's workspace, exactly as large as it has to be, full of anything, used by one
    call after another; its neighbours stay as they were."""
    import spec_verify_amd as svq
    _say("adapter workspace", M, K, N, R)
    d = _problem(9, M, K, N, R, slots)
    want = _call(d)
    n = svq.adapter_workspace_bytes(M, N, K, R, slots)
    memory = torch.empty(n + 512, dtype=torch.uint8, device="cuda")
    for fill in (0, 0xFF, 0x7F):
        memory.fill_(fill)
        assert torch.equal(_call(d, workspace=memory[256:256 + n]), want)
        assert torch.equal(_call(d, workspace=memory[256:256 + n]), want)
        assert bool((memory[:256] == fill).all()) and bool((memory[256 + n:] == fill).all())


def test_a_verify_chunk_in_one_workspace():
    """Projection, adapter in place, head and sampling on the hidden size of two adapter
    launches, all in one workspace, whose arrival counters stay at zero; eager, and as two
    captured graphs that share it."""
    import oracle
    import spec_verify_amd as svq
    import synth
    _say("one workspace")
    M, K, N, V, R, slots = 13, 5120, 256, 40960, 16, 3

    def dev(v):
        v = np.ascontiguousarray(v)
        return torch.from_numpy(v.view(np.int16) if v.dtype == np.uint16 else v).cuda()

    proj, head = synth.gen_w4a16(41, M, K, N), synth.gen_w8a16(42, M, N, V)
    d = _problem(43, M, K, N, R, slots)
    x, tiled, scales = dev(proj.x).view(torch.bfloat16), svq.q4_repack(dev(proj.qweight)), dev(proj.scales)
    hw, hs = torch.from_numpy(np.ascontiguousarray(head.w)).cuda(), dev(head.scales)
    u = torch.rand(M, device="cuda", generator=torch.Generator("cuda").manual_seed(44))
    k = torch.full((M,), 40, dtype=torch.int32, device="cuda")
    need = max(svq.w4a16_workspace_bytes(M, N, K), svq.w8a16_workspace_bytes(M, V, N),
               svq.adapter_workspace_bytes(M, N, K, R, slots), svq.sample_workspace_bytes(M, V))
    assert svq.sample_workspace_bytes(M, V) > 0 and svq.w4a16_workspace_bytes(M, N, K) > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def step(ws):
        y = svq.w4a16_gemm(x, tiled, scales, N, workspace=ws)
        base = y.clone()
        svq.adapter_add(y, x, d["a"], d["b"], d["rows"], d["scales"], out=y, workspace=ws)
        logits = svq.w8a16_gemm(y, hw, hs, workspace=ws)
        return (base, y, logits) + tuple(svq.sample(logits, u, top_k=k, workspace=ws))

    own = step(None)
    y64, _ = oracle.w4a16(proj.x, proj.qweight, proj.scales)
    assert oracle.gate(own[0].view(torch.int16).cpu().numpy().view(np.uint16), y64)[0]
    _within({**d, "x": x, "base": own[0]}, own[1], "chunk")
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(ws), own))
        assert bool((ws[:256 * 1024] == 0).all())
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(ws)
        graphs.append((g, outs))
    for rep in range(4):
        for g, outs in graphs:
            for t in outs:
                t.zero_()
            ws[256 * 1024:] = 0xA5
            g.replay()
            eager = step(ws)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) and torch.equal(e, b) for a, e, b in zip(outs, eager, own)), rep
    assert bool((ws[:256 * 1024] == 0).all())
