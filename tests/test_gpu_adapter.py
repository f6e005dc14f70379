"""GPU: low-rank adapters of many requests beside a shared projection, against the
formula in 64 bits.

Bound on an element's error. The rank-R intermediate t_r is an fp32 sum of exact
products; whatever the order inside a matrix instruction, at most 128 roundings of
at most one fp32 step each (2^-23) reach it, so it is off by at most
128 * 2^-23 * sum_k |x_k a_rk|. Scaling rounds once (2^-24) and the split into two
bf16 halves leaves 2^-16 |scale t_r|. The second sum has at most 2 * 256 + 2 terms of
exact products: 514 * 2^-23 of the sum of magnitudes. The result is rounded to bf16
once, half a step: 2^-8 of it."""
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


def _problem(seed, M, K, N, R, slots, pattern="random"):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16()
    if pattern == "random":      # none, every adapter, and indexes that name none
        rows = torch.randint(-2, slots + 1, (M,), generator=g)
    elif pattern == "chunks":    # a request's rows stand together
        rows = torch.randint(-1, slots, ((M + 3) // 4,), generator=g).repeat_interleave(4)[:M]
    elif pattern == "one":
        rows = torch.full((M,), slots - 1)
    elif pattern == "none":
        rows = torch.full((M,), -1)
    else:                        # as many different adapters in a tile as there are
        rows = torch.arange(M) % slots
    return dict(base=n(M, N, std=3.0), x=n(M, K), a=n(slots, R, K, std=K ** -0.5), b=n(slots, N, R, std=R ** -0.5),
                rows=rows.int(), scales=torch.rand(slots, generator=g) * 2 + 0.1)


def _dev(p):
    return {k: v.cuda() for k, v in p.items()}


def _call(d, **kw):
    import spec_verify_amd as svq
    return svq.adapter_add(d["base"], d["x"], d["a"], d["b"], d["rows"], d["scales"], **kw)


def _reference(p):
    """(result, bound on its error), float64 [M, N]."""
    base, x, a, b = (p[k].double() for k in ("base", "x", "a", "b"))
    out, bound = base.clone(), torch.zeros_like(base)
    for s in range(a.shape[0]):
        m = (p["rows"] == s).nonzero().flatten()
        if len(m) == 0:
            continue
        sc = float(p["scales"][s])
        t = x[m] @ a[s].T
        t_err = 128 * 2.0 ** -23 * (x[m].abs() @ a[s].abs().T) + (2.0 ** -16 + 2.0 ** -23) * t.abs()
        out[m] += sc * (t @ b[s].T)
        mags = base[m].abs() + sc * ((t.abs() + t_err) @ b[s].abs().T)
        bound[m] = sc * (t_err @ b[s].abs().T) + 514 * 2.0 ** -23 * mags
    return out, bound + 2.0 ** -8 * (out.abs() + bound)


def _check(p, out, label):
    ref, bound = _reference(p)
    err = (out.cpu().double() - ref).abs()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert bool((err <= bound).all()), f"{label}: error is {worst:.3g} of its bound"
    bare = (p["rows"] < 0) | (p["rows"] >= p["a"].shape[0])
    assert torch.equal(out.cpu()[bare].view(torch.int16), p["base"][bare].view(torch.int16)), label
    # beyond the bound: the errors of all elements together are those of one rounding
    rms = lambda v: v.double().pow(2).mean().sqrt().item()
    assert rms(err) <= 2.0 ** -8 * rms(ref), label


SHAPES = [
    # M, K, N, R, slots, pattern
    (1, 128, 16, 8, 1, "one"),
    (1, 5120, 1024, 16, 4, "one"),
    (2, 256, 32, 24, 3, "each"),
    (5, 512, 272, 16, 4, "chunks"),
    (16, 1152, 64, 32, 16, "each"),
    (17, 384, 1040, 40, 20, "each"),
    (37, 640, 1040, 24, 5, "random"),
    (20, 17408, 48, 128, 2, "random"),
    (33, 256, 80, 256, 3, "random"),
    (64, 1024, 5120, 64, 6, "chunks"),
    (128, 5120, 528, 32, 32, "chunks"),
    (128, 1280, 320, 72, 200, "each"),
    (300, 256, 48, 8, 1, "random"),
    (1003, 384, 96, 16, 7, "random"),
    (4111, 128, 32, 48, 3, "chunks"),
    (50, 256, 64, 16, 2, "none"),
]


@pytest.mark.parametrize("M,K,N,R,slots,pattern", SHAPES)
def test_against_the_formula(M, K, N, R, slots, pattern):
    _say("adapter", M, K, N, R, slots, pattern)
    p = _problem(M * 7 + R, M, K, N, R, slots, pattern)
    _check(p, _call(_dev(p)), (M, K, N, R, slots, pattern))


# few items and a short K (one launch), and either bound passed
@pytest.mark.parametrize("M,K,N,R,slots,pattern", [
    (1, 2560, 512, 16, 1, "one"),
    (1, 2688, 512, 16, 1, "one"),
    (3, 1280, 528, 32, 2, "each"),
    (3, 1408, 528, 32, 2, "each"),
    (31, 128, 1552, 24, 5, "random"),
    (256, 2560, 48, 16, 9, "random"),
    (300, 640, 1040, 24, 3, "chunks"),
    (600, 2688, 96, 16, 5, "random"),
    (129, 1280, 6160, 32, 40, "each"),
    (1000, 256, 1040, 8, 30, "random"),
    (2001, 640, 80, 8, 3, "chunks"),
    (17, 2560, 7680, 8, 16, "each"),
    (17, 2560, 7696, 8, 16, "each"),
])
def test_one_launch_and_two(M, K, N, R, slots, pattern):
    _say("adapter launches", M, K, N, R, slots, pattern)
    p = _problem(M * 5 + K, M, K, N, R, slots, pattern)
    d = _dev(p)
    out = _call(d)
    _check(p, out, (M, K, N, R, slots, pattern))
    assert torch.equal(_call(d, out=d["base"]), out)


@pytest.mark.parametrize("M,R", [(5, 16), (37, 40), (130, 136)])
def test_exact_on_integers(M, R):
    """Small whole numbers: every sum is exact in fp32 and every result in bf16
    (|t| <= 6, |out| <= 124, both whole)."""
    _say("adapter integers", M, R)
    g = torch.Generator().manual_seed(M)
    K, N, slots = 256, 144, 3
    x = torch.zeros(M, K)
    x[torch.arange(M), torch.randint(0, K, (M,), generator=g)] = torch.randint(-3, 4, (M,), generator=g).float()
    a = torch.randint(-2, 3, (slots, R, K), generator=g).float()
    b = torch.zeros(slots, N, R)
    b[:, torch.arange(N), torch.randint(0, R, (N,), generator=g)] = 1.0
    p = dict(base=torch.randint(-100, 101, (M, N), generator=g).bfloat16(), x=x.bfloat16(), a=a.bfloat16(),
             b=b.bfloat16(), rows=torch.randint(-1, slots, (M,), generator=g).int(),
             scales=torch.tensor([1.0, 2.0, 4.0]))
    ref, _ = _reference(p)
    assert torch.equal(_call(_dev(p)).cpu().double(), ref)


def test_in_place_and_column_slices():
    """One projection's columns of a fused output, in place; the other columns and
    the rows' ends stay as they were."""
    _say("adapter slices")
    p = _problem(3, 21, 512, 96, 16, 4)
    d = _dev(p)
    plain = _call(d)
    for width, first in ((96, 0), (288, 96), (104 + 96, 104)):
        wide = torch.full((21, width), 7.0, dtype=torch.bfloat16, device="cuda")
        part = wide[:, first:first + 96]
        part.copy_(d["base"])
        got = _call({**d, "base": part}, out=part)
        assert got.data_ptr() == part.data_ptr()
        assert torch.equal(part, plain)
        wide[:, first:first + 96] = 7.0
        assert bool((wide == 7.0).all())
    # out of place into a slice, from a slice
    src = torch.zeros(21, 128, dtype=torch.bfloat16, device="cuda")
    src[:, 16:112] = d["base"]
    dst = torch.full((21, 240), 5.0, dtype=torch.bfloat16, device="cuda")
    _call({**d, "base": src[:, 16:112]}, out=dst[:, 128:224])
    assert torch.equal(dst[:, 128:224], plain)
    assert bool((dst[:, :128] == 5.0).all()) and bool((dst[:, 224:] == 5.0).all())


def test_rows_and_adapters_do_not_reach_each_other():
    """Infinities and NaN in one request's row and in an adapter that only it uses
    leave every other row as it is without them."""
    _say("adapter isolation")
    p = _problem(5, 40, 384, 160, 24, 6, "each")
    d = _dev(p)
    clean = _call(d)
    bad = {k: v.clone() for k, v in d.items()}
    hit = d["rows"] == 2
    bad["a"][2, :, 5] = float("nan")
    bad["b"][2, 7] = float("inf")
    bad["x"][hit] = float("inf")
    bad["base"][hit] = float("nan")
    got = _call(bad)
    assert torch.equal(got[~hit], clean[~hit])
    # one row alone, its adapter shared with clean rows
    bad = {k: v.clone() for k, v in d.items()}
    bad["x"][8] = float("nan")
    got = _call(bad)
    keep = torch.arange(40, device="cuda") != 8
    assert torch.equal(got[keep], clean[keep])
    assert bool(got[8].isnan().all())


def test_repeated_calls_and_single_rows():
    """Equal bits from equal calls; a row by itself meets the same bound."""
    _say("adapter repeats")
    p = _problem(6, 70, 1024, 96, 16, 5, "random")
    d = _dev(p)
    whole = _call(d)
    for _ in range(3):
        assert torch.equal(_call(d), whole)
    for m in (0, 15, 16, 69):
        one = {**p, "base": p["base"][m:m + 1], "x": p["x"][m:m + 1], "rows": p["rows"][m:m + 1]}
        ref, bound = _reference(one)
        assert bool(((_call(_dev(one)).cpu().double() - ref).abs() <= bound).all()), m


def test_padded_rank():
    """An adapter of a smaller rank in a pool of a larger one."""
    p = _problem(8, 9, 256, 64, 8, 2, "random")
    q = dict(p)
    q["a"] = torch.cat([p["a"], torch.zeros(2, 56, 256).bfloat16()], 1)
    q["b"] = torch.cat([p["b"], torch.zeros(2, 64, 56).bfloat16()], 2)
    assert torch.equal(_call(_dev(q)), _call(_dev(p)))


def test_pool_past_four_gigabytes():
    """64-bit offsets: the last adapter of a pool of more than 2^32 bytes."""
    _say("adapter large pool")
    slots, N, R, K = 130, 65536, 256, 128
    p = _problem(9, 3, K, N, R, 1, "one")
    b = torch.zeros(slots, N, R, dtype=torch.bfloat16, device="cuda")
    a = torch.zeros(slots, R, K, dtype=torch.bfloat16, device="cuda")
    b[slots - 1] = p["b"][0].cuda()
    a[slots - 1] = p["a"][0].cuda()
    assert b.numel() * 2 > 1 << 32
    d = _dev(p)
    d.update(a=a, b=b, rows=torch.full((3,), slots - 1, dtype=torch.int32, device="cuda"),
             scales=d["scales"].repeat(slots))
    _check(p, _call(d), "large pool")


def test_graph_replays_and_streams():
    """Two captured graphs, eager calls between their replays, and a side stream."""
    import spec_verify_amd as svq
    _say("adapter graph")
    ps = [_problem(11, 12, 2048, 320, 16, 4, "chunks"), _problem(12, 130, 512, 96, 64, 9, "random")]
    ds = [_dev(p) for p in ps]
    want = [_call(d) for d in ds]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in ds:
        out = torch.empty_like(d["base"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _call(d, out=out)
            svq.adapter_add(out, d["x"], d["a"], d["b"], torch.full_like(d["rows"], -1), d["scales"], out=out)
        graphs.append(g)
        outs.append(out)
    for rep in range(4):
        for i in (0, 1):
            outs[i].zero_()
            graphs[i].replay()
            eager = _call(ds[1 - i])
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want[i]), (rep, i)
            assert torch.equal(eager, want[1 - i]), (rep, i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [_call(d) for d in ds]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refusals():
    import spec_verify_amd as svq
    d = _dev(_problem(13, 4, 256, 64, 16, 2))
    with pytest.raises(TypeError):
        _call({**d, "rows": d["rows"].long()})
    with pytest.raises(TypeError):
        _call({**d, "x": d["x"].float()})
    with pytest.raises(ValueError):
        _call({**d, "b": d["b"][:, :, :8]})
    with pytest.raises(ValueError):
        _call({**d, "scales": d["scales"][:1]})
    with pytest.raises(ValueError):
        _call({**d, "x": d["x"].cpu()})
    with pytest.raises(ValueError):
        _call(d, out=torch.empty(4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        _call({**d, "base": d["base"][:1].expand(4, 64)})
    with pytest.raises(svq.SvqError):
        _call(d, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(svq.SvqError):
        _call({**d, "base": d["base"][:, :40], "b": d["b"][:, :40].contiguous()})
    with pytest.raises(svq.SvqError):
        _call({**d, "base": d["base"][:0], "x": d["x"][:0], "rows": d["rows"][:0]})
