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


def _one_hot_pairs(slots, N, R):
    """B that takes the difference of two neighbouring ranks, another pair in each column."""
    b = torch.zeros(slots, N, R)
    n = torch.arange(N)
    first = 2 * (n % (R // 2))
    b[:, n, first], b[:, n, first + 1] = 1.0, -1.0
    return b.bfloat16(), first


@pytest.mark.parametrize("K,R,M", [(256, 8, 3), (640, 24, 37), (1280, 32, 5), (1408, 32, 5), (512, 64, 19), (384, 136, 40)])
def test_all_24_bits_of_the_intermediate_reach_the_output(K, R, M):
    """t is a whole number of 24 bits, put together from three exact parts; an output is the
    difference of two such numbers, below 2^7: every product and sum is exact in fp32, so the
    output is too."""
    _say("adapter 24 bits", K, R, M)
    g = torch.Generator().manual_seed(K + R)
    slots, N = 3, 80
    pairs = R // 2
    t = torch.randint(1 << 23, 1 << 24, (slots, pairs), generator=g)
    t = torch.stack([t, t ^ torch.randint(0, 1 << 7, (slots, pairs), generator=g)], 2).view(slots, R)
    a = torch.zeros(slots, R, K)
    at = torch.randperm(K, generator=g)[:3]
    for part in range(3):
        a[:, :, at[part]] = (t >> (8 * part) & 255).float() * 2.0 ** (8 * part)
    x = torch.zeros(M, K)
    x[:, at] = 1.0
    b, first = _one_hot_pairs(slots, N, R)
    rows = torch.randint(-1, slots, (M,), generator=g)
    p = dict(base=torch.zeros(M, N).bfloat16(), x=x.bfloat16(), a=a.bfloat16(), b=b, rows=rows.int(),
             scales=torch.tensor([1.0, 0.5, 4.0]))
    assert torch.equal(p["a"].float(), a)
    want = (t[:, first] - t[:, first + 1]).double() * p["scales"].double()[:, None]
    want = torch.cat([want, torch.zeros(1, N)])[rows]
    assert torch.equal(_call(p).double(), want)


@pytest.mark.parametrize("K,R", [(256, 8), (1280, 32), (1408, 32), (256, 64)])
def test_an_intermediate_next_to_the_largest_float(K, R):
    """t = 2^128 - 2^118, finite in fp32 and past the largest bf16: times 2^-10 it is
    2^118 - 2^108 and no infinity."""
    _say("adapter large intermediate", K, R)
    M, N = 4, 32
    x, a, b = torch.zeros(M, K), torch.zeros(1, R, K), torch.zeros(1, N, R)
    x[:, 5] = x[:, 9] = 1.0
    a[0, 3, 5], a[0, 3, 9] = 2.0 ** 128 - 2.0 ** 120, 0.75 * 2.0 ** 120
    b[0, :, 3] = 2.0 ** -10
    p = dict(base=torch.zeros(M, N).bfloat16(), x=x.bfloat16(), a=a.bfloat16(), b=b.bfloat16(),
             rows=torch.tensor([0, 0, -1, 0], dtype=torch.int32), scales=torch.ones(1))
    got = _call(p).double()
    want = 2.0 ** 118 - 2.0 ** 108   # 10 bits: half a bf16 step off at most
    assert bool((got[2] == 0).all())
    assert bool(((got[[0, 1, 3]] - want).abs() <= 2.0 ** -8 * want).all())


def test_more_items_than_one_launch_takes():
    """2^21 rows, each of 256 consecutive ones on an adapter of its own, at rank 256: 2^23
    workgroups of 512 threads are 2^32, which no launch may have.

    Bound: t passes at most 128 + 8 roundings of one fp32 step (a tile of K, the waves), the
    scale half a step, the second sum 3 * 256 + 2 terms, the output half a bf16 step."""
    import spec_verify_amd as svq
    _say("adapter 2^21 rows")
    M, K, N, R, slots = (1 << 21) + 700, 128, 16, 256, 256
    g = torch.Generator("cuda").manual_seed(3)
    n = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).bfloat16()
    base, x, a, b = n(M, N, std=3.0), n(M, K), n(slots, R, K, std=K ** -0.5), n(slots, N, R, std=R ** -0.5)
    scales = torch.rand(slots, device="cuda", generator=g) + 0.5
    rows = torch.arange(M, device="cuda", dtype=torch.int32) % slots
    out = svq.adapter_add(base, x, a, b, rows, scales)
    for s in range(slots):
        xs, bs, sc = x[s::slots].double(), base[s::slots].double(), scales[s].double()
        at, bt = a[s].double().t().contiguous(), b[s].double().t().contiguous()
        t = xs @ at
        t_err = 136 * 2.0 ** -23 * (xs.abs() @ at.abs()) + 2.0 ** -24 * t.abs()
        want = bs + sc * (t @ bt)
        bound = sc * (t_err @ bt.abs()) + 770 * 2.0 ** -23 * (bs.abs() + sc * ((t.abs() + t_err) @ bt.abs()))
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
        assert bool(((out[s::slots].double() - want).abs() <= bound).all()), s


@pytest.mark.parametrize("K", [512, 5120])
@pytest.mark.parametrize("width,first,second", [(192, 0, 96), (192, 96, 0), (320, 200, 8), (320, 0, 224)])
def test_from_one_column_slice_into_another(K, width, first, second):
    """base and out are different columns of one matrix: their rows alternate in memory and
    share no element."""
    import spec_verify_amd as svq
    _say("adapter slice to slice", K, width, first, second)
    g = torch.Generator("cuda").manual_seed(K)
    M, N, R, slots = 21, 96, 16, 4
    n = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).bfloat16()
    base, x, a, b = n(M, N, std=3.0), n(M, K), n(slots, R, K, std=K ** -0.5), n(slots, N, R, std=R ** -0.5)
    rows = torch.randint(-1, slots, (M,), device="cuda", generator=g, dtype=torch.int32)
    scales = torch.rand(slots, device="cuda", generator=g) + 0.5
    plain = svq.adapter_add(base, x, a, b, rows, scales)
    wide = torch.full((M, width), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, first:first + N] = base
    svq.adapter_add(wide[:, first:first + N], x, a, b, rows, scales, out=wide[:, second:second + N])
    assert torch.equal(wide[:, second:second + N], plain)
    assert torch.equal(wide[:, first:first + N], base)
    wide[:, first:first + N] = wide[:, second:second + N] = 7.0
    assert bool((wide == 7.0).all())
