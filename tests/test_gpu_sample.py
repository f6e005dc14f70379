"""GPU: sampling and draft acceptance against their definitions in 64 bits.

A token is a whole number and has to be equal. The weights and sums of both sides are
fp64 (a few 1e-16 of relative error per sum), the random numbers are 24-bit fractions
and the data random, so a draw within 1e-12 of a border does not occur by chance
(each row: less than 1e-6 for the largest vocabulary); where a test places draws on
borders, its weights are whole numbers and both sides are exact. A log-probability
is off by its rounding to fp32, half a step (2^-24 of it), and by what the two fp64
values differ: 1e-12."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

VOCAB = 248320


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


def _reference_row(l, u, T=1.0, k=0, p=1.0, min_p=0.0):
    """(token, logprob) of one row of float64 logits, from the definition."""
    l = np.where(np.isnan(l), -np.inf, l)
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    if len(order) == 0:
        return -1, -np.inf
    if not T > 0:
        return int(order[0]), 0.0
    if k > 0:
        order = order[:k]
    top = l[order[0]]
    e = np.where(l[order] == top, 0.0, (l[order] - top if np.isfinite(top) else np.full(len(order), -np.inf)))
    with np.errstate(over="ignore", invalid="ignore"):
        e = np.where(np.isinf(e), -np.inf, e / np.float64(T))
        w = np.exp(e)
    if p < 1:
        cum = np.cumsum(w.astype(np.longdouble))
        w = w[:1 + np.searchsorted(cum, np.longdouble(p) * cum[-1], side="left")]
    if min_p > 0:
        w = w[:max(1, int((w >= np.float64(min_p)).sum()))]
    cum = np.cumsum(w.astype(np.longdouble))
    u = 0.0 if not u >= 0 else min(np.float64(u), 1 - 2.0 ** -24)
    at = int(np.searchsorted(cum, np.longdouble(u) * cum[-1], side="right"))
    return int(order[at]), float(e[at] - np.log(cum[-1]))


def _check(logits, u, label, V=None, T=None, k=None, p=None, mp=None, got=None):
    import spec_verify_amd as svq
    to = lambda v, t: None if v is None else torch.tensor(np.asarray(v), dtype=t, device="cuda")
    u, T, p, mp = (None if v is None else np.asarray(v, np.float32) for v in (u, T, p, mp))
    if got is None:
        got = svq.sample(logits, to(u, torch.float32), to(T, torch.float32), to(k, torch.int32), to(p, torch.float32),
                         to(mp, torch.float32))
    tokens, logprobs = got[0].cpu().numpy(), got[1].cpu().numpy().astype(np.float64)
    l = logits.cpu().float().numpy().astype(np.float64)
    for m in range(l.shape[0]):
        pick = lambda v, d: d if v is None else v[m]
        t, lp = _reference_row(l[m], u[m], pick(T, 1.0), pick(k, 0), pick(p, 1.0), pick(mp, 0.0))
        assert tokens[m] == t, f"{label} row {m}: token {tokens[m]}, expected {t}"
        if np.isinf(lp):
            assert logprobs[m] == lp, f"{label} row {m}: logprob {logprobs[m]}"
        else:
            assert abs(logprobs[m] - lp) <= 2.0 ** -24 * abs(lp) + 1e-12, f"{label} row {m}: {logprobs[m]} {lp}"
    return got


def _logits(rng, M, V, kind="head"):
    if kind == "head":         # a wide floor and some likely tokens
        l = rng.normal(size=(M, V)) * 2.2
        n = min(40, V)
        for m in range(M):
            l[m, rng.choice(V, n, replace=False)] = 11 - 0.2 * np.arange(n) + rng.normal(size=n)
    elif kind == "ties":       # few values
        l = rng.integers(-3, 4, size=(M, V)).astype(float)
    elif kind == "equal":
        l = np.full((M, V), 1.5)
    elif kind == "zeros":      # both zeros, and nothing else
        l = np.where(rng.random((M, V)) < 0.5, 0.0, -0.0)
    elif kind == "tiny":       # magnitudes below every bin, more of them than the list holds
        l = rng.normal(size=(M, V)) * 1e-6
    elif kind == "tiny-few":   # few enough for the list, on both sides of zero
        l = np.where(rng.random((M, V)) < 300 / V, rng.normal(size=(M, V)) * 1e-6, rng.normal(size=(M, V)) * 3)
        l[:, ::17] = 0.0
    elif kind == "huge":       # magnitudes past every bin
        l = rng.normal(size=(M, V)) * 1e5
    elif kind == "masked":     # a grammar leaves a few tokens
        l = np.full((M, V), -np.inf)
        for m in range(M):
            at = rng.choice(V, min(V, 1 + m % 7), replace=False)
            l[m, at] = rng.normal(size=len(at))
    elif kind == "lowest":     # masked by the type's lowest value
        l = np.where(rng.random((M, V)) < 0.9, -3.3895313892515355e38, rng.normal(size=(M, V)))
    return torch.tensor(l, dtype=torch.bfloat16, device="cuda")


def _params(rng, M):
    kind = rng.integers(0, 6, M)
    T = np.where(kind == 0, 0.0, rng.uniform(0.3, 1.6, M))
    k = np.where((kind == 2) | (kind == 5), rng.integers(1, 100, M), 0)
    p = np.where((kind == 3) | (kind == 5), rng.uniform(0.3, 0.999, M), 1.0)
    mp = np.where(kind == 4, rng.uniform(0, 0.3, M), 0.0)
    return dict(T=T, k=k, p=p, mp=mp)


KINDS = ["head", "ties", "equal", "zeros", "tiny", "tiny-few", "huge", "masked", "lowest"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (7, 9), (5, 1000), (2, 8191), (3, 16411), (300, 515)])
def test_small_vocabularies(kind, M, V):
    _say("sample", kind, M, V)
    rng = np.random.default_rng(M * 1000 + V)
    l = _logits(rng, M, V, kind)
    u = rng.random(M).astype(np.float32)
    _check(l, u, (kind, "plain"))
    _check(l, u, (kind, "mixed"), **_params(rng, M))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 5, 20])
def test_whole_vocabulary(kind, M):
    _say("sample vocabulary", kind, M)
    rng = np.random.default_rng(M + 77)
    l = _logits(rng, M, VOCAB, kind)
    _check(l, rng.random(M).astype(np.float32), (kind, "mixed"), **_params(rng, M))


def test_large_batches():
    """More rows than compute units: one workgroup a row."""
    _say("sample large batches")
    rng = np.random.default_rng(4)
    for M, V in ((257, 32003), (700, 4099)):
        l = _logits(rng, M, V)
        l[3] = _logits(rng, 1, V, "huge")[0]
        l[5] = _logits(rng, 1, V, "tiny")[0]
        l[8] = -float("inf")
        _check(l, rng.random(M).astype(np.float32), (M, V), **_params(rng, M))


def test_every_token_of_a_flat_row_is_drawn_in_order():
    """Equal logits: token i is drawn for u in [i / V, (i + 1) / V), borders exact."""
    import spec_verify_amd as svq
    _say("sample flat")
    V = 256
    l = torch.full((2 * V, V), -2.0, dtype=torch.bfloat16, device="cuda")
    u = torch.arange(2 * V, device="cuda").float() / (2 * V)
    tokens, lp = svq.sample(l, u)
    assert torch.equal(tokens.cpu(), torch.arange(2 * V).int() // 2)
    assert bool((lp.cpu() == np.float32(-np.log(256.0))).all())
    # top_p on a border: half of the row exactly
    tokens, lp = svq.sample(l, u, top_p=torch.full((2 * V,), 0.5, device="cuda"))
    assert torch.equal(tokens.cpu(), torch.arange(2 * V).int() // 4)
    assert bool((lp.cpu() == np.float32(-np.log(128.0))).all())
    # top_k and min_p among equals: the lowest indices; all of them
    tokens, _ = svq.sample(l, u, top_k=torch.full((2 * V,), 64, dtype=torch.int32, device="cuda"))
    assert torch.equal(tokens.cpu(), torch.arange(2 * V).int() // 8)
    tokens, _ = svq.sample(l, u, min_p=torch.ones(2 * V, device="cuda"))
    assert torch.equal(tokens.cpu(), torch.arange(2 * V).int() // 2)


def test_parameters_at_their_ends():
    _say("sample parameter ends")
    rng = np.random.default_rng(8)
    V = 3001
    inf, nan = np.inf, np.nan
    rows = [  # u, T, k, p, min_p
        (0.0, 1, 0, 1, 0), (1 - 2.0 ** -24, 1, 0, 1, 0), (1.0, 1, 0, 1, 0), (7.0, 1, 0, 1, 0), (-3.0, 1, 0, 1, 0),
        (nan, 1, 0, 1, 0), (0.5, 0, 5, 0.5, 0.1), (0.5, -1, 0, 1, 0), (0.5, nan, 0, 1, 0), (0.7, inf, 0, 1, 0),
        (0.7, 1e-30, 0, 1, 0), (0.7, 1e-45, 0, 1, 0), (0.7, 1e30, 0, 1, 0), (0.9, 1, V, 1, 0), (0.9, 1, V + 5, 1, 0),
        (0.9, 1, -4, 1, 0), (0.9, 1, 1, 1, 0), (0.9, 1, 2 ** 31 - 1, 1, 0), (0.9, 1, 0, 0, 0), (0.9, 1, 0, -1, 0),
        (0.9, 1, 0, 1e-30, 0), (0.9, 1, 0, 1.5, 0), (0.9, 1, 0, nan, 0), (0.9, 1, 0, 1, 1), (0.9, 1, 0, 1, 2),
        (0.9, 1, 0, 1, -1), (0.9, 1, 0, 1, nan), (0.9, 1, 0, 1, 1e-30), (0.999, 1.7, 50, 0.9, 0.02),
        (1 - 2.0 ** -24, 2, 3000, 0.999999, 1e-9),
    ]
    M = len(rows)
    u, T, k, p, mp = (np.array(c) for c in zip(*rows))
    for kind in ("head", "ties", "tiny", "huge"):
        _check(_logits(rng, M, V, kind), u, kind, T=T, k=k, p=p, mp=mp)


def test_special_logits():
    """NaN and -inf are never drawn, +inf ones share the row, an empty row says so."""
    _say("sample special values")
    rng = np.random.default_rng(10)
    for V in (40, 5000, 20011):
        l = _logits(rng, 12, V).float()
        l[0] = -float("inf")
        l[1] = float("nan")
        l[2, 1::2] = float("nan")
        l[3, ::3] = -float("inf")
        l[4, 7] = float("inf")
        l[5, 3::5] = float("inf")
        l[6] = float("inf")
        l[7] = -3.3895313892515355e38
        l[8, 1:] = -float("inf")
        l[9, :-1] = -float("inf")
        l[10, :] = -float("inf")
        l[10, V // 2] = -3.3895313892515355e38
        l[11, 0], l[11, 1:] = float("inf"), -float("inf")
        l = l.bfloat16()
        for seed in range(3):
            u = np.random.default_rng(seed).random(12).astype(np.float32)
            tokens, lps = _check(l, u, V)
            assert tokens[0] == -1 and tokens[1] == -1
            _check(l, u, (V, "mixed"), **_params(np.random.default_rng(seed + 5), 12))


def test_unaligned_rows_and_slices():
    """Rows that begin anywhere, and a vocabulary cut out of wider rows whose other
    columns must not count."""
    _say("sample unaligned")
    rng = np.random.default_rng(12)
    for V, wide in ((4097, 4104), (4097, 4097), (30000, 30010), (6, 11), (15, 23)):
        for first in range(min(9, wide - V + 1)):
            full = torch.full((5, wide), 60.0, dtype=torch.bfloat16, device="cuda")
            part = full[:, first:first + V]
            part.copy_(_logits(rng, 5, V))
            _check(part, rng.random(5).astype(np.float32), (V, wide, first), **_params(rng, 5))
    flat = torch.full((5 * 4097 + 1,), 60.0, dtype=torch.bfloat16, device="cuda")[1:].view(5, 4097)
    flat.copy_(_logits(rng, 5, 4097))
    _check(flat, rng.random(5).astype(np.float32), "base off by one")


def test_frequencies():
    """Draws over a grid of u take each token as often as its probability says."""
    import spec_verify_amd as svq
    _say("sample frequencies")
    n, V = 4096, 37
    rng = np.random.default_rng(14)
    row = torch.tensor(rng.normal(size=V) * 2, dtype=torch.bfloat16, device="cuda")
    u = (torch.arange(n, device="cuda").float() + 0.5) / n
    tokens, _ = svq.sample(row.repeat(n, 1), u, torch.full((n,), 0.7, device="cuda"))
    p = torch.softmax(row.cpu().double() / 0.7, 0)  # T as fp32 differs by 2^-24 of it: nothing here
    seen = torch.bincount(tokens.cpu().long(), minlength=V).double() / n
    # a token's interval of u holds its length times n grid points, give or take one
    assert bool(((seen - p).abs() <= 1.0 / n + 1e-6).all())


def test_rows_are_independent_and_repeat():
    import spec_verify_amd as svq
    _say("sample repeats")
    rng = np.random.default_rng(15)
    l = _logits(rng, 9, 50000)
    l[2, ::2] = float("nan")
    l[4] = _logits(rng, 1, 50000, "tiny")[0]
    u = torch.rand(9, device="cuda")
    whole = svq.sample(l, u)
    for _ in range(3):
        again = svq.sample(l, u)
        assert torch.equal(again[0], whole[0]) and torch.equal(again[1], whole[1])
    for m in range(9):
        one = svq.sample(l[m:m + 1], u[m:m + 1])
        assert one[0][0] == whole[0][m]


def test_logits_past_two_gigabytes():
    import spec_verify_amd as svq
    _say("sample past 2 GiB")
    M, V = 4500, VOCAB
    assert M * V * 2 > 1 << 31
    l = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    l[:, 5::7] = -8.0
    rng = np.random.default_rng(16)
    last = _logits(rng, 2, V)
    l[M - 2:] = last
    u = torch.full((M,), 0.25, device="cuda")
    tokens, _ = svq.sample(l, u)
    assert tokens[0] == tokens[M // 2] == tokens[M - 3]
    for i in (0, 1):
        t, _ = _reference_row(last[i].cpu().float().numpy().astype(np.float64), np.float32(0.25))
        assert tokens[M - 2 + i] == t


def test_long_vocabulary():
    """2^24 tokens: a row's parts are as long as they get."""
    _say("sample 2^24 tokens")
    rng = np.random.default_rng(17)
    l = _logits(rng, 1, 1 << 24)
    _check(l, np.array([0.42], np.float32), "2^24")
    _check(l, np.array([0.99], np.float32), "2^24 chat", T=[0.8], k=[50], p=[0.95])


@pytest.mark.parametrize("M", [90, 300])
def test_rows_longer_than_their_quarters_count(M):
    """Vocabularies past 4 x 65512 tokens with a workgroup per row: the whole row is one
    count, with fewer rows than compute units and with more."""
    import spec_verify_amd as svq
    _say("sample long rows", M)
    rng = np.random.default_rng(M)
    V = 262145 + 8
    l = torch.randn(M, V, device="cuda", generator=torch.Generator("cuda").manual_seed(M)).mul_(2).bfloat16()
    l[7] = 0.5                                   # one value: more than 16 bits of it
    l[9] = _logits(rng, 1, V, "huge")[0]
    pick = [0, 3, 7, 9, M - 1]
    u = torch.rand(M, device="cuda")
    par = _params(rng, M)
    cast = lambda v, t: torch.tensor(v, dtype=t, device="cuda")
    got = svq.sample(l, u, cast(par["T"], torch.float32), cast(par["k"], torch.int32), cast(par["p"], torch.float32),
                     cast(par["mp"], torch.float32))
    _check(l[pick], u[pick].cpu().numpy(), "long rows", got=(got[0][pick], got[1][pick]),
           **{k: v[pick] for k, v in par.items()})
    plain = svq.sample(l, u)
    _check(l[pick], u[pick].cpu().numpy(), "long rows, plain", got=(plain[0][pick], plain[1][pick]))


@pytest.mark.parametrize("M", [1, 30, 300])
def test_heavy_values(M):
    """A whole vocabulary of one value, and of one value but for a few tokens: counts past
    16 bits, in every kernel."""
    _say("sample heavy values", M)
    rng = np.random.default_rng(M + 3)
    rows = min(M, 6)
    for value in (1.25, 0.0, -3e38, 1e-20, -10000.0):
        l = torch.full((M, VOCAB), value, dtype=torch.bfloat16, device="cuda")
        l[:, 100000:100003] = torch.tensor([value + 1, value, 0.25], dtype=torch.bfloat16, device="cuda")
        import spec_verify_amd as svq
        u = torch.rand(M, device="cuda")
        got = svq.sample(l, u)
        _check(l[:rows], u[:rows].cpu().numpy(), ("heavy", value), got=(got[0][:rows], got[1][:rows]))


@pytest.mark.parametrize("M,V", [(1, VOCAB), (3, 30011), (30, 60000), (100, VOCAB), (100, 601), (260, 50021), (2, 700003), (300, 280001)])
def test_changing_common_values(M, V):
    """Blocks of a row, each with one or two values in a share of it: masks, zeros, likely
    tokens, NaN; one row of two values below every bin, which is counted another way."""
    import spec_verify_amd as svq
    _say("sample common values", M, V)
    rng = np.random.default_rng(M * 7 + V)
    inf, nan = float("inf"), float("nan")
    kinds = [((-inf,), 0.95), ((-1e4,), 0.5), ((0.0,), 0.8), ((0.0, -0.0), 0.9), ((-3e38,), 0.3), ((7.5,), 0.6),
             ((nan,), 0.4), ((0.0, -inf), 0.7), ((-1e4, 0.0), 0.9), ((6.0,), 1.0), ((-inf,), 0.1), ((-3e38, -inf), 0.5),
             ((1.0,), 0.0)]
    rows = min(M, 5)
    l = rng.normal(size=(rows, V)) * 2.2
    for m in range(rows):
        at = 0
        while at < V:
            n = int(np.exp(rng.uniform(np.log(8), np.log(max(V // 3, 9)))))
            values, share = kinds[rng.integers(len(kinds))]
            here = l[m, at:at + n]
            chosen = rng.random(len(here)) < share
            here[chosen] = np.asarray(values)[rng.integers(0, len(values), int(chosen.sum()))]
            at += n
    l[rows - 1, rng.integers(0, V, 5)] = -2.5e38
    l = torch.tensor(l, dtype=torch.bfloat16, device="cuda").repeat((M + rows - 1) // rows, 1)[:M].contiguous()
    for draw in range(3):
        u = rng.random(M).astype(np.float32)
        T = np.where(rng.random(M) < 0.3, 4.0, 1.0)
        got = svq.sample(l, torch.tensor(u, device="cuda"), torch.tensor(T, dtype=torch.float32, device="cuda"))
        _check(l[:rows], u[:rows], ("common", M, V, draw), T=T[:rows], got=(got[0][:rows], got[1][:rows]))


def test_graph_replays_and_streams():
    import spec_verify_amd as svq
    _say("sample graph")
    rng = np.random.default_rng(18)
    sets = []
    for M, V in ((2, VOCAB), (40, 20001)):
        par = _params(rng, M)
        cast = lambda v, t: torch.tensor(v, dtype=t, device="cuda")
        sets.append((_logits(rng, M, V), torch.rand(M, device="cuda"), cast(par["T"], torch.float32),
                     cast(par["k"], torch.int32), cast(par["p"], torch.float32), cast(par["mp"], torch.float32)))
    want = [svq.sample(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(svq.sample(*s))
        graphs.append(g)
    for rep in range(4):
        for i in (0, 1):
            outs[i][0].fill_(-7)
            graphs[i].replay()
            eager = svq.sample(*sets[1 - i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), (rep, i)
            assert all(torch.equal(a, b) for a, b in zip(eager, want[1 - i])), (rep, i)
    # new logits and numbers in place: a replay reads them
    sets[0][0].copy_(_logits(rng, 2, VOCAB))
    sets[0][1].copy_(torch.rand(2, device="cuda"))
    graphs[0].replay()
    fresh = svq.sample(*sets[0])
    assert all(torch.equal(a, b) for a, b in zip(outs[0], fresh))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = svq.sample(*sets[1])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))


def test_sample_binding_refusals():
    import spec_verify_amd as svq
    l = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    u = torch.zeros(4, device="cuda")
    for bad in (dict(top_k=torch.zeros(4, device="cuda")), dict(temperature=torch.zeros(4, device="cuda").double())):
        with pytest.raises(TypeError):
            svq.sample(l, u, **bad)
    for bad in (dict(top_p=torch.zeros(3, device="cuda")), dict(min_p=torch.zeros(4))):
        with pytest.raises(ValueError):
            svq.sample(l, u, **bad)
    with pytest.raises(ValueError):
        svq.sample(l.t(), torch.zeros(64, device="cuda"))
    with pytest.raises(ValueError):
        svq.sample(l[:1].expand(4, 64), u)
    with pytest.raises(svq.SvqError):
        svq.sample(l[:0], u[:0])
    with pytest.raises(svq.SvqError):
        big = torch.zeros(1, VOCAB, dtype=torch.bfloat16, device="cuda")
        svq.sample(big, u[:1], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


# ---- draft acceptance -------------------------------------------------------------------

def _accept_reference(tokens, inputs, starts):
    M = len(tokens)
    accepted, following, committed = [], [], [-1] * M
    clamp = lambda v: min(max(v, 0), M)
    for b, e in zip(starts[:-1], starts[1:]):
        b, e = clamp(b), clamp(e)
        if e <= b:
            accepted.append(0)
            following.append(-1)
            continue
        n = 0
        while b + n + 1 < e and tokens[b + n] >= 0 and tokens[b + n] == inputs[b + n + 1]:
            n += 1
        accepted.append(n)
        following.append(tokens[b + n])
        committed[b:b + n + 1] = tokens[b:b + n + 1]
    return accepted, following, committed


def _accept_check(tokens, inputs, starts, label):
    import spec_verify_amd as svq
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    got = [t.cpu().tolist() for t in svq.accept_drafts(dev(tokens), dev(inputs), dev(starts))]
    want = _accept_reference(tokens, inputs, starts)
    for g, w, name in zip(got, want, ("accepted", "next", "committed")):
        assert g == list(w), (label, name)


@pytest.mark.parametrize("S,longest", [(1, 1), (1, 5), (3, 64), (5, 65), (4, 300), (33, 9), (1000, 9)])
def test_acceptance(S, longest):
    _say("accept", S, longest)
    rng = np.random.default_rng(S + longest)
    for hit in (0.0, 0.7, 1.0):
        lens = rng.integers(0, longest + 1, S)
        lens[-1] = longest
        starts = np.concatenate([[0], np.cumsum(lens)]) + 3
        M = int(starts[-1]) + 5
        tokens = rng.integers(0, VOCAB, M)
        inputs = rng.integers(0, VOCAB, M)
        ok = rng.random(M) < hit
        inputs[1:][ok[1:]] = tokens[:-1][ok[1:]]
        tokens[rng.random(M) < 0.02] = -1
        inputs[1:][tokens[:-1] < 0] = -1   # nothing drawn accepts nothing, even so
        _accept_check(tokens.tolist(), inputs.tolist(), starts.tolist(), (S, longest, hit))


def test_acceptance_clamps_starts():
    rng = np.random.default_rng(2)
    tokens = rng.integers(0, 9, 12).tolist()
    inputs = [0] + tokens[:-1]
    _accept_check(tokens, inputs, [-5, 4, 4, 20], "outside")
    _accept_check(tokens, inputs, [0, 12], "all accepted")
    _accept_check(tokens, inputs, [3, 3], "empty")
    _accept_check([4], [4], [0, 1], "one row")


# ---- together ------------------------------------------------------------------------------

def test_a_verify_chunk_from_projection_to_tokens():
    """A verify chunk as a server runs it: a quantized projection with each request's
    adapter, the quantized head, sampling with each request's setting, acceptance;
    eager and as one captured graph."""
    import oracle
    import spec_verify_amd as svq
    import synth
    _say("verify chunk")
    chunk = [5, 4, 1, 3]                # rows of each request: its last token and its drafts
    M, K, N, V, R, slots = sum(chunk), 512, 256, 4096, 16, 3
    starts = np.concatenate([[0], np.cumsum(chunk)])
    rng = np.random.default_rng(21)

    def dev(a):
        a = np.ascontiguousarray(a)
        return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()

    proj, head = synth.gen_w4a16(31, M, K, N), synth.gen_w8a16(32, M, N, V)
    bf = lambda *s, std: torch.tensor(rng.normal(size=s) * std, dtype=torch.bfloat16, device="cuda")
    x, tiled, scales = dev(proj.x).view(torch.bfloat16), svq.q4_repack(dev(proj.qweight)), dev(proj.scales)
    hw, hs = torch.from_numpy(np.ascontiguousarray(head.w)).cuda(), dev(head.scales)
    a, b = bf(slots, R, K, std=K ** -0.5), bf(slots, N, R, std=R ** -0.5)
    slot_of = np.array([2, -1, 0, 2])
    rows = torch.tensor(np.repeat(slot_of, chunk), dtype=torch.int32, device="cuda")
    ascale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    per = lambda v, t: torch.tensor(np.repeat(np.array(v), chunk), dtype=t, device="cuda")
    T, k = per([0.8, 0.0, 1.0, 1.2], torch.float32), per([20, 0, 0, 5], torch.int32)
    p, mp = per([0.9, 1.0, 1.0, 1.0], torch.float32), per([0.0, 0.0, 0.05, 0.0], torch.float32)
    u = torch.tensor(rng.random(M), dtype=torch.float32, device="cuda")
    inputs = torch.tensor(rng.integers(0, V, M), dtype=torch.int32, device="cuda")
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def step():
        y = svq.w4a16_gemm(x, tiled, scales, N)
        base = y.clone()
        svq.adapter_add(y, x, a, b, rows, ascale, out=y)
        logits = svq.w8a16_gemm(y, hw, hs)
        tokens, logprobs = svq.sample(logits, u, T, k, p, mp)
        return (base, y, logits, tokens, logprobs) + tuple(svq.accept_drafts(tokens, inputs, st))

    first = step()
    # drafts that the model agrees with, up to some place in each request
    drafts = first[3].cpu().tolist()
    for s, agree in enumerate((4, 2, 0, 1)):
        for j in range(min(agree, chunk[s] - 1)):
            inputs[starts[s] + j + 1] = drafts[starts[s] + j]
    base, y, logits, tokens, logprobs, accepted, following, committed = step()
    # each stage against its definition on the stage before it
    y64, _ = oracle.w4a16(proj.x, proj.qweight, proj.scales)
    assert oracle.gate(base.view(torch.int16).cpu().numpy().view(np.uint16), y64)[0]
    want = base.double().cpu()
    for m, s in enumerate(rows.tolist()):
        if s >= 0:
            want[m] += float(ascale[s]) * (b[s].double().cpu() @ (a[s].double().cpu() @ x[m].double().cpu()))
    assert (y.double().cpu() - want).abs().max() <= 2e-2 * want.pow(2).mean().sqrt()
    h64, _ = oracle.w8a16(y.view(torch.int16).cpu().numpy().view(np.uint16), head.w, head.scales)
    assert oracle.gate(logits.view(torch.int16).cpu().numpy().view(np.uint16), h64)[0]
    _check(logits, u.cpu().numpy(), "chunk", T=T.cpu().numpy(), k=k.cpu().numpy(), p=p.cpu().numpy(),
           mp=mp.cpu().numpy(), got=(tokens, logprobs))
    ref = _accept_reference(tokens.tolist(), inputs.tolist(), starts.tolist())
    assert [accepted.tolist(), following.tolist(), committed.tolist()] == [list(r) for r in ref]
    assert accepted.tolist()[0] == 4 and accepted.tolist()[2] == 0

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    eager = step()
    for rep in range(4):
        for t in captured:
            t.zero_()
        g.replay()
        again = step()
        torch.cuda.synchronize()
        for c, e, f in zip(captured, eager, again):
            assert torch.equal(c, e) and torch.equal(f, e), rep
