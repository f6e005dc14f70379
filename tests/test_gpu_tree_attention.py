"""GPU: attention of a tree of drafts to a paged cache (tree_attention) against its
definition in 64 bits: every element within a bound of its own (fp32 scores and sums, bf16
weights and result), the whole within what independent roundings add up to, and who sees
whom by values that count exactly."""
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


class Problem:
    """Inputs of one call on the device; `rows` and `lengths` per sequence, `pad` rows of no sequence on either side."""

    def __init__(self, seed, rows, lengths, H=6, G=2, D=64, page=16, e4m3=False, tree=True, window=0, sinks=0, pad=0,
                 spread=1.0):
        import spec_verify_amd as svq
        self.svq = svq
        rng = np.random.default_rng(seed)
        self.H, self.G, self.D, self.page, self.window, self.sinks = H, G, D, page, window, sinks
        S, n = len(rows), sum(rows)
        M = n + 2 * pad
        self.starts = np.concatenate([[pad], pad + np.cumsum(rows)]).astype(np.int32)
        self.lengths = np.array(lengths, dtype=np.int32)
        self.parents = None
        if tree:
            self.parents = np.full(M, -1, dtype=np.int32)
            for a, k in ref.sequences(self.starts, M):
                for i in range(1, k):
                    self.parents[a + i] = i - 1 - int(rng.random() ** 2 * i)
        most = max(1, max(-(-l // page) for l in lengths))
        used = sum(-(-l // page) for l in lengths)
        order = rng.permutation(used + 3).astype(np.int32)
        self.table = np.full((S, most), -7, dtype=np.int32)  # entries past a sequence's pages name none
        at = 0
        for s, l in enumerate(lengths):
            c = -(-l // page)
            self.table[s, :c] = order[at:at + c]
            at += c
        g = torch.Generator().manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g)
        self.q = (normal(M, H, D) * spread).bfloat16()
        self.k, self.v = normal(M, G, D).bfloat16(), normal(M, G, D).bfloat16()
        self.scales = [None, None]
        self.caches = []
        for i in range(2):
            c = normal(used + 3, page, G, D)
            if e4m3:
                self.scales[i] = torch.rand(G, generator=g) * 0.05 + 0.01
                self.caches.append((c / self.scales[i][:, None]).to(torch.float8_e4m3fn))
            else:
                self.caches.append(c.bfloat16())

    def call(self, **change):
        def dev(x):
            return None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()
        a = dict(q=self.q, k=self.k, v=self.v, k_cache=self.caches[0], v_cache=self.caches[1], page_table=self.table,
                 lengths=self.lengths, starts=self.starts, parents=self.parents, window=self.window, sinks=self.sinks,
                 k_scale=self.scales[0], v_scale=self.scales[1])
        a.update(change)
        tensors = [n for n in a if n not in ("window", "sinks", "scale", "out", "workspace", "lengths")]
        a = {n: dev(x) if n in tensors or isinstance(x, np.ndarray) else x for n, x in a.items()}
        return self.svq.tree_attention(**a)

    def expected(self, scale=None):
        caches = []
        for c, s in zip(self.caches, self.scales):
            c = c.double()
            caches.append((c if s is None else c * s.double()[:, None]).numpy())
        return ref.attend(self.q.double().numpy(), self.k.double().numpy(), self.v.double().numpy(), *caches, self.table,
                          self.lengths, self.starts, self.parents, self.D ** -0.5 if scale is None else scale, self.window,
                          self.sinks)

    def check(self, label, got=None, overall=True):
        _say("attend", label)
        got = (self.call() if got is None else got).double().cpu().numpy()
        want, bound, inside = self.expected()
        got, want, bound = got[inside], want[inside], bound[inside]
        assert np.isfinite(got).all() == np.isfinite(want).all()
        over = np.abs(got - want) > bound
        assert not over.any(), (label, int(over.sum()), np.argwhere(over)[:4].tolist(), got[over][:4], want[over][:4])
        if overall and got.size >= 2000:
            # values are independent of mean zero, so the weights' roundings and the result's, each 2^-8 / sqrt(3)
            # at most in the mean square, give sqrt(2 / 3) 2^-8 together
            rel = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert rel < 2.0 ** -8, (label, rel)


# row counts from one to several blocks of rows, lengths around tiles of 64 and of nothing
SHAPES = [
    ("one-token", [1], [1], {}),
    ("one-token-no-cache", [1], [0], {}),
    ("one-token-64", [1], [64], {}),
    ("one-token-long", [1], [5000], {}),
    ("chain-5", [5], [1000], dict(tree=False)),
    ("chain-of-nothing-cached", [5, 3], [0, 0], dict(tree=False)),
    ("tree-13", [13], [63], {}),
    ("tree-64", [64], [65], {}),
    ("tree-65", [65], [191], {}),
    ("tree-200", [200], [100], dict(H=4, G=2)),
    ("ragged", [1, 7, 30, 2, 64], [0, 1, 127, 128, 900], {}),
    ("empty-sequences", [0, 3, 0, 0, 5, 0], [9, 70, 3, 0, 200, 1], dict(pad=3)),
    ("many-sequences", [1 + i % 3 for i in range(70)], [i * 3 for i in range(70)], dict(H=2, G=1)),
    ("one-head-each", [9, 4], [100, 333], dict(H=3, G=3)),
    ("group-of-12", [5, 2], [100, 333], dict(H=12, G=1)),
    ("group-of-17", [3, 6], [100, 40], dict(H=17, G=1)),
    ("blocks-of-16", [2, 2], [300, 77], dict(H=8, G=1, D=256)),
    ("blocks-of-32", [5], [300], dict(H=12, G=2, D=256)),
    ("blocks-of-64", [10], [300], dict(H=12, G=2, D=256)),
    ("blocks-of-128", [40, 64], [300, 129], dict(H=12, G=2, D=256)),
    ("d-128", [12, 1, 33], [130, 64, 500], dict(D=128)),
    ("page-1", [4, 5], [70, 129], dict(page=1)),
    ("page-7", [4, 5], [70, 129], dict(page=7)),
    ("page-100", [4, 5], [70, 1290], dict(page=100)),
    ("page-1000", [4, 5], [70, 1290], dict(page=1000)),
    ("window-1", [9], [100], dict(window=1)),
    ("window-5-sinks-2", [9, 20], [100, 3], dict(window=5, sinks=2)),
    ("window-64", [20], [500], dict(window=64)),
    ("window-300-sinks-4", [30, 5], [1000, 290], dict(window=300, sinks=4)),
    ("window-50-sinks-200", [20, 9], [1000, 100], dict(window=50, sinks=200)),
    ("window-chain", [20, 3], [500, 63], dict(window=8, sinks=3, tree=False)),
    ("window-past-all", [20], [500], dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1)),
    ("peaked", [6, 6], [700, 64], dict(spread=8.0)),
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("label,rows,lengths,more", SHAPES, ids=[s[0] for s in SHAPES])
def test_against_the_definition(label, rows, lengths, more, e4m3):
    Problem(5000 + len(label), rows, lengths, e4m3=e4m3, **more).check(label)


def _count_problem(rows, lengths, e4m3, **more):
    """Equal weights (q is zero) and values that are unit vectors: out counts who is seen."""
    p = Problem(77, rows, lengths, e4m3=e4m3, **more)
    p.q.zero_()
    D = p.D
    for s, (a, n) in enumerate(ref.sequences(p.starts, len(p.v))):
        for j in range(n):
            p.v[a + j] = torch.eye(D)[(lengths[s] + j) % D].bfloat16()
    c = torch.zeros(p.caches[1].shape)
    for s, l in enumerate(lengths):
        for j in range(l):
            c[p.table[s, j // p.page], j % p.page] = torch.eye(D)[j % D]
    p.caches[1] = c.to(p.caches[1].dtype)
    if e4m3:
        p.scales[1] = torch.ones(p.G)
    return p


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows,lengths,more", [
    ([13, 40], [60, 130], {}), ([13, 40], [60, 130], dict(tree=False)), ([70], [10], dict(H=4, G=2)),
    ([13, 40], [60, 130], dict(window=9, sinks=3)), ([13, 40], [60, 130], dict(window=9, sinks=3, tree=False)),
    ([20], [300], dict(window=100, sinks=70, page=7)), ([20], [30], dict(window=3, sinks=45)),
    ([300], [5], dict(window=90, sinks=2, H=1, G=1)), ([1100], [70], dict(H=1, G=1)),
    ([1100], [3], dict(H=1, G=1, window=40)),
])
def test_who_sees_whom(rows, lengths, e4m3, more):
    _say("count", rows, lengths, more)
    p = _count_problem(rows, lengths, e4m3, **more)
    got = p.call().double().cpu().numpy()
    want, _, _ = p.expected()
    # a count over a count: one fp32 reciprocal and product, then bf16
    assert (np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -21)).all()
    assert ((got == 0) == (want == 0)).all()


def test_pages_that_name_nothing_are_not_seen():
    p = Problem(3, [6, 4], [200, 90], page=16)
    for bad in (-1, p.caches[0].shape[0], 2 ** 31 - 1, -2 ** 31):
        p.table[0, 3] = bad
        p.check(f"page {bad}")
    p.table[:] = -1
    p.check("no page at all")


def test_lengths_and_starts_are_clamped():
    p = Problem(4, [6, 4], [64, 64], page=16)
    p.lengths[:] = [10 ** 9, -5]
    p.check("lengths")
    p = Problem(4, [6, 4], [64, 64], page=16)
    p.starts[0], p.starts[2] = -3, 100
    p.check("starts")


def test_parents_that_name_nothing_are_none():
    p = Problem(6, [9], [40])
    p.parents[:] = [5, 0, -3, 3, 2 ** 31 - 1, 1, 100, 6, -2 ** 31]
    p.check("parents")


def test_rows_of_no_sequence_and_other_columns_are_left():
    p = Problem(8, [5, 3], [70, 10], pad=4)
    wide = torch.full((16, 3 * p.H * p.D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, p.H * p.D:2 * p.H * p.D].view(16, p.H, p.D)
    p.check("wide", p.call(out=out))
    host = wide.cpu().float().view(16, 3, -1)
    assert (host[:, [0, 2]] == 7).all() and (host[:4] == 7).all() and (host[12:] == 7).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_fused_projections_and_cache_orders(e4m3):
    """q, k and v as columns of one fused output; caches head-major, token-major, and K beside V."""
    p = Problem(9, [6, 11], [100, 300], e4m3=e4m3, H=6, G=2)
    M, H, G, D = len(p.q), 6, 2, 64
    fused = torch.cat([p.k.reshape(M, -1), p.v.reshape(M, -1), p.q.reshape(M, -1)], 1).cuda()
    cols = fused.split([G * D, G * D, H * D], 1)
    k, v, q = (c.view(M, -1, D) for c in cols)
    want = p.call()
    p.check("contiguous", want)
    same = lambda **c: torch.equal(p.call(**c).view(torch.int16), want.view(torch.int16))
    assert same(q=q, k=k, v=v)
    dev = [c.cuda() for c in p.caches]
    heads = [c.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for c in dev]
    assert same(k_cache=heads[0], v_cache=heads[1])
    both = torch.stack([c.view(torch.uint8) if e4m3 else c for c in dev], 2)
    assert same(k_cache=both[:, :, 0], v_cache=both[:, :, 1])
    assert same(k_cache=heads[0], v_cache=both[:, :, 1].view(torch.float8_e4m3fn) if e4m3 else both[:, :, 1])
    twice = [torch.cat([c, c], 1)[:, :c.shape[1]] for c in dev]   # pages apart
    assert same(k_cache=twice[0], v_cache=twice[1])
    table = torch.full((2, p.table.shape[1] + 5), 1, dtype=torch.int32, device="cuda")
    table[:, :p.table.shape[1]] = torch.from_numpy(p.table)
    assert same(page_table=table[:, :p.table.shape[1]])


def test_scale_and_head_scales():
    p = Problem(10, [5], [200], e4m3=True)
    for name, at in (("k_scale", 0), ("v_scale", 1)):
        keep = p.scales[at]
        p.scales[at] = None
        if at == 0:
            p.caches[0] = (p.caches[0].float() * 0.03).to(torch.float8_e4m3fn)
        p.check(f"without {name}")
        p.scales[at] = keep
    p = Problem(11, [5], [200])
    got = p.call(scale=0.01).double().cpu().numpy()
    want, bound, _ = p.expected(scale=0.01)
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("H,rows,D", [(2, [9, 20], 64), (12, [9, 20], 64), (24, [9, 30], 256)])
def test_infinities_and_nan_reach_only_who_sees_them(H, rows, D, e4m3):
    """In what no row sees (a page's other tokens, pages of nobody), in drafts that some rows see, at
    the edge of a window: rows that do not see them keep their bits; rows that do are as defined."""
    p = Problem(12, rows, [50, 130], H=H, G=2, D=D, e4m3=e4m3, window=40, sinks=5)
    clean = p.call().cpu()
    odd = torch.tensor([float("inf"), float("-inf"), float("nan")])
    used = set(p.table[p.table >= 0].tolist())
    ugly = [c.clone() for c in p.caches]
    for c in ugly:  # E4M3 has NaN alone
        for page in set(range(c.shape[0])) - used:
            c[page] = float("nan")
        for s, l in enumerate([50, 130]):
            c[p.table[s, (l - 1) // 16], (l - 1) % 16 + 1:] = float("nan")
            for j in range(6, l - 39 - 1):
                c[p.table[s, j // 16], j % 16] = float("nan")
    _say("nonfinite where nobody looks")
    got = p.call(k_cache=ugly[0].cuda(), v_cache=ugly[1].cuda()).cpu()
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))
    # a draft of the second sequence, and the oldest token of the first one's window (seen by its first row)
    for name in ("v", "k"):
        for i, x in enumerate(odd):
            _say("nonfinite", name, float(x))
            q = Problem(12, rows, [50, 130], H=H, G=2, D=D, e4m3=e4m3, window=40, sinks=5)
            t = getattr(q, name)
            t[rows[0] + 4, :, i] = x
            if not e4m3 or i == 2:
                q.caches[name == "v"][q.table[0, 11 // 16], 11 % 16, :, i] = x
            _say("call")
            got = q.call().double().cpu().numpy()
            want, bound, _ = q.expected()
            same = np.zeros(got.shape, dtype=bool)
            for a, n in ref.sequences(q.starts, len(got)):
                for r, path in enumerate(ref.paths(q.parents[a:a + n], n)):
                    hit = 4 in path if a else (e4m3 and i != 2) is False and len(path) == 1
                    if not hit:
                        same[a + r] = True
            assert (got[same] == clean.double().numpy()[same]).all(), (name, float(x))
            assert (np.isnan(got) == np.isnan(want)).all(), (name, float(x))
            fine = np.isfinite(want)
            assert (np.isfinite(got) == fine).all() and (got[~fine & ~np.isnan(want)] == want[~fine & ~np.isnan(want)]).all()
            assert (np.abs(got - want)[fine] <= bound[fine]).all(), (name, float(x))


def test_scores_of_minus_infinity_have_no_weight():
    """A visible key that gives -inf counts as unseen; a row that sees nothing else is zero."""
    p = Problem(13, [3], [70], H=2, G=1, tree=False)
    p.q[:] = p.q.abs() + 0.1
    p.caches[0][p.table[0, 1], 3:5] = float("-inf")
    p.check("two cached keys", overall=False)
    p.caches[0][:] = float("-inf")
    p.k[:] = float("-inf")
    got = p.call().float().cpu()
    assert (got == 0).all()


def test_long_cache_past_32_bits():
    """A pool of more than 4 GiB: pages at both ends of it, bf16 and E4M3."""
    for dtype, size in ((torch.bfloat16, 2), (torch.float8_e4m3fn, 1)):
        page, G, D = 64, 2, 256
        pages = (9 << 29) // (page * G * D * size) + 5   # 4.5 GiB
        _say("pool of", pages, "pages", dtype)
        p = Problem(14, [5], [300], H=4, G=G, D=D, page=page, e4m3=size == 1)
        at = [pages - 1, 0, pages // 2, pages - 2, 1]
        big = [torch.zeros(pages, page, G, D, dtype=torch.uint8 if size == 1 else dtype, device="cuda") for _ in range(2)]
        for b, c in zip(big, p.caches):
            for i, to in enumerate(at):
                b[to] = (c.view(torch.uint8) if size == 1 else c)[p.table[0, i]].cuda()
        table = torch.tensor([at], dtype=torch.int32, device="cuda")
        p.check("long pool", p.call(k_cache=big[0], v_cache=big[1], page_table=table))
        del big


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page,window,sinks", [(1, 0, 0), (1, 1700, 300), (3, 0, 0)])
def test_more_pages_than_are_kept_at_a_time(page, window, sinks, e4m3):
    """Workgroups that pass thousands of table entries of a sequence."""
    n = 32 if page == 1 else 16
    Problem(20, [1 + i % 2 for i in range(n)], [2500 * page - 7 * i for i in range(n)], H=16, G=8, page=page, e4m3=e4m3,
            window=window, sinks=sinks).check(f"pages of {page}")


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30, 3.0])
def test_any_scale(scale):
    p = Problem(21, [5, 20], [200, 3], tree=True)
    _say("scale", scale)
    got = p.call(scale=scale).double().cpu().numpy()
    want, bound, _ = p.expected(scale=scale)
    assert (np.abs(got - want) <= bound).all()


def test_two_streams_at_once():
    a, b = Problem(22, [64, 30], [3000, 900], H=12, G=2, D=256), Problem(23, [5], [20000], H=12, G=2, D=128)
    want = [x.call() for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = []
    for x in (a, b):
        held.append({k: v for k, v in dict(
            q=x.q.cuda(), k=x.k.cuda(), v=x.v.cuda(), k_cache=x.caches[0].cuda(), v_cache=x.caches[1].cuda(),
            page_table=torch.from_numpy(x.table).cuda(), lengths=torch.from_numpy(x.lengths).cuda(),
            starts=torch.from_numpy(x.starts).cuda(), parents=torch.from_numpy(x.parents).cuda()).items()})
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                outs[i].append(x.call(**held[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o.view(torch.int16), want[i].view(torch.int16)) for o in outs[i])


def test_starts_that_do_not_ascend_write_nothing():
    p = Problem(24, [20, 30, 14], [500, 3, 70], tree=True)
    for starts in ([0, 64, 0, 64], [0, 20, 10, 64], [64, 0, 64, 0]):
        p.starts = np.array(starts, dtype=np.int32)
        _say("starts", starts)
        out = torch.full_like(p.q, 7.0).cuda()
        p.call(out=out)
        torch.cuda.synchronize()
        assert (out == 7.0).all()


def test_starts_outside_are_clamped():
    p = Problem(25, [20, 30, 14], [500, 3, 70], tree=True)
    want = p.call()
    p.starts = np.array([-5, 20, 50, 2 ** 31 - 1], dtype=np.int32)
    assert torch.equal(p.call().view(torch.int16), want.view(torch.int16))


def test_a_pool_of_one_page_has_any_stride():
    """Of a page that has no other beside it the stride is not looked at, 4 GiB or more included."""
    p = Problem(26, [3], [10], tree=True)
    p.table[0, 0] = 0
    p.caches = [c[:1].contiguous() for c in p.caches]
    want = p.call()
    wide = [c.cuda().as_strided(c.shape, (1 << 40,) + c.stride()[1:]) for c in p.caches]
    got = p.call(k_cache=wide[0], v_cache=wide[1])
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    p.check("one page")


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_pages_shared_by_sequences(e4m3):
    p = Problem(27, [5, 9, 2], [300, 280, 299], H=12, G=2, D=256, e4m3=e4m3)
    p.table[1, :10] = p.table[0, :10]
    p.table[2, :15] = p.table[0, :15]
    p.check("a common prefix")


@pytest.mark.parametrize("rows,lengths", [([200, 1, 1, 1, 1, 1], [70, 3000, 0, 1, 64, 900]), ([1] * 40 + [600], [50] * 41)])
def test_sequences_of_very_different_rows(rows, lengths):
    """The shape follows the average: long ones take many blocks, some members of a team none."""
    Problem(28, rows, lengths, H=8, G=1, D=64).check(f"{max(rows)} rows of {sum(rows)}")
    Problem(29, rows, lengths, H=8, G=1, D=64, window=40, sinks=5, e4m3=True).check(f"{max(rows)} rows of {sum(rows)}, window")


def test_split_sequences_are_as_whole_ones():
    """One sequence over all workgroups, and the same among many, where it has few: the same within the bound."""
    one = Problem(15, [5], [20000], H=12, G=2, D=128)
    one.check("alone")
    many = Problem(15, [5] + [2] * 40, [20000] + [300] * 40, H=12, G=2, D=128)
    many.check("among others")


def test_determinism_streams_and_callers_workspace():
    import spec_verify_amd as svq
    p = Problem(16, [64, 5, 30], [3000, 10, 700], H=12, G=2, D=128)
    want = p.call()
    need = svq.tree_attention_workspace_bytes(99, 3, 12, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(p.call(workspace=ws).view(torch.int16), want.view(torch.int16))
    assert (ws[:256 * 1024] == 255).all()   # the counters of the GEMMs
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = p.call()
    s.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_graph_replays_follow_the_lengths():
    """A captured call reads lengths, tables and trees when it is replayed; two graphs share nothing."""
    p = Problem(17, [20, 5], [700, 300], H=12, G=2, D=128)
    r = Problem(18, [64], [2000], H=12, G=2, D=128)
    held = []
    for x in (p, r):
        dev = dict(q=x.q.cuda(), k=x.k.cuda(), v=x.v.cuda(), k_cache=x.caches[0].cuda(), v_cache=x.caches[1].cuda(),
                   page_table=torch.from_numpy(x.table).cuda(), lengths=torch.from_numpy(x.lengths).cuda(),
                   starts=torch.from_numpy(x.starts).cuda(), parents=torch.from_numpy(x.parents).cuda())
        x.call(**dev)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = x.call(**dev)
        held.append((x, dev, g, out))
    torch.cuda.synchronize()
    for lengths in ([700, 300], [64, 0], [1, 300], [700, 299]):
        p.lengths[:] = lengths
        held[0][1]["lengths"].copy_(torch.from_numpy(p.lengths))
        for x, dev, g, out in held:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for x, dev, g, out in held:
            x.check(f"replay {lengths}", out)
            assert torch.equal(x.call().view(torch.int16), out.view(torch.int16))


def test_refusals():
    import spec_verify_amd as svq
    p = Problem(19, [4], [40])
    with pytest.raises(ValueError, match="workspace"):
        p.call(workspace=torch.empty(10, dtype=torch.uint8))
    with pytest.raises(svq.SvqError, match="status 8"):
        p.call(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous rows"):
        p.call(q=p.q.cuda().transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="must be on"):
        p.call(lengths=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="v_cache must be"):
        p.call(v_cache=p.caches[1].cuda().float())
    with pytest.raises(svq.SvqError, match="status 10"):
        p.call(k_scale=torch.ones(2, device="cuda"))
    q = p.q.cuda()
    with pytest.raises(svq.SvqError, match="status 7"):
        p.call(q=q, out=q)
