"""GPU: adjust_logits against its definition in 64 bits: changed logits within a few fp32
roundings and one of bf16, all others bit for bit."""
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
    def __init__(self, seed, rows, lengths, V, tree=True, prompts=True, penalties=True, biases=0, masks=0, pad=0):
        rng = np.random.default_rng(seed)
        S, n = len(rows), sum(rows)
        M = n + 2 * pad
        self.V = V
        self.starts = np.concatenate([[pad], pad + np.cumsum(rows)]).astype(np.int32)
        self.lengths = np.array(lengths, dtype=np.int32)
        self.logits = torch.randn(M, V, generator=torch.Generator().manual_seed(seed)).mul(2.5).bfloat16()
        common = rng.integers(0, V, 20)

        def text(*shape):
            return np.where(rng.random(shape) < 0.4, common[rng.integers(0, 20, shape)],
                            rng.integers(0, V, shape)).astype(np.int32)
        self.history, self.inputs = text(S, max(lengths) + 2), text(M)
        self.parents = None
        if tree:
            self.parents = np.full(M, -1, dtype=np.int32)
            for a, k in ref.sequences(self.starts, M):
                for i in range(1, k):
                    self.parents[a + i] = i - 1 - int(rng.random() ** 2 * i)
        self.prompt_lengths = rng.integers(0, self.lengths + 1).astype(np.int32) if prompts else None
        self.repetition = rng.uniform(0.8, 1.5, S).astype(np.float32) if penalties else None
        self.presence = rng.uniform(-1, 1, S).astype(np.float32) if penalties else None
        self.frequency = rng.uniform(-0.5, 0.5, S).astype(np.float32) if penalties else None
        self.bias = None
        if biases:
            per = rng.integers(0, biases + 1, S)
            self.bias = (np.concatenate([[0], np.cumsum(per)]).astype(np.int32),
                         rng.integers(0, V, int(per.sum())).astype(np.int32),
                         rng.uniform(-8, 8, int(per.sum())).astype(np.float32))
        self.allowed = self.mask_rows = None
        if masks:
            words = (V + 31) // 32
            self.allowed = rng.integers(0, 1 << 32, (masks, words), dtype=np.uint32).view(np.int32)
            self.allowed[0] = 0
            self.mask_rows = rng.integers(-2, masks + 2, M).astype(np.int32)

    def args(self):
        keys = ("history", "lengths", "inputs", "starts", "parents", "prompt_lengths", "repetition", "presence",
                "frequency", "bias", "allowed", "mask_rows")
        return {k: getattr(self, k) for k in keys}

    def call(self, logits=None, **change):
        import spec_verify_amd as svq

        def dev(x):
            if isinstance(x, tuple):
                return tuple(dev(y) for y in x)
            return torch.from_numpy(x).cuda() if isinstance(x, np.ndarray) else x
        a = {k: dev(x) for k, x in {**self.args(), **change}.items()}
        return svq.adjust_logits(self.logits.cuda() if logits is None else logits, **a)

    def check(self, label, got=None):
        _say("adjust", label)
        got = (self.call() if got is None else got).cpu()
        a = self.args()
        a.pop("parents")
        want, bound, inside, plain = ref.adjust(self.logits.double().numpy(), parents=self.parents, **a)
        bits = got.view(torch.int16).numpy()
        keep = self.logits.view(torch.int16).numpy()
        assert (bits[inside][plain[inside]] == keep[inside][plain[inside]]).all(), label
        x, w = got.double().numpy()[inside], want[inside]
        assert (np.isnan(x) == np.isnan(w)).all()
        same = (x == w) | np.isnan(w)
        with np.errstate(invalid="ignore"):
            over = ~same & ~(np.abs(x - w) <= bound[inside])
        assert not over.any(), (label, int(over.sum()), np.argwhere(over)[:4].tolist(), x[over][:4], w[over][:4])


CASES = [
    ("one", [1], [30], 1000, {}),
    ("nothing-before", [1], [0], 1000, {}),
    ("one-token-vocabulary", [3], [5], 1, dict(biases=2, masks=2)),
    ("seven-tokens", [3, 2], [5, 0], 7, dict(biases=3, masks=3)),
    ("chain", [5, 3], [100, 40], 5000, dict(tree=False)),
    ("tree-all", [13, 64, 1], [100, 400, 3], 5000, dict(biases=10, masks=5)),
    ("odd-vocabulary", [9, 4], [300, 50], 32001, dict(biases=30, masks=4)),
    ("vocabulary", [4, 2], [3000, 100], 248320, dict(biases=40, masks=3)),
    ("many-sequences", [1 + i % 3 for i in range(300)], [i for i in range(300)], 257, dict(biases=4, masks=9)),
    ("empty-sequences", [0, 4, 0, 0, 2], [3, 50, 9, 0, 70], 999, dict(biases=4, masks=3, pad=3)),
    ("penalties-alone", [6], [200], 3000, dict(prompts=False)),
    ("biases-alone", [6, 2], [200, 30], 3000, dict(penalties=False, prompts=False, biases=50)),
    ("masks-alone", [6, 2], [200, 30], 3003, dict(penalties=False, prompts=False, masks=4)),
    ("deep-chain", [1500], [20], 300, dict(tree=False)),
    ("wide-tree", [1500], [20], 300, {}),
    ("many-biases", [3], [20], 200, dict(biases=900)),
]


@pytest.mark.parametrize("label,rows,lengths,V,more", CASES, ids=[c[0] for c in CASES])
def test_against_the_definition(label, rows, lengths, V, more):
    Problem(900 + len(label), rows, lengths, V, **more).check(label)


def test_infinities_nan_and_lowest_values():
    p = Problem(1, [4, 3], [60, 20], 2000, biases=20, masks=2)
    low = torch.finfo(torch.bfloat16).min
    for x in (float("inf"), float("-inf"), float("nan"), low, 0.0, -0.0, -1e9):
        p.logits[:, ::3] = x
        p.check(f"logits of {x}")
    p.logits.view(torch.int16)[:, 5:50] = 0x7FA5   # a NaN of its own pattern
    p.check("a NaN's bits")


def test_tokens_outside_the_vocabulary_are_passed_over():
    p = Problem(2, [4, 3], [60, 20], 500, biases=10)
    p.history[:, ::4] = 500
    p.history[:, 1::4] = -1
    p.inputs[::2] = 2 ** 31 - 1
    p.bias[1][::2] = -2 ** 31
    p.check("tokens")


def test_lengths_starts_and_parents_are_clamped():
    p = Problem(3, [4, 3], [60, 20], 500, biases=10, masks=2)
    p.lengths[:] = [10 ** 6, -4]
    p.prompt_lengths[:] = [10, -4]
    p.check("lengths")
    p.starts[0], p.starts[2] = -7, 50
    p.check("starts")
    p.parents[:] = [4, 0, -2, 2 ** 31 - 1, 0, 1, -2 ** 31]
    p.check("parents")
    p.bias[0][:] = [-5, 3, 10 ** 6]
    p.check("bias starts")


def test_counts_of_one_token_over_and_over():
    p = Problem(4, [6], [20000], 300)
    p.history[:] = 7
    p.inputs[:] = 7
    p.frequency[:] = 0.001
    p.check("one token")


@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("V,ld", [(1000, 1000), (1001, 1001), (1000, 1013), (77, 1024)])
def test_columns_of_wider_matrices_and_in_place(offset, V, ld):
    _say("columns", offset, V, ld)
    p = Problem(5, [5, 9], [60, 20], V, biases=10, masks=2)
    M = len(p.logits)
    want = p.call()
    p.check("contiguous", want)

    def wide():
        w = torch.full((M, ld + 16), 3.0, dtype=torch.bfloat16, device="cuda")
        return w, w[:, offset:offset + V]
    a, src = wide()
    src.copy_(p.logits)
    b, dst = wide()
    p.call(src, out=dst)
    assert torch.equal(dst.contiguous().view(torch.int16), want.view(torch.int16))
    p.call(p.logits.cuda(), out=dst)          # rows of one and of another alignment
    assert torch.equal(dst.contiguous().view(torch.int16), want.view(torch.int16))
    p.call(src, out=src)
    assert torch.equal(src.contiguous().view(torch.int16), want.view(torch.int16))
    for w in (a, b):
        w[:, offset:offset + V] = 3.0
        assert (w == 3.0).all()


def test_rows_of_no_sequence_are_left():
    p = Problem(6, [5, 3], [20, 9], 700, masks=3, pad=4)
    out = torch.full((16, 700), 5.0, dtype=torch.bfloat16, device="cuda")
    p.check("padded", p.call(out=out))
    assert (out[:4] == 5).all() and (out[12:] == 5).all()


def test_graph_replays_and_streams():
    p = Problem(7, [5, 30], [700, 300], 40000, biases=20, masks=4)
    want = p.call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = p.call()
    s.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    dev = {k: tuple(torch.from_numpy(y).cuda() for y in x) if isinstance(x, tuple) else torch.from_numpy(x).cuda()
           for k, x in p.args().items()}
    logits = p.logits.cuda()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = p.call(logits, **dev)
    for lengths in ([700, 300], [3, 0], [700, 1]):
        p.lengths[:] = lengths
        dev["lengths"].copy_(torch.from_numpy(p.lengths))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        p.check(f"replay {lengths}", out)
        assert torch.equal(p.call().view(torch.int16), out.view(torch.int16))


def test_refusals():
    import spec_verify_amd as svq
    p = Problem(8, [4], [40], 100, biases=3, masks=2)
    with pytest.raises(ValueError, match="together"):
        p.call(allowed=None)
    with pytest.raises(ValueError, match="words"):
        p.call(allowed=torch.zeros(2, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="repetition must be"):
        p.call(repetition=torch.ones(1, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        p.call(inputs=torch.zeros(5, dtype=torch.int32, device="cuda"))
    x = p.logits.cuda()
    big = torch.zeros(5, 100, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(svq.SvqError, match="status 7"):
        p.call(big[:4], out=big[1:])
    with pytest.raises(ValueError, match="out must have shape"):
        p.call(x, out=big)
