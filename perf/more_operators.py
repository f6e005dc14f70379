"""Measured cases of verifying trees of drafted tokens.

A verify chunk holds, for each sequence, its last committed token and drafts that
branch from it. Three steps depend on that tree: every row attends to the sequence's
paged cache and to its own ancestors (``tree_attention``, over the whole cache or over a
sliding window and a few first tokens), the head's logits are adjusted by what stands
before the row (``adjust_logits``: penalties for repeated tokens, biases, grammar
masks), and the longest path that the main model's samples follow is accepted
(``accept_tree``).

``own`` selects the framework's kernels; otherwise the operators run in their plain
form, elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

HEADS, KV_HEADS, HEAD_DIM = 24, 4, 256
VOCAB = 248320


# ---- cases -------------------------------------------------------------------

def _attend(name, streams, nodes, length, heads=HEADS, kv_heads=KV_HEADS, dim=HEAD_DIM, page=16, cache="bf16",
            tree=True, ragged="", window=0, sinks=0):
    """`streams` sequences of `nodes` rows over caches of `length` tokens; ragged: "lengths"
    spreads the caches' lengths, "all" the trees' sizes too."""
    return {"name": name, "op": "attend", "streams": streams, "nodes": nodes, "length": length, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache, "tree": tree, "ragged": ragged,
            "window": window, "sinks": sinks}


def _adjust(name, streams, nodes, length, V=VOCAB, tree=True, ragged="", masked=0, biases=0):
    """Rows of `nodes` per stream behind histories of about `length` tokens; every
    `masked`-th stream under a grammar (0: none), `biases` biased tokens a stream."""
    return {"name": name, "op": "adjust", "streams": streams, "nodes": nodes, "length": length, "V": V,
            "tree": tree, "ragged": ragged, "masked": masked, "biases": biases}


def _accept(name, streams, nodes, ragged=""):
    return {"name": name, "op": "accept", "streams": streams, "nodes": nodes, "ragged": ragged}


def listed():
    return [
        # one token of one chat request: the smallest call, latency counts
        _attend("attend-decode-1", 1, 1, 1500),
        # one request's chunk of five behind a long document: one long axis to split
        _attend("attend-verify-5-long", 1, 5, 65000, page=64, tree=False),
        # batched verify, 32 requests of 1 + 3 tokens, lengths of their own, 8-bit cache
        _attend("attend-batch-128-fp8", 32, 4, 8192, cache="e4m3", tree=False, ragged="lengths"),
        # wide trees for many requests: as many products as bytes
        _attend("attend-tree-32x64", 32, 64, 4096, page=32, ragged="lengths"),
        # sliding window with sinks over long caches, other heads and pages
        _attend("attend-window-16x24", 16, 24, 40000, heads=20, dim=128, page=128, window=2000, sinks=4),
        # odd everything: heads that fill no tile, pages of seven tokens, trees of one to thirteen
        _attend("attend-odd", 7, 13, 777, heads=9, kv_heads=3, dim=64, page=7, cache="e4m3", ragged="all"),
        # one token of one chat request with penalties and some biased tokens
        _adjust("adjust-decode-1", 1, 1, 1500, biases=20),
        # batched verify: long histories, every other request under a grammar
        _adjust("adjust-batch-128", 32, 4, 8192, tree=False, ragged="lengths", masked=2, biases=20),
        # wide trees of eight requests, each node behind its own path
        _adjust("adjust-tree-8x64", 8, 64, 4096, masked=4),
        # one small tree; wide trees of a batch; a large serving batch of trees of all sizes
        _accept("accept-tree-1x8", 1, 8),
        _accept("accept-tree-32x64", 32, 64),
        _accept("accept-tree-2048-ragged", 2048, 32, ragged="all"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "adjust", "adjust", "accept"])
    if op == "attend":
        kv_heads = rng.randint(1, 8)
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 8, 12])
        dim = rng.choice([64, 128, 256])
        nodes, streams = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        # no more cached values than the listed batch's, no more products than the listed trees'
        most = min(65000, (32 * 8192 * KV_HEADS * HEAD_DIM) // (streams * kv_heads * dim),
                   (32 * 64 * 4096 * HEADS * HEAD_DIM) // (streams * nodes * heads * dim))
        windowed = rng.random() < 0.3
        c = _attend("", streams, nodes, _log_int(rng, 1, max(1, most)), heads, kv_heads, dim,
                    page=rng.choice([1, 7, 16, 16, 32, 64, 100, 128, 256]), cache=rng.choice(["bf16", "e4m3"]),
                    tree=rng.random() < 0.6, ragged=rng.choice(["", "lengths", "all"]),
                    window=_log_int(rng, 1, 8192) if windowed else 0, sinks=rng.randint(0, 70) if windowed else 0)
    elif op == "adjust":
        streams = _log_int(rng, 1, 64)
        nodes = _log_int(rng, 1, max(1, min(64, 512 // streams)))
        c = _adjust("", streams, nodes, _log_int(rng, 1, 32768), _log_int(rng, 100, VOCAB), tree=rng.random() < 0.6,
                    ragged=rng.choice(["", "lengths", "all"]), masked=rng.choice([0, 0, 1, 2, 3]), biases=rng.choice([0, 0, 3, 40]))
    else:
        c = _accept("", _log_int(rng, 1, 2048), _log_int(rng, 1, 64), rng.choice(["", "all"]))
    del c["name"]
    return c


def _sizes(case):
    """(rows of each stream, tokens before each stream's rows)."""
    S, n, L = case["streams"], case["nodes"], case.get("length", 0)
    rows = [1 + (i * 7 + n - 1) % n for i in range(S)] if case["ragged"] == "all" else [n] * S
    if not case["ragged"]:
        return rows, [L] * S
    # from a quarter of the length to seven quarters
    return rows, [max(1, int(L * (0.25 + 1.5 * ((i * 5) % S + 0.5) / S))) for i in range(S)]


# ---- inputs --------------------------------------------------------------------

def _trees(case, rows, gen, dev):
    """Parents within each stream (-1: the first row): a chain, or nodes that hang on an
    earlier one, more often on one of the last."""
    M, n = sum(rows), max(rows)
    i = torch.arange(n, device=dev)[None].expand(len(rows), n)
    if case.get("tree", True):
        back = (torch.rand(len(rows), n, generator=gen, device=dev) ** 2 * i).long()
        parents = torch.where(i > 0, i - 1 - back, -1)
    else:
        parents = i - 1
    keep = i < torch.tensor(rows, device=dev)[:, None]
    parents = parents[keep].to(torch.int32)
    assert parents.shape[0] == M
    return parents


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    def integers(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=gen, device=dev, dtype=torch.int32)

    rows, lengths = _sizes(case)
    S, M = len(rows), sum(rows)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=dev)
    parents = _trees(case, rows, gen, dev)
    st = {"case": case, "starts": starts, "parents": parents,
          "lengths": torch.tensor(lengths, dtype=torch.int32, device=dev)}
    if case["op"] == "attend":
        H, G, D, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
        most = -(-max(lengths) // page)
        pool = sum(-(-l // page) for l in lengths) + 3
        table = torch.zeros(S, most, dtype=torch.int32, device=dev)
        order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
        at = 0
        for s, l in enumerate(lengths):
            c = -(-l // page)
            table[s, :c] = order[at:at + c]
            at += c
        st |= {"q": normal(M, H, D, std=2.0).bfloat16(), "k": normal(M, G, D).bfloat16(),
               "v": normal(M, G, D).bfloat16(), "page_table": table, "k_scale": None, "v_scale": None}
        for name in ("k", "v"):
            cache = torch.empty(pool, page, G, D, dtype=torch.bfloat16, device=dev)
            cache.normal_(generator=gen)
            if case["cache"] == "e4m3":
                # one scale a head, as a calibrated 8-bit cache has
                scale = uniform(0.01, 0.02, G)
                cache = (cache / scale[:, None].bfloat16()).to(torch.float8_e4m3fn)
                st[name + "_scale"] = scale
            st[name + "_cache"] = cache
        return st
    if case["op"] == "adjust":
        V = case["V"]
        most = max(lengths)
        # words repeat: a third of a text's tokens come from a few hundred
        common = torch.randint(0, V, (300,), generator=gen, device=dev, dtype=torch.int32)

        def text(*shape):
            return torch.where(uniform(0, 1, *shape) < 0.33, common[integers(0, 300, shape).long()],
                               integers(0, V, shape))
        b = case["biases"]
        st |= {"logits": normal(M, V, std=2.5).bfloat16(), "history": text(S, most), "inputs": text(M),
               "prompt_lengths": (st["lengths"] * uniform(0.2, 0.9, S)).int(),
               "repetition": uniform(1.0, 1.3, S), "presence": uniform(-0.2, 0.6, S),
               "frequency": uniform(0.0, 0.3, S), "bias": None, "allowed": None, "mask_rows": None}
        if b:
            st["bias"] = (torch.arange(0, S * b + 1, b, dtype=torch.int32, device=dev), integers(0, V, (S * b,)),
                          uniform(-5, 5, S * b))
        if case["masked"]:
            # a grammar lets through nearly nothing, or all but a few
            stream = torch.arange(S, device=dev).repeat_interleave(torch.tensor(rows, device=dev))
            under = stream % case["masked"] == 0
            A = sum(r for s, r in enumerate(rows) if s % case["masked"] == 0)
            words = (V + 31) // 32
            some = integers(0, 1 << 30, (A, words)) & integers(0, 1 << 30, (A, words))
            few = torch.where(uniform(0, 1, A, words) < 0.01, some, torch.zeros_like(some))
            st["allowed"] = torch.where((torch.arange(A, device=dev) % 3 > 0)[:, None], few, ~few)
            st["mask_rows"] = torch.where(under, torch.cumsum(under, 0) - 1, -1).to(torch.int32)
        return st
    tokens = integers(0, VOCAB, (M,))
    inputs = integers(0, VOCAB, (M,))
    # a draft is what the main model samples behind its parent about one time in two
    first = starts[:-1].long().repeat_interleave(torch.tensor(rows, device=dev))
    up = (first + parents.long().clamp(min=0))
    hit = (torch.rand(M, generator=gen, device=dev) < 0.5) & (parents >= 0)
    st |= {"tokens": tokens, "inputs": torch.where(hit, tokens[up], inputs)}
    return st


# ---- one pass ------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import spec_verify_amd as svq
        if op == "attend":
            c = state["case"]
            return svq.tree_attention(state["q"], state["k"], state["v"], state["k_cache"], state["v_cache"],
                                      state["page_table"], state["lengths"], state["starts"],
                                      parents=state["parents"] if c["tree"] else None, window=c["window"],
                                      sinks=c["sinks"], k_scale=state["k_scale"], v_scale=state["v_scale"])
        if op == "adjust":
            return svq.adjust_logits(state["logits"], state["history"], state["lengths"], state["inputs"],
                                     state["starts"], parents=state["parents"] if state["case"]["tree"] else None,
                                     prompt_lengths=state["prompt_lengths"], repetition=state["repetition"],
                                     presence=state["presence"], frequency=state["frequency"], bias=state["bias"],
                                     allowed=state["allowed"], mask_rows=state["mask_rows"])
        return svq.accept_tree(state["tokens"], state["inputs"], state["parents"], state["starts"])
    if op == "attend":
        return _plain_attend(state)
    if op == "adjust":
        return _plain_adjust(state)
    return _plain_accept(state["tokens"], state["inputs"], state["parents"], state["starts"])


def _grid(state):
    """Rows as a [streams, most nodes] grid: (row numbers, which of them exist, parents, ancestors and self)."""
    starts, parents, n = state["starts"].long(), state["parents"], state["case"]["nodes"]
    i = torch.arange(n, device=starts.device)
    there = i[None] < (starts[1:] - starts[:-1])[:, None]
    at = torch.where(there, starts[:-1, None] + i[None], 0)
    up = torch.where(there, parents[at].long(), -1)
    line = ((up[:, :, None] == i[None, None]) | (i[:, None] == i[None])[None]).float()
    for _ in range(max(1, (n - 1).bit_length())):
        line = torch.matmul(line, line).clamp(max=1.0)
    return at, there, up, line > 0


def _plain_attend(st):
    c = st["case"]
    H, G, D, page, n = (c[k] for k in ("heads", "kv_heads", "dim", "page", "nodes"))
    S, g = c["streams"], c["heads"] // c["kv_heads"]
    at, there, _, line = _grid(st)
    lengths = st["lengths"].long()
    pos = torch.arange(max(_sizes(c)[1]), device=lengths.device)
    pages = st["page_table"].long()[:, pos // page]

    def keys(name):
        cached = st[name + "_cache"][pages, pos % page].float()
        if st[name + "_scale"] is not None:
            cached = cached * st[name + "_scale"][:, None]
        return torch.cat([cached, st[name][at].float()], 1).transpose(1, 2).contiguous()

    # positions and visibility of [streams, node, token]
    depth = line.sum(-1) - 1
    here = lengths[:, None] + depth
    where = torch.cat([pos[None].expand(S, -1), here], 1)
    seen = torch.cat([(pos[None] < lengths[:, None])[:, None].expand(S, n, -1), line], 2)
    if c["window"] > 0:
        seen = seen & ((here[:, :, None] - where[:, None] < c["window"]) | (where < c["sinks"])[:, None])
    q = st["q"][at].float().reshape(S, n, G, g, D).permute(0, 2, 1, 3, 4).reshape(S, G, n * g, D)
    scores = torch.matmul(q, keys("k").transpose(2, 3).contiguous()) * D ** -0.5
    scores = scores.view(S, G, n, g, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.view(S, G, n * g, -1), keys("v")).view(S, G, n, g, D) / total
    return out.permute(0, 2, 1, 3, 4).reshape(S, n, H, D)[there].bfloat16()


def _plain_adjust(st):
    logits, history, lengths = st["logits"], st["history"].long(), st["lengths"].long()
    M, V = logits.shape
    S, L = history.shape
    at, there, _, line = _grid(st)
    stream = torch.arange(S, device=logits.device)[:, None].expand_as(at)[there]
    pos = torch.arange(L, device=logits.device)[None]
    before = (pos < lengths[:, None]).float()
    said = before * (pos >= st["prompt_lengths"].long()[:, None])

    def count(weight):
        return torch.zeros(S, V, device=logits.device).scatter_add_(1, history, weight)
    path = torch.zeros(M, V, device=logits.device).scatter_add_(
        1, st["inputs"].long()[at][stream], (line & there[:, None])[there].float())
    out = count(said)[stream] + path
    known = (count(before)[stream] + path) > 0
    x = logits.float()
    r = st["repetition"][stream][:, None]
    x = torch.where(known, torch.where(x > 0, x / r, x * r), x)
    x = x - st["frequency"][stream][:, None] * out - st["presence"][stream][:, None] * (out > 0)
    if st["bias"] is not None:
        first, tokens, values = st["bias"]
        owner = torch.searchsorted(first[1:].long(), torch.arange(tokens.shape[0], device=logits.device), right=True)
        x = x + torch.zeros(S, V, device=logits.device).index_put_((owner, tokens.long()), values,
                                                                   accumulate=True)[stream]
    if st["allowed"] is not None:
        v = torch.arange(V, device=logits.device)
        rows = st["mask_rows"].long()
        bits = (st["allowed"][rows.clamp(min=0)][:, v // 32] >> (v % 32).int()) & 1
        x = torch.where((rows >= 0)[:, None] & (bits == 0), -math.inf, x)
    return x.bfloat16()


def _plain_accept(tokens, inputs, parents, starts):
    M, S = tokens.shape[0], starts.shape[0] - 1
    r = torch.arange(M, device=tokens.device)
    first = starts[:-1].long()
    stream = torch.searchsorted(starts[1:].long(), r, right=True)
    up = torch.where(parents >= 0, first[stream] + parents, r)
    follows = (parents >= 0) & (tokens[up] == inputs)
    # of siblings that hold the same token the first one counts
    lead = torch.full((M,), M, device=tokens.device).scatter_reduce(
        0, up, torch.where(follows, r, torch.full_like(r, M)), "amin")
    good = (r == first[stream]) | (follows & (lead[up] == r))
    depth = (parents >= 0).long()
    for _ in range(16):
        good, depth, up = good & good[up], depth + depth[up], up[up]
    n = torch.zeros(S, dtype=torch.long, device=tokens.device).scatter_add_(0, stream, good.long())
    to = torch.where(good, first[stream] + depth, M)
    spare = torch.full((M + 1,), -1, dtype=torch.int32, device=tokens.device)
    committed = spare.scatter(0, to, tokens)[:M]
    path = spare.scatter(0, to, (r - first[stream]).int())[:M]
    return (n - 1).int(), committed[first + n - 1], committed, path


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    rows, lengths = _sizes(case)
    M, S = sum(rows), len(rows)
    if case["op"] == "attend":
        H, G, D = (case[k] for k in ("heads", "kv_heads", "dim"))
        w = case["window"]
        # what a stream's first row sees of its cache; a tree's rows see themselves at least
        seen = [min(l, max(0, w - 1) + min(case["sinks"], max(0, l - w + 1))) if w else l for l in lengths]
        size = 1 if case["cache"] == "e4m3" else 2
        return {"bytes": 2 * sum(seen) * G * D * size + 4 * M * (H + G) * D + 4 * (M + 2 * S + 1)
                + 4 * sum(-(-l // case["page"]) for l in seen),
                "flops": 4 * H * D * sum(r * (l + 1) for r, l in zip(rows, seen))}
    if case["op"] == "adjust":
        V, m = case["V"], case["masked"]
        under = sum(r for s, r in enumerate(rows) if m and s % m == 0)
        return {"bytes": 4 * M * V + 4 * sum(lengths) + 8 * S * case["biases"] + under * (V // 8) + 12 * M + 20 * S,
                "flops": M * V}
    return {"bytes": 20 * M + 12 * S + 4, "flops": M}


# ---- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    starts, parents, lengths = (st[k].tolist() for k in ("starts", "parents", "lengths"))
    if not case.get("tree", True):
        parents = [i - 1 for a, b in zip(starts, starts[1:]) for i in range(b - a)]
    if case["op"] == "accept":
        tokens, inputs = st["tokens"].tolist(), st["inputs"].tolist()
        accepted, following, committed, path = [], [], [-1] * len(tokens), [-1] * len(tokens)
        for a, b in zip(starts, starts[1:]):
            node, n = 0, 0
            while node is not None:
                committed[a + n], path[a + n] = tokens[a + node], node
                node = next((j for j in range(node + 1, b - a)
                             if parents[a + j] == node and inputs[a + j] == tokens[a + node]), None)
                n += 1
            accepted.append(n - 1)
            following.append(committed[a + n - 1])
        return tuple(torch.tensor(x, dtype=torch.int32) for x in (accepted, following, committed, path))
    paths = []  # of every row: the rows of its sequence from the first one to itself
    for a, b in zip(starts, starts[1:]):
        for i in range(b - a):
            paths.append((paths[a + parents[a + i]] if parents[a + i] >= 0 else []) + [i])
    if case["op"] == "attend":
        return _exact_attend(case, st, starts, lengths, paths)
    return _exact_adjust(st, starts, lengths, paths)


def _exact_attend(case, st, starts, lengths, paths):
    H, G, D, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    g, w, sinks = H // G, case["window"], case["sinks"]
    out = torch.zeros(len(paths), H, D, dtype=torch.float64, device="cuda")
    for s, L in enumerate(lengths):
        a, b = starts[s], starts[s + 1]
        used = st["page_table"][s, :-(-L // page)].long()
        n = b - a
        seen = torch.zeros(n, L + n, dtype=torch.bool)
        for i in range(n):
            p = L + len(paths[a + i]) - 1
            seen[i, (max(0, p - w + 1) if w else 0):L] = True
            if w:
                seen[i, :min(sinks, L)] = True
            for d, j in enumerate(paths[a + i]):
                seen[i, L + j] = not w or p - (L + d) < w or L + d < sinks
        seen = seen.cuda()
        for h in range(G):
            kv = []
            for name in ("k", "v"):
                x = st[name + "_cache"][used, :, h].reshape(-1, D)[:L].double()
                if st[name + "_scale"] is not None:
                    x = x * st[name + "_scale"][h].double()
                kv.append(torch.cat([x, st[name][a:b, h].double()]))
            q = st["q"][a:b, h * g:(h + 1) * g].double().reshape(n * g, D)
            e = (torch.mm(q, kv[0].t().contiguous()) / math.sqrt(D)).view(n, g, L + n)
            e = torch.where(seen[:, None], e, torch.full_like(e, -math.inf))
            p = torch.softmax(e, -1).view(n * g, L + n)
            out[a:b, h * g:(h + 1) * g] = torch.mm(p, kv[1]).view(n, g, D)
    return out


def _exact_adjust(st, starts, lengths, paths):
    logits, dev = st["logits"], st["logits"].device
    M, V = logits.shape
    out = torch.empty(M, V, dtype=torch.float64, device=dev)
    inputs = st["inputs"].tolist()
    for s, L in enumerate(lengths):
        prompt = int(st["prompt_lengths"][s])
        tokens = st["history"][s, :L].long()
        known = torch.bincount(tokens, minlength=V)
        said = torch.bincount(tokens[prompt:], minlength=V)
        bias = torch.zeros(V, dtype=torch.float64, device=dev)
        if st["bias"] is not None:
            lo, hi = int(st["bias"][0][s]), int(st["bias"][0][s + 1])
            bias = torch.bincount(st["bias"][1][lo:hi].long(), weights=st["bias"][2][lo:hi].double(), minlength=V)
        rep, pres, freq = (st[k][s].double() for k in ("repetition", "presence", "frequency"))
        for m in range(starts[s], starts[s + 1]):
            own_path = torch.tensor([inputs[starts[s] + i] for i in paths[m]], device=dev)
            more = torch.bincount(own_path, minlength=V)
            x = logits[m].double()
            x = torch.where(known + more > 0, torch.where(x > 0, x / rep, x * rep), x)
            x = x - freq * (said + more) - pres * (said + more > 0).double() + bias
            if st["allowed"] is not None and int(st["mask_rows"][m]) >= 0:
                words = st["allowed"][int(st["mask_rows"][m])].cpu().numpy().view(np.uint8)
                free = torch.from_numpy(np.unpackbits(words, bitorder="little")[:V].astype(bool)).to(dev)
                x = torch.where(free, x, torch.full_like(x, -math.inf))
            out[m] = x
    return out
