"""Measured cases of the per-request operators of a verify chunk.

A decode or verify step runs every request's tokens through shared quantized
projections. Three things differ from request to request in the same batch: its
low-rank adapter (``adapter_add``, behind a shared projection), its sampling
parameters (``sample``, behind the vocabulary head) and its drafted tokens
(``accept_drafts``, behind the sampler).

``own`` selects the framework's kernels; otherwise the operators run in their
plain form, elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

HIDDEN = 5120
INTERMEDIATE = 17408
VOCAB = 248320


# ---- cases -------------------------------------------------------------------

def _adapter(name, streams, chunk, K, N, R, slots, bare=0):
    """`streams` requests of `chunk` tokens each, request i on adapter i % slots of
    a shuffled pool; the last `bare` requests carry no adapter."""
    return {"name": name, "op": "adapter", "streams": streams, "chunk": chunk, "K": K, "N": N, "R": R,
            "slots": slots, "bare": bare}


def _sample(name, M, V, mode):
    return {"name": name, "op": "sample", "M": M, "V": V, "mode": mode}


def _accept(name, streams, drafts, ragged):
    return {"name": name, "op": "accept", "streams": streams, "drafts": drafts, "ragged": ragged}


def listed():
    return [
        # one request decoding one token, adapter beside an attention projection: the smallest call
        _adapter("adapter-decode-1", 1, 1, HIDDEN, HIDDEN, 16, 4),
        # one request's verify chunk (four drafts) beside the gate or up projection
        _adapter("adapter-verify-5", 1, 5, HIDDEN, INTERMEDIATE, 16, 8),
        # batched verify, every request with its own adapter, some without one
        _adapter("adapter-batch-128-up", 32, 4, HIDDEN, INTERMEDIATE, 32, 32, bare=3),
        # batched verify beside the down projection: long K, few adapters shared by many requests
        _adapter("adapter-batch-128-down", 32, 4, INTERMEDIATE, HIDDEN, 64, 6),
        # odd everything: ragged row tiles, a rank that fills no tile, a narrow projection
        _adapter("adapter-odd-37", 37, 1, 640, 1040, 24, 5, bare=2),
        # prompts of three requests in one batch
        _adapter("adapter-prompt-2001", 3, 667, HIDDEN, 6144, 16, 3),
        # one token of one request, a usual chat setting
        _sample("sample-decode-1", 1, VOCAB, "chat"),
        # one verify chunk of five tokens
        _sample("sample-verify-5", 5, VOCAB, "chat"),
        # batched verify, each request with its own setting (greedy, plain, chat, top-k, top-p, min-p)
        _sample("sample-batch-128", 128, VOCAB, "mixed"),
        # a large serving batch, nothing filtered: the whole distribution counts
        _sample("sample-batch-1024-plain", 1024, VOCAB, "plain"),
        # one stream's chunk, and a large batch with zero to eight drafts a request
        _accept("accept-1x4", 1, 4, False),
        _accept("accept-2048-ragged", 2048, 8, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adapter", "adapter", "sample", "sample", "accept"])
    if op == "adapter":
        chunk = _log_int(rng, 1, 600)
        streams = _log_int(rng, 1, max(1, min(128, 2000 // chunk)))
        slots = _log_int(rng, 1, 32)
        K = 128 * _log_int(rng, 1, INTERMEDIATE // 128)
        N = 16 * _log_int(rng, 1, INTERMEDIATE // 16)
        R = 8 * _log_int(rng, 1, 16)
        bare = rng.randint(0, max(0, streams // 4))
        c = _adapter("", streams, chunk, K, N, R, slots, bare)
    elif op == "sample":
        V = _log_int(rng, 2, VOCAB)
        M = _log_int(rng, 1, 1024)
        c = _sample("", M, V, rng.choice(["mixed", "mixed", "chat", "plain", "greedy"]))
    else:
        c = _accept("", _log_int(rng, 1, 2048), rng.randint(0, 8), rng.random() < 0.5)
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    def integers(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=gen, device=dev, dtype=torch.int32)

    if case["op"] == "adapter":
        streams, chunk, K, N, R, slots = (case[k] for k in ("streams", "chunk", "K", "N", "R", "slots"))
        M = streams * chunk
        order = torch.randperm(slots, generator=gen, device=dev)
        slot = order[torch.arange(streams, device=dev) % slots].to(torch.int32)
        if case["bare"]:
            slot[streams - case["bare"]:] = -1
        return {
            "case": case,
            # hidden states after a norm, and a projection's output for them
            "x": normal(M, K).bfloat16(),
            "base": normal(M, N, std=3.0).bfloat16(),
            "a": normal(slots, R, K, std=K ** -0.5).bfloat16(),
            "b": normal(slots, N, R, std=R ** -0.5).bfloat16(),
            "scales": torch.rand(slots, generator=gen, device=dev) + 0.5,
            "rows": slot.repeat_interleave(chunk).contiguous(),
        }
    if case["op"] == "sample":
        M, V = case["M"], case["V"]
        # a head's logits: a wide floor, and some tens of likely tokens that fall off
        logits = normal(M, V, std=2.2)
        peaks = min(60, V)
        heights = 13.0 - 0.18 * torch.arange(peaks, device=dev) + normal(M, peaks)
        first = torch.randint(0, V, (M, 1), generator=gen, device=dev)
        likely = torch.randperm(V, generator=gen, device=dev)[:peaks]
        logits.scatter_(1, (first + likely) % V, heights)
        logits = logits.bfloat16()
        T = torch.rand(M, generator=gen, device=dev) * 0.9 + 0.4
        k = integers(2, 200, (M,))
        p = torch.rand(M, generator=gen, device=dev) * 0.5 + 0.49
        mp = torch.rand(M, generator=gen, device=dev) * 0.2
        kind = {"mixed": integers(0, 6, (M,)), "chat": torch.full((M,), 5, device=dev),
                "plain": torch.ones(M, device=dev), "greedy": torch.zeros(M, device=dev)}[case["mode"]]
        # 0 greedy, 1 temperature alone, 2 top-k, 3 top-p, 4 min-p, 5 top-k and top-p together
        return {
            "case": case, "logits": logits,
            "u": torch.rand(M, generator=gen, device=dev),
            "temperature": torch.where(kind == 0, torch.zeros_like(T), T),
            "top_k": torch.where((kind == 2) | (kind == 5), k, torch.zeros_like(k)),
            "top_p": torch.where((kind == 3) | (kind == 5), p, torch.ones_like(p)),
            "min_p": torch.where(kind == 4, mp, torch.zeros_like(mp)),
        }
    S, d = case["streams"], case["drafts"]
    drafts = torch.full((S,), d, device=dev)
    if case["ragged"]:
        drafts = (torch.arange(S, device=dev) % (d + 1))[torch.randperm(S, generator=gen, device=dev)]
    starts = torch.zeros(S + 1, dtype=torch.int32, device=dev)
    starts[1:] = torch.cumsum(drafts + 1, 0)
    M = int(starts[-1])
    tokens = integers(0, VOCAB, (M,))
    inputs = integers(0, VOCAB, (M,))
    # a draft is what the main model samples about two times in three
    hit = torch.rand(M, generator=gen, device=dev) < 0.67
    if M > 1:
        inputs[1:] = torch.where(hit[1:], tokens[:-1], inputs[1:])
    return {"case": case, "tokens": tokens, "inputs": inputs, "starts": starts}


# ---- one pass ------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import spec_verify_amd as svq
        if op == "adapter":
            return svq.adapter_add(state["base"], state["x"], state["a"], state["b"], state["rows"],
                                   state["scales"])
        if op == "sample":
            return svq.sample(state["logits"], state["u"], temperature=state["temperature"],
                              top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
        return svq.accept_drafts(state["tokens"], state["inputs"], state["starts"])
    if op == "adapter":
        return _plain_adapter(state["base"], state["x"], state["a"], state["b"], state["rows"],
                              state["scales"])
    if op == "sample":
        return _plain_sample(state["logits"], state["u"], state["temperature"], state["top_k"],
                             state["top_p"], state["min_p"])
    return _plain_accept(state["tokens"], state["inputs"], state["starts"])


def _plain_adapter(base, x, a, b, rows, scales):
    xf, out = x.float(), base.float()
    for s in range(a.shape[0]):
        low = xf @ a[s].float().t().contiguous()
        delta = (low * scales[s]) @ b[s].float().t().contiguous()
        out = torch.where((rows == s)[:, None], out + delta, out)
    return out.bfloat16()


def _plain_sample(logits, u, temperature, top_k, top_p, min_p):
    """In 64 bits: a draw next to a border has to fall on the right side of it."""
    V = logits.shape[1]
    vals, order = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    greedy = (temperature <= 0)[:, None]
    scaled = (vals - vals[:, :1]) / torch.where(greedy, 1.0, temperature.double()[:, None])
    place = torch.arange(V, device=logits.device)[None]
    k = torch.where(greedy, 1, top_k.long()[:, None])
    w = torch.exp(scaled) * ((k <= 0) | (place < k))
    cum = torch.cumsum(w, 1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
    p = top_p.double()[:, None]
    w = w * ((p >= 1) | (place == 0) | (before < p * cum[:, -1:])) * (w >= min_p.double()[:, None])
    cum = torch.cumsum(w, 1)
    at = (cum <= u.double()[:, None] * cum[:, -1:]).sum(1, keepdim=True)
    at = torch.minimum(at, (w > 0).sum(1, keepdim=True) - 1)
    logprob = scaled.gather(1, at) - torch.log(cum[:, -1:])
    return order.gather(1, at)[:, 0].int(), logprob[:, 0].float()


def _plain_accept(tokens, inputs, starts):
    M, S = tokens.shape[0], starts.shape[0] - 1
    r = torch.arange(M, device=tokens.device)
    first, last = starts[:-1].long(), starts[1:].long() - 1
    stream = torch.searchsorted(starts[1:].long(), r, right=True)
    following = torch.cat([inputs[1:], inputs[:1]])
    stop = (r == last[stream]) | (tokens != following)
    at = torch.full((S,), M, device=tokens.device).scatter_reduce(
        0, stream, torch.where(stop, r, torch.full_like(r, M)), "amin")
    committed = torch.where(r <= at[stream], tokens, torch.full_like(tokens, -1))
    return (at - first).int(), tokens[at], committed


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    if case["op"] == "adapter":
        streams, chunk, K, N, R, slots = (case[k] for k in ("streams", "chunk", "K", "N", "R", "slots"))
        with_adapter = streams - case["bare"]
        M, m, used = streams * chunk, with_adapter * chunk, min(slots, with_adapter)
        return {"bytes": 2 * m * K + 2 * used * R * (K + N) + 4 * M * N + 4 * M + 4 * used,
                "flops": 2 * m * R * (K + N)}
    if case["op"] == "sample":
        M, V = case["M"], case["V"]
        return {"bytes": 2 * M * V + (5 * 4 + 8) * M, "flops": 2 * M * V}
    S, d = case["streams"], case["drafts"]
    M = S + (sum(i % (d + 1) for i in range(S)) if case["ragged"] else S * d)
    return {"bytes": 12 * M + 12 * S + 4, "flops": M}


# ---- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adapter":
        base, x, a, b = (st[k].double() for k in ("base", "x", "a", "b"))
        rows = st["rows"].long().tolist()
        out = base.clone()
        groups = {}
        for m, s in enumerate(rows):
            groups.setdefault(s, []).append(m)
        for s, members in groups.items():
            if s >= 0:
                idx = torch.tensor(members, device=base.device)
                low = torch.mm(a[s], x[idx].t().contiguous())
                out[idx] += float(st["scales"][s]) * torch.mm(b[s], low).t()
        return out
    if case["op"] == "sample":
        bits = st["logits"].view(torch.int16).cpu().numpy()
        values = st["logits"].float().cpu().numpy()
        par = {k: st[k].cpu().numpy() for k in ("u", "temperature", "top_k", "top_p", "min_p")}
        tokens, logprobs = [], []
        for m in range(case["M"]):
            t, lp = _exact_row(bits[m], values[m], *(par[k][m] for k in ("u", "temperature", "top_k", "top_p",
                                                                      "min_p")))
            tokens.append(t)
            logprobs.append(lp)
        return torch.tensor(tokens, dtype=torch.int32), torch.tensor(logprobs, dtype=torch.float64)
    tokens, inputs, starts = (st[k].tolist() for k in ("tokens", "inputs", "starts"))
    accepted, following, committed = [], [], [-1] * len(tokens)
    for first, end in zip(starts[:-1], starts[1:]):
        n = 0
        while first + n + 1 < end and tokens[first + n] == inputs[first + n + 1]:
            n += 1
        accepted.append(n)
        following.append(tokens[first + n])
        committed[first:first + n + 1] = tokens[first:first + n + 1]
    return tuple(torch.tensor(v, dtype=torch.int32) for v in (accepted, following, committed))


def _exact_row(bits, values, u, T, k, p, min_p):
    # 16-bit keys that ascend as the values descend (-0 counts as 0): a stable sort keeps the lowest index first
    bits = np.where(bits == -32768, 0, bits).astype(np.int64)
    key = np.where(bits < 0, (bits & 0x7FFF), -bits).astype(np.int16)
    order = np.argsort(key, kind="stable")
    if T <= 0:
        return int(order[0]), 0.0
    if 0 < k < len(order):
        order = order[:k]
    l = values[order].astype(np.float64)
    e = (l - l[0]) / np.float64(T)
    w = np.exp(e)
    if p < 1:
        run_sum = np.cumsum(w.astype(np.longdouble))
        w = w[:1 + int(np.searchsorted(run_sum, np.longdouble(p) * run_sum[-1], side="left"))]
    if min_p > 0:
        w = w[w >= np.float64(min_p)]
    run_sum = np.cumsum(w.astype(np.longdouble))
    at = int(np.searchsorted(run_sum, np.longdouble(u) * run_sum[-1], side="right"))
    at = min(at, len(w) - 1)
    return int(order[at]), float(e[at] - np.log(run_sum[-1]))
