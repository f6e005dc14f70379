"""The operators of a tree of drafts from their definitions, in 64 bits on the CPU."""
import numpy as np


def paths(parents, n):
    """The path of every row of one sequence: its ancestors from the top, then itself. parents None: a chain."""
    out = []
    for i in range(n):
        p = i - 1 if parents is None else int(parents[i])
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def sequences(starts, M):
    """(first row, number of rows) of each sequence."""
    b = [min(max(int(x), 0), M) for x in starts]
    return [(a, max(0, e - a)) for a, e in zip(b, b[1:])]


def attend(q, k, v, k_cache, v_cache, table, lengths, starts, parents, scale, window=0, sinks=0):
    """(out, bound on a kernel's error, rows of sequences): all arrays float64; caches [pages, page, KVH, D]
    already scaled. The kernel holds scores and sums in fp32 and its weights and result in bf16."""
    M, H, D = q.shape
    G = k.shape[1]
    g = H // G
    pages, page = k_cache.shape[:2]
    out, bound = np.zeros((M, H, D)), np.zeros((M, H, D))
    inside = np.zeros(M, dtype=bool)
    for s, (a, n) in enumerate(sequences(starts, M)):
        par = None if parents is None else parents[a:a + n]
        L = min(max(int(lengths[s]), 0), table.shape[1] * page)
        pos = np.arange(L)
        at = table[s][pos // page] if L else np.zeros(0, dtype=np.int64)
        good = (at >= 0) & (at < pages)
        kc = np.concatenate([k_cache[np.where(good, at, 0), pos % page] if L else np.zeros((0, G, D)), k[a:a + n]])
        vc = np.concatenate([v_cache[np.where(good, at, 0), pos % page] if L else np.zeros((0, G, D)), v[a:a + n]])
        for i, path in enumerate(paths(par, n)):
            p = L + len(path) - 1
            where = np.concatenate([pos[good], [L + d for d in range(len(path))]]).astype(np.int64)
            idx = np.concatenate([np.nonzero(good)[0], [L + j for j in path]]).astype(np.int64)
            if window > 0:
                keep = (p - where < window) | (where < sinks)
                idx = idx[keep]
            inside[a + i] = True
            for h in range(H):
                kk, vv, qq = kc[idx, h // g], vc[idx, h // g], q[a + i, h]
                with np.errstate(invalid="ignore", over="ignore"):
                    e = kk @ qq * scale
                    seen = ~(e == -np.inf)
                    if not seen.any():
                        continue
                    e, kk, vv = e[seen], kk[seen], vv[seen]
                    w = np.exp(e - np.max(e))
                    w /= w.sum()
                    o = w @ vv
                    out[a + i, h] = o
                    # a score is off by its products' sums, the scale and the subtraction of the maximum; a
                    # weight by that, the exponential and bf16; sums of N terms by N roundings
                    N = len(e)
                    de = (2 * D * 2.0 ** -24 * abs(scale) * (np.abs(kk) @ np.abs(qq))
                          + 2.0 ** -22 * (np.abs(e) + np.abs(e - np.max(e))))
                    dw = w * (de + 2.0 ** -22)
                    slack = 2 * (N + 8) * 2.0 ** -24
                    mass = w @ np.abs(vv)
                    err = (dw + w * (2.0 ** -8 + slack)) @ np.abs(vv) + (dw.sum() + slack) * mass
                    bound[a + i, h] = err * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o) + 1e-38
    return out, bound, inside


def adjust(logits, history, lengths, inputs, starts, parents=None, prompt_lengths=None, repetition=None, presence=None,
           frequency=None, bias=None, allowed=None, mask_rows=None):
    """(out float64, bound on a kernel's error, rows of sequences, logits that nothing applies to)."""
    M, V = logits.shape
    out, bound = logits.astype(np.float64).copy(), np.zeros((M, V))
    inside, plain = np.zeros(M, dtype=bool), np.ones((M, V), dtype=bool)

    def count(tokens):
        t = np.asarray(tokens, dtype=np.int64)
        return np.bincount(t[(t >= 0) & (t < V)], minlength=V)
    for s, (a, n) in enumerate(sequences(starts, M)):
        L = min(max(int(lengths[s]), 0), history.shape[1])
        prompt = 0 if prompt_lengths is None else min(max(int(prompt_lengths[s]), 0), L)
        seen, said = count(history[s, :L]), count(history[s, prompt:L])
        r = 1.0 if repetition is None else float(repetition[s])
        pres = 0.0 if presence is None else float(presence[s])
        freq = 0.0 if frequency is None else float(frequency[s])
        add, biased = np.zeros(V), np.zeros(V, dtype=bool)
        mass = np.zeros(V)
        if bias is not None:
            b0, b1 = (min(max(int(x), 0), len(bias[1])) for x in bias[0][s:s + 2])
            for t, x in zip(bias[1][b0:max(b0, b1)], bias[2][b0:max(b0, b1)]):
                if 0 <= t < V:
                    add[t] += float(x)
                    mass[t] += 2 * abs(float(x))
                    biased[t] = True
        for i, path in enumerate(paths(None if parents is None else parents[a:a + n], n)):
            m = a + i
            inside[m] = True
            mine = count(inputs[a + np.array(path)])
            known, c = seen + mine > 0, said + mine
            with np.errstate(invalid="ignore", over="ignore"):
                x = logits[m].astype(np.float64)
                y = np.where(known, np.where(x > 0, x / r, x * r), x)
                z = y - freq * c - np.where(c > 0, pres, 0.0) + add
                size = np.abs(y) + freq * c * np.sign(freq) + abs(pres) + mass
                # one rounding of 1 / r, of the product, and two or three of sums in fp32; then bf16
                bound[m] = np.where(np.isfinite(z), 8 * 2.0 ** -24 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(z), 0)
            plain[m] = ~(known | biased)
            if mask_rows is not None and 0 <= mask_rows[m] < len(allowed):
                bits = np.unpackbits(np.ascontiguousarray(allowed[mask_rows[m]]).view(np.uint8),
                                     bitorder="little")[:V].astype(bool)
                z = np.where(bits, z, -np.inf)
                plain[m] &= bits
                bound[m][~bits] = 0
            out[m] = z
    return out, bound, inside, plain


def accept(tokens, inputs, parents, starts):
    M = len(tokens)
    accepted, following = [], []
    committed, path = np.full(M, -1), np.full(M, -1)
    for a, n in sequences(starts, M):
        at, k, token = 0, 0, -1
        while n:
            token = tokens[a + at]
            committed[a + k], path[a + k] = token, at
            k += 1
            to = [j for j in range(at + 1, n) if parents[a + j] == at and inputs[a + j] == token] if token >= 0 else []
            if not to:
                break
            at = to[0]
        accepted.append(max(k - 1, 0))
        following.append(token)
    return np.array(accepted), np.array(following), committed, path
