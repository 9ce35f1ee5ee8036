"""Plain 64-bit definitions of sampled decoding and of eviction from the 8-bit
paged cache, on the CPU: probabilities row by row, verification as a loop over
the drafts, weights position by position, eviction as list operations."""

import math

import numpy as np

from tests.kv8_plain import PAGE, round_e4m3


# ------------------------------------------------------------------ probabilities

def probs(x, t, min_p=0.0):
    """One row of logits (float64 values of the type's numbers), temperature t.
    Returns (p, d): probabilities and (x - m) / t of each token (0 without weight)."""
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    p, d = np.zeros(len(x)), np.zeros(len(x))
    if m == -np.inf:
        return p, d
    if t == 0:
        p[int(np.argmax(x))] = 1.0
        return p, d
    keep = x > -np.inf
    if min_p > 0:
        border = float(m) + float(t) * math.log(min(float(min_p), 1.0))
        up = np.float32(border)
        if float(up) < border:
            up = np.nextafter(up, np.float32(np.inf))
        keep &= x >= float(up)
    with np.errstate(invalid="ignore", over="ignore"):
        d[keep] = np.where(x[keep] == m, 0.0, (x[keep] - m) / float(t))
    with np.errstate(under="ignore"):
        p[keep] = np.exp(d[keep])
    d = np.where(np.isfinite(d), d, 0.0)
    return p / p.sum(), d


# ------------------------------------------------------------------ verification

def clean(p):
    p = np.asarray(p, dtype=np.float64)
    return np.where((p > 0) & (p < 2.0 ** 100), p, 0.0)


def pick(w, u):
    """The first token whose running sum passes u * sum; the last with weight
    where none does, -1 without weight."""
    total = math.fsum(w)
    at = np.nonzero(w > 0)[0]
    if len(at) == 0:
        return -1
    run = np.cumsum(w.astype(np.longdouble))
    with np.errstate(invalid="ignore"):
        over = [v for v in np.nonzero(run > np.longdouble(u) * np.longdouble(total))[0][:1] if w[v] > 0] \
            if not math.isnan(u) else []
    if u < 0:
        return int(at[0])
    return int(over[0]) if over else int(at[-1])


def verify(p, ids, u, row_start, q=None, kv_len=None):
    """p, q [rows][vocab] float64 values of fp32 numbers.  Returns (tokens as
    {row: token}, n_tokens, new_len)."""
    tokens, n_tokens, new_len, vocab = {}, [], [], p.shape[1]
    for s in range(len(row_start) - 1):
        r0, n = row_start[s], row_start[s + 1] - row_start[s]
        kv = kv_len[s] if kv_len is not None else 0
        if n == 0:
            n_tokens.append(0)
            new_len.append(kv)
            continue
        a, refused = 0, None
        for i in range(1, n):
            d = ids[r0 + i]
            if not 0 <= d < vocab:
                break
            qd = 1.0 if q is None else float(clean(q[r0 + i, d]))
            if float(u[r0 + i]) * qd < float(clean(p[r0 + i - 1, d])):
                a += 1
            else:
                refused = d
                break
        base = clean(p[r0 + a])
        w = base
        if refused is not None:
            if q is None:
                w = base.copy()
                w[refused] = 0.0
            else:
                w = np.maximum(base - clean(q[r0 + a + 1]), 0.0)
            if not w.any():
                w = base
        v = pick(w, float(u[r0]))
        for i in range(n):
            tokens[r0 + i] = int(ids[r0 + i + 1]) if i < a else (v if i == a else -1)
        n_tokens.append(a + (v >= 0))
        new_len.append(kv - (n - 1 - a))
    return tokens, n_tokens, new_len


# ------------------------------------------------------------------ accumulated weights

def weigh(q, lse, kc, k_scale, table, kv_len, row_start, weights, count=None, observe=0, fresh=False, causal=True,
          window=0, scale=1.0):
    """q [rows][n_q][dim], kc the pool's code values [pages][n_kv][64][dim],
    k_scale, lse, weights as float64 numpy.  Returns (weights, bound): bound is
    what each position's fp32 sum may be off by."""
    out, bound = weights.copy(), np.zeros_like(weights)
    n_q, dim = q.shape[1:]
    group = n_q // kc.shape[1]
    for s, kv in enumerate(kv_len):
        r0, n = row_start[s], row_start[s + 1] - row_start[s]
        i1 = n if count is None else min(max(count[s], 0), n)
        i0 = max(i1 - observe, 0) if observe else 0
        for j in range(kv):
            pg, off = table[s][j // PAGE], j % PAGE
            got = err = 0.0
            terms = 0
            for i in range(i0, i1):
                p = kv - n + i
                if causal and (j > p or (window and j <= p - window)):
                    continue
                if not causal and window and j < kv - n - window:
                    continue
                k = np.repeat(kc[pg, :, off] * k_scale[pg][:, None], group, 0)
                x = (q[r0 + i] * k).sum(1) * scale
                with np.errstate(invalid="ignore"):
                    e = x - lse[r0 + i]                  # NaN (a NaN code, inf - inf) adds nothing
                    t = np.where(np.isnan(e) | (lse[r0 + i] == -np.inf), 0.0, np.exp(e))
                # dim products in fp32, the factor and its product; elements of q held as
                # f16 beside the row's largest; lse in base 2; the difference; ex2
                with np.errstate(invalid="ignore"):
                    d = (dim + 10) * 2.0 ** -24 * np.abs(q[r0 + i] * k).sum(1) * scale
                    d += 2.0 ** -25 * np.abs(q[r0 + i]).max(1) * np.abs(k).sum(1) * scale
                l = np.where(np.isfinite(lse[r0 + i]), np.abs(lse[r0 + i]), 0.0)
                d = np.where(np.isfinite(x), d, 0.0)
                x = np.where(np.isfinite(x), x, 0.0)
                d += 2.0 ** -23 * l + 2.0 ** -24 * (np.abs(x) + l) + 2.0 ** -22
                got += t.sum()
                err += (t * (d + d * d)).sum()
                terms += n_q
            old = 0.0 if fresh and j >= kv - n else out[pg, off]
            out[pg, off] = old + got
            bound[pg, off] = err + (terms + 8) * 2.0 ** -24 * got + 2.0 ** -24 * abs(old + got) + terms * 2.0 ** -126
    return out, bound


# ------------------------------------------------------------------ eviction

def evict(layers, table, kv_len, weights, budget, keep_first, keep_last):
    """layers: [(k values, v values, k scales, v scales), ..] numpy, changed in
    place (values are the codes' without the scale); weights numpy, changed in
    place.  Returns (new_len, source lists, gone)."""
    new_len, source, gone = [], [], []
    for s, n in enumerate(kv_len):
        b, pages = budget[s], table[s]
        if not (b > 0 and n > b):
            new_len.append(n)
            source.append(list(range(n)))
            gone.append(0)
            continue
        w = [weights[pages[j // PAGE], j % PAGE] for j in range(n)]
        last = min(keep_last, b)
        first = min(keep_first, b - last)
        rank = lambda j: (-math.inf if math.isnan(w[j]) else float(w[j]))       # noqa: E731
        lightest = lambda j: (0 if not math.isnan(w[j]) else 1, -rank(j), j)    # noqa: E731
        middle = sorted(range(first, n - last), key=lightest)[:b - first - last]
        keep = sorted(list(range(first)) + middle + list(range(n - last, n)))
        for c in layers:
            for values, scale in ((c[0], c[2]), (c[1], c[3])):
                old, olds = values.copy(), scale.copy()
                for d in range(-(-b // PAGE)):
                    rows = keep[d * PAGE:(d + 1) * PAGE]
                    if rows == list(range(d * PAGE, d * PAGE + len(rows))):
                        continue
                    came = np.stack([olds[pages[j // PAGE]] for j in rows])      # [rows][heads]
                    unit = came.max(0)
                    for i, j in enumerate(rows):
                        x = old[pages[j // PAGE], :, j % PAGE]
                        same = (came[i] == unit)[:, None]
                        with np.errstate(invalid="ignore"):
                            moved = round_e4m3(x * (came[i] / unit)[:, None])
                        values[pages[d], :, i] = np.where(same, x, moved)
                    scale[pages[d]] = unit
        for i, j in enumerate(keep):
            weights[pages[i // PAGE], i % PAGE] = w[j]
        new_len.append(b)
        source.append(keep)
        gone.append(n - b)
    return new_len, source, gone
