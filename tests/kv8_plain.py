"""Plain 64-bit definitions of the 8-bit paged cache's operators, on the CPU:
page plans as a loop over the sequences, rotary positions as complex
rotations, the append as a loop over pages, attention row by row."""

import math

import numpy as np
import torch

PAGE = 64


# ------------------------------------------------------------------ pages

def plan(kv_len, q_len, free, n_free, table, rows):
    """Returns (table, row_start, positions, slots, kv_after, n_free)."""
    table = [list(t) for t in table]
    width = len(table[0])
    pages = given = used = want_pages = want_rows = 0
    start, pos, slot, after = [0], [], [], []
    for s, (kv, q) in enumerate(zip(kv_len, q_len)):
        fine = kv >= 0 and q >= 0 and -(-(kv + q) // PAGE) <= width
        n = 0
        if fine:
            need = -(-(kv + q) // PAGE) - -(-kv // PAGE)
            want_pages += need
            want_rows += q
            if want_pages <= n_free and want_rows <= rows:
                for j in range(need):
                    table[s][-(-kv // PAGE) + j] = free[n_free - 1 - used]
                    used += 1
                n = q
        for p in range(kv, kv + n):
            pos.append(p)
            slot.append(table[s][p // PAGE] * PAGE + p % PAGE)
        start.append(start[-1] + n)
        after.append(kv + n)
    pad = rows - len(pos)
    return table, start, pos + [-1] * pad, slot + [-1] * pad, after, n_free - used


def trim(kv_len, new_len, free, n_free, table):
    free, table, out = list(free), [list(t) for t in table], []
    for s, (kv, to) in enumerate(zip(kv_len, new_len)):
        to = max(to, 0)
        if kv > to and kv <= len(table[s]) * PAGE:
            for j in range(-(-kv // PAGE) - 1, -(-to // PAGE) - 1, -1):
                free[n_free] = table[s][j]
                table[s][j] = -1
                n_free += 1
            out.append(to)
        else:
            out.append(kv)
    return out, free, n_free, table


# ------------------------------------------------------------------ rotary positions

def frequencies(rotary, theta, scaling="none", factor=1.0, original_len=0, alpha=1.0, beta=32.0):
    f = []
    for i in range(rotary // 2):
        w = theta ** (-2.0 * i / rotary)
        if scaling == "linear":
            w /= factor
        elif scaling == "parts":
            g = min(1.0, max(0.0, (original_len * w / (2 * math.pi) - alpha) / (beta - alpha)))
            w = (1 - g) * w / factor + g * w
        f.append(w)
    return f


def rope(x, positions, rotary, interleaved, freq, scale=1.0):
    """x [rows][heads][dim] as float64; rows at negative positions stay."""
    y = x.double().clone()
    p = positions.double()
    for i, w in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        c, s = torch.cos(p * w)[:, None] * scale, torch.sin(p * w)[:, None] * scale
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return torch.where((positions >= 0)[:, None, None], y, x.double())


# ------------------------------------------------------------------ codes

def round_e4m3(y):
    """Nearest e4m3 value (ties to even, saturating at 448), float64 numpy."""
    y = np.asarray(y, dtype=np.float64)
    mag = np.minimum(np.abs(y), 448.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(mag > 0, mag, 1.0)))
    e = np.where(np.ldexp(1.0, e.astype(int)) > mag, e - 1, e)
    unit = np.ldexp(1.0, (np.clip(e, -6, 8) - 3).astype(int))
    r = np.minimum(np.rint(mag / unit) * unit, 448.0)
    return np.where(np.isnan(y), np.nan, np.copysign(r, y))


def scale_for(x):
    """The smallest power of two 2^e, -100 <= e <= 119, with amax <= 448 * 2^e."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    top = np.max(np.where(np.isfinite(x), x, 0.0), initial=0.0)
    e = -100
    while e < 119 and top > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


def append(x, slots, values, scale):
    """x [rows][heads][dim] float64 numpy; values [pages][heads][64][dim] are
    the codes' values without the scale.  Changes values and scale."""
    r, cap = 0, values.shape[0] * PAGE
    while r < len(slots):
        s = slots[r]
        if s < 0 or s >= cap:
            r += 1
            continue
        n = 1
        while r + n < len(slots) and slots[r + n] == s + n and (s + n) % PAGE:
            n += 1
        page, off = s // PAGE, s % PAGE
        for h in range(x.shape[1]):
            new = scale_for(x[r:r + n, h])
            if off and scale[page, h] >= new:
                new = scale[page, h]
            elif off:
                values[page, h, :off] = round_e4m3(values[page, h, :off] * (scale[page, h] / new))
            scale[page, h] = new
            values[page, h, off:off + n] = round_e4m3(x[r:r + n, h] / new)
        r += n


# ------------------------------------------------------------------ attention

def attend(q, kc, vc, k_scale, v_scale, table, kv_len, row_start, causal, window, scale):
    """q [rows][n_q][dim]; kc, vc the pool's code values [pages][n_kv][64][dim]
    and scales [pages][n_kv], all float64.  Returns a dict: out and lse (rows
    in no sequence: NaN) and what the kernel's error bounds are made of:
    mag = sum w |v| per output element, terms = the largest sum |q_d k_d| *
    scale of a visible key, qabs = the largest max|q| sum |k_d| * scale,
    unit = n * 448 * the largest (weight * v scale) (one f16 step of a
    flushed weight, in outputs)."""
    rows, n_q, dim = q.shape
    group = n_q // kc.shape[1]
    nan = float("nan")
    r = {"out": torch.full((rows, n_q, dim), nan, dtype=torch.float64),
         "mag": torch.zeros((rows, n_q, dim), dtype=torch.float64),
         "lse": torch.full((rows, n_q), nan, dtype=torch.float64),
         "terms": torch.zeros((rows, n_q), dtype=torch.float64),
         "qabs": torch.zeros((rows, n_q), dtype=torch.float64),
         "unit": torch.zeros((rows, n_q, 1), dtype=torch.float64)}
    for s, kv in enumerate(kv_len):
        r0, n = row_start[s], row_start[s + 1] - row_start[s]
        pages = table[s][:-(-kv // PAGE)]
        for h in range(kc.shape[1] if n > 0 else 0):
            ks = (kc[pages, h] * k_scale[pages, h][:, None, None]).reshape(-1, dim)[:kv]
            vs = (vc[pages, h] * v_scale[pages, h][:, None, None]).reshape(-1, dim)[:kv]
            sc = v_scale[pages, h].repeat_interleave(PAGE)[:kv]
            for i in range(n):
                p = kv - n + i
                lo, hi = 0, (p + 1 if causal else kv)
                if window:
                    lo = (p + 1 if causal else kv - n) - window
                lo, hi = max(lo, 0), max(hi, 0)
                g = slice(h * group, (h + 1) * group)
                if lo >= hi:
                    r["out"][r0 + i, g], r["lse"][r0 + i, g] = 0.0, -math.inf
                    continue
                x = q[r0 + i, g] @ ks[lo:hi].T * scale
                w = torch.softmax(x, 1)
                r["out"][r0 + i, g] = w @ vs[lo:hi]
                r["mag"][r0 + i, g] = w @ vs[lo:hi].abs()
                r["lse"][r0 + i, g] = torch.logsumexp(x, 1)
                r["terms"][r0 + i, g] = (q[r0 + i, g].abs() @ ks[lo:hi].abs().T).amax(1) * scale
                r["qabs"][r0 + i, g] = q[r0 + i, g].abs().amax(1) * ks[lo:hi].abs().sum(1).max() * scale
                r["unit"][r0 + i, g, 0] = (w * sc[lo:hi]).amax(1) * 448 * (hi - lo)
    return r
