"""The 8-bit paged KV cache's operators as measured work: page plans, rotary
positions, the cache's append and the attention that reads it.

A case names an operator and its sizes; `prepare` makes what a serving loop
has in hand, `run` is one call (or, for "layer", the calls of one decoder
layer in a row), in plain torch where `own` is false and through
`block_diffusion_speculative_gather_gb300.capi` where it is true.

Head counts, head_dim, block rows, windows and cache lengths are those of the
package's workloads (32 q / 8 kv heads of 128, blocks of 16 rows, a window of
2048, caches of 1024 to 16384 positions), head_dim 64 with an uneven head
group beside them.
"""

import math
import random

import torch

own = False

PAGE = 64          # tokens of a page; one scale per page and kv head
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

_lib = None


def _capi():
    global _lib
    if _lib is None:
        from block_diffusion_speculative_gather_gb300 import capi
        _lib = capi
    return _lib


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the page plan of one verify round: 32 sequences, 16 rows each
        {"name": "plan_32", "op": "plan", "seqs": 32, "rows": 16, "keys": 16384, "lens": 1},
        # a scheduler's largest step: 2048 sequences, ragged prompt chunks
        {"name": "plan_2048", "op": "plan", "seqs": 2048, "rows": 64, "keys": 8192, "lens": 2},
        # q and k of one 16-row verify forward
        {"name": "rope_16", "op": "rope", "rows": 16, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "scaling": "none", "type": "bf16", "far": 1088},
        # a long prompt far out: half of the head rotated, pairs side by side, scaled by parts
        {"name": "rope_16384", "op": "rope", "rows": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 64, "interleaved": True, "scaling": "parts", "type": "bf16", "far": 1 << 20},
        # one new token for each of 32 sequences: pages partly filled
        {"name": "append_32", "op": "append", "seqs": 32, "rows": 1, "keys": 4096, "kv_heads": 8,
         "dim": 128, "type": "bf16", "lens": 3},
        # four long prompts entering the cache
        {"name": "append_prompt", "op": "append", "seqs": 4, "rows": 4096, "keys": 8192, "kv_heads": 8,
         "dim": 128, "type": "f16", "lens": 4},
        # one token of one sequence over a short cache: latency alone
        {"name": "attend_1", "op": "attend", "seqs": 1, "rows": 1, "keys": 1088, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16", "causal": True, "window": 0, "lens": 5},
        # single tokens of 32 sequences over long, ragged caches: the cache's bytes
        {"name": "attend_32", "op": "attend", "seqs": 32, "rows": 1, "keys": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16", "causal": True, "window": 0, "lens": 6},
        # verify of 16 rows for each of 8 sequences
        {"name": "attend_verify", "op": "attend", "seqs": 8, "rows": 16, "keys": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "f16", "causal": True, "window": 0, "lens": 7},
        # the drafter's masked blocks: bidirectional, window of 2048, head_dim 64, 5 q heads per kv head
        {"name": "attend_draft", "op": "attend", "seqs": 32, "rows": 16, "keys": 5000, "heads": 20,
         "kv_heads": 4, "dim": 64, "type": "bf16", "causal": False, "window": 2048, "lens": 8},
        # ragged prompt chunks behind earlier context
        {"name": "attend_prompt", "op": "attend", "seqs": 4, "rows": 2048, "keys": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16", "causal": True, "window": 0, "lens": 9},
        # plan, rotary positions, append and attention of one layer's verify rows
        {"name": "layer_verify", "op": "layer", "seqs": 8, "rows": 16, "keys": 4096, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16", "causal": True, "window": 0, "lens": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "rope", "append", "attend", "attend", "attend", "layer"))
    lens = rng.randrange(1 << 30)
    if op == "plan":
        return {"op": op, "seqs": _log(rng, 1, 2048), "rows": _log(rng, 1, 64),
                "keys": _log(rng, 64, 8192), "lens": lens}
    dim = rng.choice((64, 128))
    kind = rng.choice(("bf16", "f16"))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8))
    if op == "rope":
        dim = rng.choice((32, 64, 80, 96, 128))
        return {"op": op, "rows": _log(rng, 1, 8192), "heads": kv_heads * min(group, 5), "kv_heads": kv_heads,
                "dim": dim, "rotary": rng.choice((dim, dim // 2, dim // 4)),
                "interleaved": rng.random() < 0.5, "scaling": rng.choice(("none", "linear", "parts")),
                "type": rng.choice(("bf16", "f16", "f32")), "far": _log(rng, 64, 1 << 20)}
    if op == "append":
        seqs = _log(rng, 1, 32)
        rows = _log(rng, 1, 4096 // seqs)
        return {"op": op, "seqs": seqs, "rows": rows, "keys": rows + _log(rng, 1, 2048),
                "kv_heads": kv_heads, "dim": dim, "type": rng.choice(("bf16", "f16", "f32")), "lens": lens}
    causal = rng.random() < 0.75 or op == "layer"
    seqs = _log(rng, 1, 24)
    if op == "layer" or not causal:
        rows = rng.randint(2, 16)
    else:
        rows = rng.choice((1, rng.randint(2, 16), _log(rng, 17, 1024)))
    keys = rows + _log(rng, 1, 12000)
    while seqs > 1 and (seqs * keys > 180000 or seqs * rows * keys > 16000000):
        seqs -= 1
    window = rng.choice((0, 0, _log(rng, 16, 4096)))
    return {"op": op, "seqs": seqs, "rows": rows, "keys": keys, "heads": kv_heads * min(group, 5),
            "kv_heads": kv_heads, "dim": dim, "type": kind, "causal": causal,
            "window": 0 if op == "layer" else window, "lens": lens}


def _lengths(case):
    """Rows and cached tokens (rows included) of each sequence, from the case
    alone: the first sequence has the most of both, the others are ragged."""
    r = random.Random(case["lens"])
    rows, held = [], []
    for s in range(case["seqs"]):
        n = case["rows"] if s == 0 or case["rows"] == 1 else r.randint(max(1, case["rows"] // 4), case["rows"])
        past = case["keys"] - case["rows"]
        past = past if s == 0 else r.randint(past // 4, past)
        rows.append(n)
        held.append(past + n)
    return rows, held


def _visible(case):
    """(query, key) pairs that the masks leave, and keys that some row sees."""
    rows, held = _lengths(case)
    w, pairs, keys = case["window"], 0, 0
    for n, kv in zip(rows, held):
        first = kv - n
        if case["causal"]:
            pairs += sum(min(p + 1, w) if w else p + 1 for p in range(first, kv))
            keys += kv - (max(0, first + 1 - w) if w else 0)
        else:
            lo = max(0, first - w) if w else 0
            pairs += n * (kv - lo)
            keys += kv - lo
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "plan":
        rows, held = _lengths(case)
        new = sum(-(-kv // PAGE) - -(-(kv - n) // PAGE) for n, kv in zip(rows, held))
        # lengths, free pages and the entries that positions look up; row maps, lengths, new entries
        look = sum(-(-kv // PAGE) - (kv - n) // PAGE for n, kv in zip(rows, held))
        return {"bytes": 4.0 * (4 * case["seqs"] + 2 * new + look + 2 * sum(rows)), "flops": 0.0}
    if op == "rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"])
        size = TYPES[case["type"]].itemsize
        return {"bytes": 2.0 * n * case["dim"] * size + 4.0 * case["rows"], "flops": 3.0 * n * case["rotary"]}
    if op == "append":
        rows, held = _lengths(case)
        n = 2.0 * sum(rows) * case["kv_heads"] * case["dim"]
        return {"bytes": n * (TYPES[case["type"]].itemsize + 1) + 4.0 * sum(rows), "flops": 2.0 * n}
    rows, held = _lengths(case)
    pairs, keys = _visible(case)
    size = TYPES[case["type"]].itemsize
    b = 2.0 * keys * case["kv_heads"] * (case["dim"] + 4.0 / PAGE) + 4.0 * keys / PAGE
    b += 2.0 * sum(rows) * case["heads"] * case["dim"] * size + 4.0 * sum(rows) * case["heads"]
    f = 4.0 * pairs * case["heads"] * case["dim"]
    if op == "layer":
        n = sum(rows) * (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        b += 2.0 * n * size
        f += 5.0 * n
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(case, seed, pages, g):
    """A cache pool whose pages hold quantised tokens: codes of a spread that
    uses the format, scales that differ from page to page."""
    def codes():
        c = torch.randn((pages, case["kv_heads"], PAGE, case["dim"]), generator=g, device="cuda")
        return (c * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales():
        e = torch.randint(-8, -5, (pages, case["kv_heads"]), generator=g, device="cuda")
        return torch.exp2(e.float())
    return {"k_codes": codes(), "v_codes": codes(), "k_scale": scales(), "v_scale": scales()}


def _tables(held, width, order):
    """Block table with the pages of `order` handed out in turn, -1 behind."""
    table, at = [], 0
    for kv in held:
        n = -(-kv // PAGE)
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return _ints(table), at


def _prepare_rows(case, seed, st, g):
    """Row starts, positions and slots of the case's new rows, with two rows
    of padding behind the last sequence."""
    rows, held = _lengths(case)
    width = -(-case["keys"] // PAGE)
    pages = sum(-(-kv // PAGE) for kv in held)
    order = list(range(pages + 2))
    random.Random(seed).shuffle(order)
    st["table"], _ = _tables(held, width, order)
    start, pos, slot, at = [0], [], [], 0
    for n, kv in zip(rows, held):
        for p in range(kv - n, kv):
            pos.append(p)
            slot.append(order[at + p // PAGE] * PAGE + p % PAGE)
        at += -(-kv // PAGE)
        start.append(start[-1] + n)
    st["row_start"], st["kv_len"] = _ints(start), _ints(held)
    st["positions"], st["slots"] = _ints(pos + [-1, -1]), _ints(slot + [-1, -1])
    st["max_rows"] = max(rows)
    return pages + 2


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    op = case["op"]
    if op in ("plan", "layer"):
        rows, held = _lengths(case)
        width = -(-case["keys"] // PAGE) + 1
        before = [kv - n for n, kv in zip(rows, held)]
        used = sum(-(-kv // PAGE) for kv in before)
        need = sum(-(-kv // PAGE) for kv in held)
        order = list(range(need + 8))
        random.Random(seed).shuffle(order)
        st["table"], at = _tables(before, width, order)
        st["free"] = _ints(order[at:] + [-1] * used)
        st["n_free"] = _ints([len(order) - at])
        st["before"], st["q_len"] = _ints(before), _ints(rows)
        total = sum(rows) + 2
        st["row_start"] = _ints([0] * (len(rows) + 1))
        st["positions"], st["slots"] = _ints([0] * total), _ints([0] * total)
        st["kv_len"], st["n_free_out"] = _ints([0] * len(rows)), _ints([0])
        st["max_rows"] = max(rows)
        if op == "plan":
            return st
        st |= _pool(case, seed, need + 8, g)
    if op == "rope":
        kind, far = TYPES[case["type"]], case["far"]
        first = max(0, far - case["rows"])
        # rows of one sequence up to position `far`
        pos = torch.arange(first, first + case["rows"], device="cuda", dtype=torch.int32)
        st["positions"] = pos
        n = case["heads"] + case["kv_heads"]
        st["qk"] = torch.randn((case["rows"], n, case["dim"]), generator=g, device="cuda").to(kind)
        st["out"] = torch.empty_like(st["qk"])
        return st
    if op in ("append", "attend"):
        pages = _prepare_rows(case, seed, st, g)
        st |= _pool(case, seed, pages, g)
    kind, total = TYPES[case["type"]], st["positions"].numel()
    if op == "append":
        # k and v stand in one projection's rows: strided views of it
        kv = torch.randn((total, 2, case["kv_heads"], case["dim"]), generator=g, device="cuda")
        kv *= torch.exp(0.5 * torch.randn((total, 1, 1, 1), generator=g, device="cuda"))
        st["kv"] = kv.to(kind)
        return st
    if op == "layer":
        n = case["heads"] + 2 * case["kv_heads"]
        st["qkv"] = torch.randn((total, n, case["dim"]), generator=g, device="cuda").to(kind)
        st["rot"] = torch.empty((total, n - case["kv_heads"], case["dim"]), dtype=kind, device="cuda")
        st["rot"].zero_()
    else:
        # rows a user has scaled to attend sharply to some keys
        q = 1.5 * torch.randn((total, case["heads"], case["dim"]), generator=g, device="cuda")
        st["q"] = q.to(kind)
    st["out"] = torch.full((total, case["heads"], case["dim"]), 0.5, dtype=kind, device="cuda")
    st["lse"] = torch.full((total, case["heads"]), 0.5, device="cuda")
    return st


# ------------------------------------------------------------------ rotary settings

def _rope_settings(case):
    """theta, kind of scaling, its factor and original length, and the scale
    of the rotated values."""
    if case["op"] != "rope" or case["scaling"] == "none":
        return {"theta": 1e6, "scaling": "none", "factor": 1.0, "original_len": 0, "scale": 1.0}
    if case["scaling"] == "linear":
        return {"theta": 1e4, "scaling": "linear", "factor": 4.0, "original_len": 0, "scale": 1.0}
    return {"theta": 1e6, "scaling": "parts", "factor": 32.0, "original_len": 32768, "scale": 1.2}


def _frequencies(rotary, settings):
    """Radians a position, in 64 bits."""
    i = torch.arange(rotary // 2, dtype=torch.float64, device="cuda")
    f = settings["theta"] ** (-2.0 * i / rotary)
    if settings["scaling"] == "linear":
        return f / settings["factor"]
    if settings["scaling"] == "parts":
        turns = settings["original_len"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return (1 - keep) * f / settings["factor"] + keep * f
    return f


# ------------------------------------------------------------------ plain forms

def _plan_plain(st):
    before, q, table = st["before"].long(), st["q_len"].long(), st["table"]
    width, total = table.shape[1], st["positions"].numel()
    old, new = (before + PAGE - 1) // PAGE, (before + q + PAGE - 1) // PAGE
    fine = new <= width
    need, rows = torch.where(fine, new - old, 0), torch.where(fine, q, 0)
    ok = fine & (need.cumsum(0) <= st["n_free"]) & (rows.cumsum(0) <= total)
    need, rows = torch.where(ok, need, 0), torch.where(ok, rows, 0)
    start = torch.cat((torch.zeros_like(rows[:1]), rows.cumsum(0)))
    handed = need.cumsum(0) - need
    j = torch.arange(width, device=table.device)
    i = handed[:, None] + j - old[:, None]
    fresh = (j >= old[:, None]) & (j < (old + need)[:, None])
    page = st["free"][(st["n_free"].long() - 1 - i).clamp(0, st["free"].numel() - 1)]
    table = torch.where(fresh, page, table)
    r = torch.arange(total, device=table.device)
    s = torch.searchsorted(start[1:], r, right=True).clamp(max=rows.numel() - 1)
    pos = before[s] + r - start[s]
    slot = table[s, (pos // PAGE).clamp(0, width - 1)].long() * PAGE + pos % PAGE
    there = r < start[-1]
    return {"table": table, "row_start": start.int(), "positions": torch.where(there, pos, -1).int(),
            "slots": torch.where(there, slot, -1).int(), "kv_len": (before + rows).int(),
            "n_free": (st["n_free"] - need.sum()).int()}


def _rope_plain(case, x, positions, rotary, interleaved):
    settings = _rope_settings(case)
    angle = positions.double()[:, None] * _frequencies(rotary, settings)
    c = (angle.cos() * settings["scale"]).float()[:, None, :]
    s = (angle.sin() * settings["scale"]).float()[:, None, :]
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rotary:2], y[..., 1:rotary:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = y[..., :rotary // 2], y[..., rotary // 2:rotary]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, y[..., rotary:]), -1).to(x.dtype)


def _step(amax):
    """The smallest power of two that brings `amax` within the format."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-100, 119)
    return torch.exp2(torch.where(amax > 0, e, -100).float())


def _append_plain(st, x, slots, row_start, codes, scale):
    x, total = x.float(), row_start[-1].long()
    r = torch.arange(slots.numel(), device=x.device)
    r = torch.minimum(r, total - 1)  # padding repeats the last row
    x, slot = x[r], slots[r].long()
    page, off = slot // PAGE, slot % PAGE
    pages, heads = scale.shape
    first = torch.full((pages,), PAGE, device=x.device, dtype=torch.long).scatter_reduce(0, page, off, "amin")
    top = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
    step = _step(top)
    new = torch.where((first > 0)[:, None], torch.maximum(scale, step), step)
    new = torch.where((first < PAGE)[:, None], new, scale)
    # only a sequence's first page of the call can hold earlier tokens
    p = page[torch.minimum(row_start[:-1].long(), total - 1)]
    held = codes[p].view(torch.float8_e4m3fn).float() * (scale / new)[p][:, :, None, None]
    keep = torch.arange(PAGE, device=x.device)[None, None, :, None] < first[p][:, None, None, None]
    codes[p] = torch.where(keep, held.to(torch.float8_e4m3fn).view(torch.uint8), codes[p])
    y = (x / new[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes[page, :, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(new)


def _attend_plain(st, q):
    case, table = st["case"], st["table"].clamp(min=0).long()
    seqs, dim, kvh = case["seqs"], case["dim"], case["kv_heads"]
    group, most = case["heads"] // kvh, st["max_rows"]
    start, held = st["row_start"].long(), st["kv_len"].long()
    keys = table.shape[1] * PAGE

    def cached(codes, scale):
        v = codes[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return v.transpose(1, 2).reshape(seqs, kvh, keys, dim)

    k, v = cached(st["k_codes"], st["k_scale"]), cached(st["v_codes"], st["v_scale"])
    i = torch.arange(most, device=q.device)
    at = (start[:-1, None] + i).clamp(max=q.shape[0] - 1)
    n = start[1:] - start[:-1]
    rows = q[at].float().view(seqs, most, kvh, group, dim).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(rows.reshape(seqs, kvh, group * most, dim), k.transpose(2, 3))
    scores = scores.view(seqs, kvh, group, most, keys).mul_(dim ** -0.5)
    j = torch.arange(keys, device=q.device)
    first = (held - n)[:, None, None]
    pos = first + i[:, None]
    if case["causal"]:
        seen = j <= pos
        if case["window"]:
            seen &= j > pos - case["window"]
    else:
        seen = j < held[:, None, None]
        if case["window"]:
            seen = seen & (j >= first - case["window"])
    seen = seen & (j < held[:, None, None])
    scores.masked_fill_(~seen[:, None, None].expand(seqs, 1, 1, most, keys), -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, kvh, group * most, keys), v).view(seqs, kvh, group, most, dim)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log()).squeeze(-1)
    r = torch.arange(q.shape[0], device=q.device)
    s = torch.searchsorted(start[1:], r, right=True).clamp(max=seqs - 1)
    w = (r - start[s]).clamp(0, most - 1)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, most, kvh * group, dim)[s, w].to(q.dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(seqs, most, kvh * group)[s, w]
    there = r < start[-1]
    return {"out": torch.where(there[:, None, None], o, st["out"]),
            "lse": torch.where(there[:, None], lse, st["lse"])}


def _cache_values(st):
    """The cache as the values its codes stand for, beside their scales."""
    return {"k": st["k_codes"].view(torch.float8_e4m3fn), "v": st["v_codes"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "plan":
        return _plan_plain(st)
    if op == "rope":
        return _rope_plain(case, st["qk"], st["positions"], case["rotary"], case["interleaved"])
    if op == "append":
        _append_plain(st, st["kv"][:, 0], st["slots"], st["row_start"], st["k_codes"], st["k_scale"])
        _append_plain(st, st["kv"][:, 1], st["slots"], st["row_start"], st["v_codes"], st["v_scale"])
        return _cache_values(st)
    if op == "attend":
        return _attend_plain(st, st["q"])
    plan = _plan_plain(st)
    h, n = case["heads"], case["heads"] + case["kv_heads"]
    there = (plan["positions"] >= 0)[:, None, None]
    rot = _rope_plain(case, st["qkv"][:, :n], plan["positions"].clamp(min=0), case["dim"], False)
    rot = torch.where(there, rot, st["rot"])
    _append_plain(st, rot[:, h:], plan["slots"], plan["row_start"], st["k_codes"], st["k_scale"])
    _append_plain(st, st["qkv"][:, n:], plan["slots"], plan["row_start"], st["v_codes"], st["v_scale"])
    return _attend_plain({**st, **plan}, rot[:, :h]) | _cache_values(st)


# ------------------------------------------------------------------ the framework's calls

def _plan_own(c, st):
    c.dflash_pages_plan(st["before"], st["q_len"], st["free"], st["n_free"], st["table"], st["row_start"],
                        st["positions"], st["slots"], st["kv_len"], st["n_free_out"])
    return {"table": st["table"], "row_start": st["row_start"], "positions": st["positions"],
            "slots": st["slots"], "kv_len": st["kv_len"], "n_free": st["n_free_out"]}


def _rope_own(c, st, q, k, out_q, out_k, rotary, interleaved):
    if "turns" not in st:
        w = _rope_settings(st["case"])
        st["rope"] = c.rope_config(rotary_dim=rotary, interleaved=interleaved, **w)
        st["turns"] = torch.empty(rotary // 2, dtype=torch.int64, device="cuda")
        c.dflash_rope_turns(st["rope"], st["turns"])
    c.dflash_rope(st["rope"], st["turns"], st["positions"], q, out_q, k, out_k)


def _err(st):
    if "err" not in st:
        st["err"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    return st["err"]


def _append_own(c, st, k, v):
    c.dflash_kv8_append(k, v, st["slots"], st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], _err(st))


def _attend_own(c, st, q):
    case = st["case"]
    if "workspace" not in st:
        size = c.dflash_kv8_workspace_bytes(q.shape[0], case["seqs"], case["heads"], case["kv_heads"],
                                            case["dim"], st["table"].shape[1])
        st["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    c.dflash_kv8_attention(q, st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"],
                           st["kv_len"], st["row_start"], st["out"], st["workspace"], _err(st),
                           lse=st["lse"], causal=case["causal"], window=case["window"])
    return {"out": st["out"], "lse": st["lse"]}


def _run_own(st):
    c, case, op = _capi(), st["case"], st["case"]["op"]
    if op == "plan":
        return _plan_own(c, st)
    if op == "rope":
        h = case["heads"]
        _rope_own(c, st, st["qk"][:, :h], st["qk"][:, h:], st["out"][:, :h], st["out"][:, h:],
                  case["rotary"], case["interleaved"])
        return st["out"]
    if op == "append":
        _append_own(c, st, st["kv"][:, 0], st["kv"][:, 1])
        return _cache_values(st)
    if op == "attend":
        return _attend_own(c, st, st["q"])
    h, n = case["heads"], case["heads"] + case["kv_heads"]
    _plan_own(c, st)
    _rope_own(c, st, st["qkv"][:, :h], st["qkv"][:, h:n], st["rot"][:, :h], st["rot"][:, h:], case["dim"], False)
    _append_own(c, st, st["rot"][:, h:], st["qkv"][:, n:])
    return _attend_own(c, st, st["rot"][:, :h]) | _cache_values(st)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ 64-bit definitions

def _exact_round(y):
    """e4m3 of values within the format: three bits below the leading one, steps of 2^-9 at the least."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > y.abs(), e - 1, e).clamp(min=-6)
    unit = torch.exp2(e - 3)
    return torch.round(y / unit) * unit


def _exact_append(x, rows, held, pages_of, codes, scale):
    """Page by page: the scale, the earlier tokens re-rounded, the new ones."""
    values = codes.view(torch.float8_e4m3fn).double()
    scale = scale.double().clone()
    at = 0
    for s, (n, kv) in enumerate(zip(rows, held)):
        p = kv - n
        while p < kv:
            stop = min(kv, (p // PAGE + 1) * PAGE)
            page, off = pages_of[s][p // PAGE], p % PAGE
            new = x[at:at + stop - p].double().transpose(0, 1)
            top = new.abs().amax((1, 2))
            e = torch.ceil(torch.log2(top / E4M3_MAX))
            e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= top, e - 1, e)
            e = torch.where(torch.exp2(e) * E4M3_MAX < top, e + 1, e)
            unit = torch.exp2(e.clamp(-100, 119))
            if off:
                unit = torch.maximum(unit, scale[page])
                values[page, :, :off] = _exact_round(values[page, :, :off] * (scale[page] / unit)[:, None, None])
            values[page, :, off:off + stop - p] = _exact_round(new / unit[:, None, None])
            scale[page] = unit
            at += stop - p
            p = stop
    return values, scale


def _exact_rope(case, x, positions, rotary, interleaved):
    w = _rope_settings(case)
    x, out = x.double(), x.double().clone()
    for i in range(rotary // 2):
        f = w["theta"] ** (-2.0 * i / rotary)
        if w["scaling"] == "linear":
            f = f / w["factor"]
        elif w["scaling"] == "parts":
            g = min(1.0, max(0.0, (w["original_len"] * f / (2 * math.pi) - 1.0) / 31.0))
            f = f * g + f / w["factor"] * (1 - g)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        z = torch.polar(torch.full_like(positions, w["scale"], dtype=torch.float64), positions.double() * f)
        turned = torch.complex(x[..., a], x[..., b]) * z[:, None]
        out[..., a], out[..., b] = turned.real, turned.imag
    return out


def _exact_attend(case, q, pages_of, k, v, out, lse):
    """Sequence by sequence; k and v are the whole pool's values."""
    rows, held = _lengths(case)
    group, at = case["heads"] // case["kv_heads"], 0
    for s, (n, kv) in enumerate(zip(rows, held)):
        pages = torch.tensor(pages_of[s], device="cuda")
        ks = k[pages].transpose(1, 2).flatten(0, 1)[:kv]
        vs = v[pages].transpose(1, 2).flatten(0, 1)[:kv]
        j = torch.arange(kv, device="cuda")
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        if case["causal"]:
            hide = j > p
            if case["window"]:
                hide |= j <= p - case["window"]
        else:
            hide = (j < (kv - n - case["window"]) if case["window"] else j < 0).expand(n, kv)
        for h in range(case["heads"]):
            x = q[at:at + n, h].double() @ ks[:, h // group].T / math.sqrt(case["dim"])
            x = x.masked_fill(hide, -math.inf)
            lse[at:at + n, h] = torch.logsumexp(x, 1)
            out[at:at + n, h] = torch.softmax(x, 1) @ vs[:, h // group]
        at += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    st = prepare(case, seed)
    if op == "rope":
        return _exact_rope(case, st["qk"], st["positions"], case["rotary"], case["interleaved"])
    rows, held = _lengths(case)
    pages_of = st["table"].tolist()
    if op == "attend":
        pages_of = [t[:-(-kv // PAGE)] for t, kv in zip(pages_of, held)]
        k, v = (st[n + "_codes"].view(torch.float8_e4m3fn).double() * st[n + "_scale"].double()[..., None, None]
                for n in "kv")
        return _exact_attend(case, st["q"], pages_of, k, v, st["out"].double(), st["lse"].double())
    if op == "append":
        k, ks = _exact_append(st["kv"][:, 0], rows, held, pages_of, st["k_codes"], st["k_scale"])
        v, vs = _exact_append(st["kv"][:, 1], rows, held, pages_of, st["v_codes"], st["v_scale"])
        return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}
    # one layer: the rotated rows are rounded to the rows' type before they are cached and attended with
    free = st["free"].tolist()[:int(st["n_free"])]
    for s, (n, kv) in enumerate(zip(rows, held)):
        had = -(-(kv - n) // PAGE)
        pages_of[s] = pages_of[s][:had] + [free.pop() for _ in range(had, -(-kv // PAGE))]
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in zip(rows, held)]).cuda()
    h, m = case["heads"], case["heads"] + case["kv_heads"]
    rot = _exact_rope(case, st["qkv"][:len(pos), :m], pos, case["dim"], False).to(TYPES[case["type"]])
    k, ks = _exact_append(rot[:, h:], rows, held, pages_of, st["k_codes"], st["k_scale"])
    v, vs = _exact_append(st["qkv"][:, m:], rows, held, pages_of, st["v_codes"], st["v_scale"])
    got = _exact_attend(case, rot[:, :h], pages_of, k * ks[..., None, None], v * vs[..., None, None],
                        st["out"].double(), st["lse"].double())
    return got | {"k": None, "v": None, "k_scale": ks, "v_scale": vs}
