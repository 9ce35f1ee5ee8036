"""What stays of a serving step, as measured work: probabilities of logits,
verification of drafted tokens from given random numbers, and eviction from
the 8-bit paged cache by accumulated attention weight.

A case names an operator and its sizes; `prepare` makes what a serving loop
has in hand, `run` is one call (or, for "step", the calls between two forwards
in a row), in plain torch where `own` is false and through
`block_diffusion_speculative_gather_gb300.capi` where it is true.

Vocabularies, head counts, block rows and cache lengths are those of the
package's workloads (151936 and 4096 tokens, 32 q / 8 kv heads of 128, blocks
of 16 rows, 1024 to 16384 positions, 5 drafter layers), with uneven ones
beside them.
"""

import math
import random

import torch

own = False

PAGE = 64          # positions of a page; one scale per page and kv head
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
        # the next token's probabilities of one sequence: latency
        {"name": "probs_1", "op": "probs", "rows": 1, "vocab": 151936, "type": "f32", "min_p": False},
        # bf16 logits of an odd vocabulary (rows of every alignment), small probabilities cut off
        {"name": "probs_odd", "op": "probs", "rows": 77, "vocab": 32003, "type": "bf16", "min_p": True},
        # the verify rows of 32 sequences
        {"name": "probs_512", "op": "probs", "rows": 512, "vocab": 151936, "type": "f32", "min_p": True},
        # one sequence's 16 verify rows
        {"name": "verify_1", "op": "verify", "seqs": 1, "rows": 16, "vocab": 151936, "drafts": "probs", "lens": 1},
        # 32 sequences, ragged blocks of up to 16 rows
        {"name": "verify_32", "op": "verify", "seqs": 32, "rows": 16, "vocab": 151936, "drafts": "probs", "lens": 2},
        # drawing the drafts themselves: 480 rows, a token each
        {"name": "draw_480", "op": "verify", "seqs": 480, "rows": 1, "vocab": 151936, "drafts": "ids", "lens": 3},
        # one token of one sequence over a short cache: latency
        {"name": "weigh_1", "op": "weigh", "seqs": 1, "rows": 1, "keys": 1088, "heads": 32, "kv_heads": 8,
         "dim": 128, "type": "bf16", "observe": 0, "causal": True, "window": 0, "count": False, "lens": 4},
        # single tokens of 32 sequences over long, ragged caches: the cached keys' bytes
        {"name": "weigh_32", "op": "weigh", "seqs": 32, "rows": 1, "keys": 16384, "heads": 32, "kv_heads": 8,
         "dim": 128, "type": "bf16", "observe": 0, "causal": True, "window": 0, "count": False, "lens": 5},
        # the last 64 rows of four prompts count
        {"name": "weigh_prompt", "op": "weigh", "seqs": 4, "rows": 1024, "keys": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "type": "f16", "observe": 64, "causal": True, "window": 0, "count": False, "lens": 6},
        # one sequence of the drafter's five layers is halved
        {"name": "evict_1", "op": "evict", "seqs": 1, "keys": 4096, "budget": 2048, "first": 4, "last": 128,
         "layers": 5, "kv_heads": 8, "dim": 128, "lens": 7},
        # eight ragged sequences of ten layers
        {"name": "evict_8", "op": "evict", "seqs": 8, "keys": 6000, "budget": 2500, "first": 4, "last": 256,
         "layers": 10, "kv_heads": 8, "dim": 128, "lens": 8},
        # between two forwards of 8 sequences: verify, trim, evict, trim, plan, positions
        {"name": "step_8", "op": "step", "seqs": 8, "rows": 16, "vocab": 151936, "drafts": "probs", "keys": 2100,
         "budget": 2048, "first": 4, "last": 256, "layers": 5, "kv_heads": 8, "dim": 128, "lens": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("probs", "probs", "verify", "verify", "weigh", "weigh", "weigh", "evict", "evict", "step"))
    lens = rng.randrange(1 << 30)
    vocab = rng.choice((4096, 151936, _log(rng, 1000, 151936)))
    if op == "probs":
        return {"op": op, "rows": _log(rng, 1, 400), "vocab": vocab, "type": rng.choice(("f32", "bf16", "f16")),
                "min_p": rng.random() < 0.5}
    if op == "verify":
        drafts = rng.choice(("probs", "probs", "ids"))
        rows = rng.choice((1, rng.randint(2, 16)))
        return {"op": op, "seqs": _log(rng, 1, 400 // rows), "rows": rows, "vocab": vocab, "drafts": drafts,
                "lens": lens}
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    if op == "weigh":
        group = rng.choice((1, 2, 4, 5, 8))
        causal = rng.random() < 0.75
        rows = rng.choice((1, rng.randint(2, 16), _log(rng, 17, 1024))) if causal else rng.randint(2, 16)
        observe = rng.choice((16, 32, 64)) if rows > 16 else rng.choice((0, 0, 8))
        seqs = _log(rng, 1, 24)
        keys = rows + _log(rng, 1, 12000)
        while seqs > 1 and (seqs * keys > 120000 or seqs * rows * keys > 16000000):
            seqs -= 1
        return {"op": op, "seqs": seqs, "rows": rows, "keys": keys, "heads": kv_heads * min(group, 4 + 12 // kv_heads),
                "kv_heads": kv_heads, "dim": dim, "type": rng.choice(("bf16", "f16")), "observe": observe,
                "causal": causal, "window": rng.choice((0, 0, _log(rng, 16, 4096))),
                "count": rows <= 16 and rng.random() < 0.5, "lens": lens}
    budget = _log(rng, 100, 2000)
    last = rng.randint(0, budget // 4)
    step = op == "step"
    rows = rng.randint(2, 16)
    keys = budget + (rows + rng.randint(0, 60) if step else _log(rng, 1, 3000))
    case = {"op": op, "seqs": _log(rng, 1, 8), "keys": keys, "budget": budget, "first": rng.choice((0, 1, 4)),
            "last": last, "layers": rng.randint(1, 5 if step else 8), "kv_heads": kv_heads, "dim": dim, "lens": lens}
    if step:
        case |= {"rows": rows, "vocab": vocab, "drafts": rng.choice(("probs", "ids"))}
    return case


def _lengths(case):
    """Rows and held positions (rows included) of each sequence, from the case
    alone: the first sequence has the most of both, the others are ragged."""
    r = random.Random(case["lens"])
    rows, held = [], []
    for s in range(case["seqs"]):
        most = case.get("rows", 1)
        n = most if s == 0 or most == 1 else r.randint(max(1, most // 4), most)
        past = case.get("keys", most) - most
        if case["op"] == "evict":
            # one in eight sequences is below its budget
            past = past if s == 0 else r.randint(past // 2, past) if s % 8 else min(past, case["budget"] - 2)
        elif case["op"] != "step":
            past = past if s == 0 else r.randint(past // 4, past)
        rows.append(n)
        held.append(past + n)
    return rows, held


def _counted(case):
    """Of each sequence: the first counted row and the one behind the last."""
    rows, _ = _lengths(case)
    r = random.Random(case["lens"] + 1)
    out = []
    for n in rows:
        c = r.randint(1, n) if case["count"] else n
        out.append((max(0, c - case["observe"]) if case["observe"] else 0, c))
    return out


def _visible(case):
    """(row, key) pairs that count and are seen, and keys that some counted row sees."""
    rows, held = _lengths(case)
    w, pairs, keys = case["window"], 0, 0
    for (i0, i1), n, kv in zip(_counted(case), rows, held):
        first = kv - n
        if case["causal"]:
            pairs += sum(min(first + i + 1, w) if w else first + i + 1 for i in range(i0, i1))
            keys += first + i1 - (max(0, first + i0 + 1 - w) if w else 0)
        else:
            lo = max(0, first - w) if w else 0
            pairs += (i1 - i0) * (kv - lo)
            keys += kv - lo
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "probs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (TYPES[case["type"]].itemsize + 4.0) + 8.0 * case["rows"], "flops": 4.0 * n}
    b = f = 0.0
    if op in ("verify", "step"):
        rows, _ = _lengths(case)
        # one row of each sequence whole, and the drafts' own two numbers
        q = case["drafts"] == "probs"
        n = float(case["seqs"]) * case["vocab"]
        b += n * (8 if q else 4) + 24.0 * sum(rows) + 12.0 * case["seqs"]
        f += 3.0 * n
    if op == "weigh":
        pairs, keys = _visible(case)
        counted = sum(b1 - a1 for a1, b1 in _counted(case))
        _, held = _lengths(case)
        b += keys * case["kv_heads"] * (case["dim"] + 4.0 / PAGE) + 8.0 * sum(held)
        b += counted * case["heads"] * (case["dim"] * 2.0 + 4.0)
        f += 2.0 * pairs * case["heads"] * case["dim"] + 3.0 * pairs * case["heads"]
    if op in ("evict", "step"):
        _, held = _lengths(case)
        moved = sum(case["budget"] - case["first"] for kv in held if kv > case["budget"])
        b += 4.0 * sum(held) + 8.0 * moved
        b += 4.0 * moved * case["layers"] * case["kv_heads"] * (case["dim"] + 4.0 / PAGE)
        f += moved
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _logits(rows, vocab, g):
    """A model's logits: a wide body and a few likely tokens a row."""
    x = torch.randn((rows, vocab), generator=g, device="cuda").mul_(2.0)
    at = torch.randint(0, vocab, (rows, 24), generator=g, device="cuda")
    up = 14.0 * torch.rand((rows, 24), generator=g, device="cuda")
    return x.scatter_(1, at, up + 3.0)


def _softmax(x):
    x = x.sub_(x.amax(1, keepdim=True)).exp_()
    return x.div_(x.sum(1, keepdim=True))


def _starts(rows):
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    return start


def _prepare_verify(case, st, g):
    """Target and drafter probabilities of the rows, the drafts drawn from the
    drafter's (or its likeliest tokens), and two rows of padding."""
    rows, held = _lengths(case)
    start, vocab = _starts(rows), case["vocab"]
    total = start[-1] + 2
    st["row_start"], st["kv_len"] = _ints(start), _ints(held)
    x = _logits(total, vocab, g)
    if case["drafts"] == "probs":
        # the drafter sees the row before: a noisy copy of the target's logits
        y = torch.empty_like(x)
        y[1:], y[0] = x[:-1], x[-1]
        y += 0.8 * torch.randn(y.shape, generator=g, device="cuda")
        y = _softmax(y)
        race = torch.empty_like(y).exponential_(generator=g)
        st["ids"] = torch.argmax(race.reciprocal_().mul_(y), 1).int()
        st["draft_probs"] = y
        del race
    else:
        y = x[[total - 1] + list(range(total - 1))] if max(rows) > 1 else x
        st["ids"] = torch.argmax(y, 1).int()
        st["draft_probs"] = None
    st["probs"] = _softmax(x)
    st["uniform"] = torch.rand(total, generator=g, device="cuda")
    st["tokens"] = _ints([-2] * total)
    st["n_tokens"], st["new_len"] = _ints([-2] * case["seqs"]), _ints([-2] * case["seqs"])


def _pool(case, layers, pages, g):
    """Pools whose pages hold quantised positions: codes of a spread that uses
    the format, scales that differ from page to page."""
    def codes():
        c = torch.empty((layers, pages, case["kv_heads"], PAGE, case["dim"]), dtype=torch.uint8, device="cuda")
        for i in range(layers):
            x = torch.randn(c.shape[1:], generator=g, device="cuda").mul_(100).clamp_(-E4M3_MAX, E4M3_MAX)
            c[i] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        return c

    def scales():
        e = torch.randint(-8, -5, (layers, pages, case["kv_heads"]), generator=g, device="cuda")
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


def _weights(pages, g):
    """Accumulated attention: a few heavy positions, many light ones, some never seen."""
    u = torch.rand((pages, PAGE), generator=g, device="cuda")
    w = u.pow(6).mul_(40.0)
    return torch.where(u < 0.05, torch.zeros_like(w), w)


def prepare(case, seed):
    g = _generator(seed)
    st, op = {"case": case}, case["op"]
    if op == "probs":
        x = _logits(case["rows"], case["vocab"], g)
        # some tokens are not allowed
        x.masked_fill_(torch.rand(case["vocab"], generator=g, device="cuda") < 0.05, -math.inf)
        st["logits"] = x.to(TYPES[case["type"]])
        st["temperature"] = 0.5 + 0.8 * torch.rand(case["rows"], generator=g, device="cuda")
        if case["rows"] > 8:
            st["temperature"][3::17] = 0.0       # greedy requests in the batch
        st["min_p"] = (0.02 + 0.08 * torch.rand(case["rows"], generator=g, device="cuda")) if case["min_p"] else None
        st["out"] = torch.zeros(x.shape, device="cuda")
        return st
    if op in ("verify", "step"):
        _prepare_verify(case, st, g)
    if op == "verify":
        return st
    rows, held = _lengths(case)
    width = -(-case["keys"] // PAGE) + 1
    used = sum(-(-kv // PAGE) for kv in held)
    order = list(range(used + 2 * case["seqs"]))
    random.Random(seed).shuffle(order)
    st["table"], at = _tables(held, width, order)
    st["kv_len"] = _ints(held)
    if op == "weigh":
        st |= {k: v[0] for k, v in _pool(case, 1, len(order), g).items()}
        start = _starts(rows)
        st["row_start"] = _ints(start)
        q = 1.5 * torch.randn((start[-1] + 2, case["heads"], case["dim"]), generator=g, device="cuda")
        st["q"] = q.to(TYPES[case["type"]])
        st["count"] = _ints([c for _, c in _counted(case)]) if case["count"] else None
        st["lse"] = _prepare_lse(st)
        st["weights"] = _weights(len(order), g)
        return st
    st |= _pool(case, case["layers"], len(order), g)
    st["weights"] = _weights(len(order), g)
    st["weights_out"] = torch.zeros_like(st["weights"])
    st["budget"] = _ints([case["budget"]] * case["seqs"])
    st["source"] = torch.full((case["seqs"], width * PAGE), -1, dtype=torch.int32, device="cuda")
    st["kept"], st["dropped"] = _ints([-2] * case["seqs"]), _ints([0] * case["seqs"])
    if op == "step":
        total = sum(rows) + 2
        st["free"], st["n_free"] = _ints(order[at:] + [-1] * at), _ints([len(order) - at])
        st["q_len"] = _ints(rows)
        st["positions"], st["slots"], st["angles"] = _ints([-1] * total), _ints([-1] * total), _ints([-1] * total)
    return st


def _prepare_lse(st):
    """What the attention of the step has left: the log of each row's sum."""
    case, rows, held = st["case"], *_lengths(st["case"])
    group, lse = case["heads"] // case["kv_heads"], []
    for s, (n, kv) in enumerate(zip(rows, held)):
        pages = st["table"][s, :-(-kv // PAGE)].long()
        k = st["k_codes"][pages].view(torch.float8_e4m3fn).float() * st["k_scale"][pages][..., None, None]
        k = k.transpose(0, 1).flatten(1, 2)[:, :kv]
        at = sum(rows[:s])
        q = st["q"][at:at + n].float().view(n, case["kv_heads"], group, case["dim"]).permute(1, 2, 0, 3)
        x = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).view(case["kv_heads"], group, n, kv)
        x *= case["dim"] ** -0.5
        j, p = torch.arange(kv, device="cuda"), torch.arange(kv - n, kv, device="cuda")[:, None]
        x.masked_fill_(~_seen(case, j, p, kv - n, kv), -math.inf)
        lse.append(torch.logsumexp(x, -1).permute(2, 0, 1).reshape(n, case["heads"]))
    lse.append(torch.zeros((2, case["heads"]), device="cuda"))
    return torch.cat(lse)


def _seen(case, j, p, first, kv):
    """Keys j that a row at position p sees; first: the sequence's first row."""
    w = case["window"]
    if case["causal"]:
        seen = j <= p
        return seen & (j > p - w) if w else seen
    seen = (j < kv) & (p == p)
    return seen & (j >= first - w) if w else seen


# ------------------------------------------------------------------ plain forms

def _probs_plain(st):
    x, t = st["logits"].float(), st["temperature"][:, None]
    x = torch.where(x == x, x, -math.inf)
    top = x.amax(1, keepdim=True)
    j = torch.arange(x.shape[1], device=x.device)
    best = torch.where(x == top, j, x.shape[1]).amin(1, keepdim=True)
    w = torch.exp((x - torch.where(top > -math.inf, top, 0.0)) / torch.where(t > 0, t, 1.0))
    if st["min_p"] is not None:
        # values next to the border: in 64 bits
        border = top.double() + t.double() * torch.log(st["min_p"].double())[:, None]
        w = torch.where(x.double() >= border, w, 0.0)
    total = w.sum(1, keepdim=True)
    p = torch.where(total > 0, w / total, 0.0)
    greedy = ((j == best) & (top > -math.inf)).float()
    return torch.where(t > 0, p, greedy)


def _verify_plain(st, probs, kv_len):
    ids, u, start = st["ids"].long(), st["uniform"].double(), st["row_start"].long()
    q, (total, vocab), seqs = st["draft_probs"], probs.shape, st["n_tokens"].numel()
    n = start[1:] - start[:-1]
    r = torch.arange(total, device=ids.device)
    s = torch.searchsorted(start[1:], r, right=True).clamp(max=seqs - 1)
    i, there = r - start[s], r < start[-1]
    there_id = (ids >= 0) & (ids < vocab)
    d = torch.where(there_id, ids, 0)
    p_d = probs[(r - 1).clamp(min=0), d].double()
    q_d = q[r, d].double() if q is not None else torch.ones_like(p_d)
    refused = there & (i > 0) & ~(there_id & (u * q_d < p_d))
    a = n.scatter_reduce(0, s, torch.where(refused, i, total), "amin") - 1
    at = (start[:-1] + a).clamp(max=total - 1)
    nxt = (at + 1).clamp(max=total - 1)
    drafted = (a + 1 < n) & there_id[nxt]
    w = probs[at].double()
    if q is not None:
        less = (w - q[nxt].double()).clamp(min=0)
    else:
        less = w.scatter(1, d[nxt][:, None], 0.0)
    less = torch.where(drafted[:, None], less, w)
    w = torch.where(less.sum(1, keepdim=True) > 0, less, w)
    cum = w.cumsum(1)
    goal = u[start[:-1].clamp(max=total - 1)] * cum[:, -1]
    v = torch.searchsorted(cum, goal[:, None], right=True)[:, 0].clamp(max=vocab - 1)
    shifted = ids[(r + 1).clamp(max=total - 1)]
    tok = torch.where(i < a[s], shifted, torch.where(i == a[s], v[s], -1))
    return {"tokens": torch.where(there, tok, st["tokens"].long()).int(),
            "n_tokens": torch.where(n > 0, a + 1, 0).int(),
            "new_len": (kv_len.long() - torch.where(n > 0, n - 1 - a, 0)).int()}


def _weigh_plain(st):
    case, table = st["case"], st["table"].clamp(min=0).long()
    seqs, dim, kvh = case["seqs"], case["dim"], case["kv_heads"]
    group, keys = case["heads"] // kvh, table.shape[1] * PAGE
    start, held = st["row_start"].long(), st["kv_len"].long()
    n = start[1:] - start[:-1]
    stop = st["count"].long() if st["count"] is not None else n
    begin = (stop - case["observe"]).clamp(min=0) if case["observe"] else torch.zeros_like(stop)
    most = min(case["rows"], case["observe"] or case["rows"])
    k = st["k_codes"][table].view(torch.float8_e4m3fn).float() * st["k_scale"][table][..., None, None]
    k = k.transpose(1, 2).reshape(seqs, kvh, keys, dim)
    i = begin[:, None] + torch.arange(most, device=table.device)
    at = (start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().view(seqs, most, kvh, group, dim).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(seqs, kvh, group * most, dim), k.transpose(2, 3))
    x = x.view(seqs, kvh, group, most, keys).mul_(dim ** -0.5)
    x -= st["lse"][at].view(seqs, most, kvh, group).permute(0, 2, 3, 1)[..., None]
    j = torch.arange(keys, device=table.device)
    first = (held - n)[:, None, None]
    seen = _seen(case, j, first + i[..., None], first, held[:, None, None]) & (i < stop[:, None])[..., None]
    x.masked_fill_(~seen[:, None, None].expand(seqs, 1, 1, most, keys), -math.inf)
    got = x.exp_().sum((1, 2, 3))
    slot = table[:, j // PAGE] * PAGE + j % PAGE
    w = st["weights"].view(-1)
    old = torch.where(j >= first[..., 0], 0.0, w[slot])     # the step's own positions start anew
    live = j < held[:, None]
    w[slot[live]] = (old + got)[live]
    return st["weights"]


def _moved_plain(codes, scale, src, dst, valid, pages):
    """Codes [layers][pages][kv heads][64][dim]: positions at slots src to slots
    dst (both [S][M], M whole pages) where valid; scales of the pages reached."""
    layers, heads = codes.shape[0], codes.shape[2]
    seqs, most = src.shape
    held = scale[:, src // PAGE]                                      # [layers][S][M][heads]
    there = valid[None, :, :, None]
    new = torch.where(there, held, 0.0).view(layers, seqs, most // PAGE, PAGE, heads).amax(3)
    ratio = held / new.repeat_interleave(PAGE, 2).where(there, held)
    x = codes.view(torch.float8_e4m3fn).float()[:, src // PAGE, :, src % PAGE]   # [S][M][layers][heads][dim]
    x = x * ratio.permute(1, 2, 0, 3)[..., None]
    x = x.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[:, (dst // PAGE)[valid], :, (dst % PAGE)[valid]] = x[valid]
    reached = valid.view(seqs, -1, PAGE).any(2)
    scale[:, pages[reached]] = new.transpose(0, 1).transpose(1, 2)[reached].transpose(0, 1)


def _evict_plain(st):
    case, table = st["case"], st["table"].clamp(min=0).long()
    held, budget, keys = st["kv_len"].long(), st["budget"].long(), table.shape[1] * PAGE
    j = torch.arange(keys, device=table.device)
    slot = table[:, j // PAGE] * PAGE + j % PAGE
    w = st["weights"].view(-1)[slot]
    goes = (budget > 0) & (held > budget)
    new = torch.where(goes, budget, held)
    last = new.clamp(max=case["last"])
    first = torch.minimum(new - last, torch.full_like(new, case["first"]))
    stays = (j < first[:, None]) | (j >= (held - last)[:, None])
    key = torch.where(stays, math.inf, w)
    key = torch.where(j < held[:, None], key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    keep = torch.zeros_like(stays).scatter(1, order, j < new[:, None])
    live = j < new[:, None]
    at = torch.sort((~keep).int(), dim=1, stable=True).indices       # kept positions first, in order
    st["source"].copy_(torch.where(live, at, st["source"].long()))
    most = min(keys, -(-case["budget"] // PAGE) * PAGE)
    src, dst, valid = slot.gather(1, at)[:, :most], slot[:, :most], (live & goes[:, None])[:, :most]
    pages = table[:, :most // PAGE]
    _moved_plain(st["k_codes"], st["k_scale"], src, dst, valid, pages)
    _moved_plain(st["v_codes"], st["v_scale"], src, dst, valid, pages)
    st["weights_out"].view(-1)[slot[live]] = w.gather(1, at)[live]
    st["dropped"] += (held - new).int()
    st["kept"].copy_(new)
    return _cache_values(st) | {"source": st["source"], "weights_out": st["weights_out"], "kept": st["kept"],
                                "dropped": st["dropped"]}


def _trim_plain(st, to):
    """Pages behind the new lengths back onto the free list, each sequence's last page first."""
    kv, table = st["kv_len"].long(), st["table"]
    to = torch.minimum(kv, to.long().clamp(min=0))
    had, has = (kv + PAGE - 1) // PAGE, (to + PAGE - 1) // PAGE
    gone = had - has
    before = st["n_free"].long() + gone.cumsum(0) - gone
    j = torch.arange(table.shape[1], device=table.device)
    leave = (j >= has[:, None]) & (j < had[:, None])
    at = before[:, None] + had[:, None] - 1 - j
    st["free"][at[leave]] = table[leave]
    st["n_free"] += gone.sum().int()
    st["table"].copy_(torch.where(leave, -1, table))
    st["kv_len"].copy_(to)


def _plan_plain(st):
    before, q, table = st["kv_len"].long(), st["q_len"].long(), st["table"]
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
    table.copy_(torch.where(fresh, page, table))
    r = torch.arange(total, device=table.device)
    s = torch.searchsorted(start[1:], r, right=True).clamp(max=rows.numel() - 1)
    pos = before[s] + r - start[s]
    slot = table[s, (pos // PAGE).clamp(0, width - 1)].long() * PAGE + pos % PAGE
    there = r < start[-1]
    st["row_start"].copy_(start)
    st["positions"].copy_(torch.where(there, pos, -1))
    st["slots"].copy_(torch.where(there, slot, -1))
    st["kv_len"].copy_(before + rows)
    st["n_free"] -= need.sum().int()
    # a sequence's true positions: those it has lost count
    st["dropped"].copy_(torch.where((rows > 0) & (before == 0), 0, st["dropped"]))
    st["angles"].copy_(torch.where(there, pos + st["dropped"][s], -1))


def _step_outputs(st):
    return {n: st[n] for n in ("table", "free", "n_free", "row_start", "positions", "slots", "kv_len", "angles")}


def _cache_values(st):
    """The cache as the values its codes stand for, beside their scales."""
    return {"k": st["k_codes"].view(torch.float8_e4m3fn), "v": st["v_codes"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _run_plain(st):
    op = st["case"]["op"]
    if op == "probs":
        return _probs_plain(st)
    if op == "verify":
        return _verify_plain(st, st["probs"], st["kv_len"])
    if op == "weigh":
        return _weigh_plain(st)
    if op == "evict":
        return _evict_plain(st)
    got = _verify_plain(st, st["probs"], st["kv_len"])
    _trim_plain(st, got["new_len"])
    got |= _evict_plain(st)
    _trim_plain(st, got["kept"])
    _plan_plain(st)
    return got | _step_outputs(st)


# ------------------------------------------------------------------ the framework's calls

def _err(st):
    if "err" not in st:
        st["err"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    return st["err"]


def _space(st, name, size):
    if name not in st:
        st[name] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return st[name]


def _verify_own(c, st):
    seqs, (rows, vocab) = st["n_tokens"].numel(), st["probs"].shape
    c.dflash_verify_drafts(st["probs"], st["ids"], st["uniform"], st["row_start"], st["tokens"], st["n_tokens"],
                           _space(st, "verify_space", c.dflash_verify_workspace_bytes(seqs, vocab)), _err(st),
                           draft_probs=st["draft_probs"], kv_len=st["kv_len"], new_len=st["new_len"])
    return {n: st[n] for n in ("tokens", "n_tokens", "new_len")}


def _evict_own(c, st):
    case = st["case"]
    if "layers" not in st:
        st["layers"] = c.kv8_layers([(st["k_codes"][i], st["v_codes"][i], st["k_scale"][i], st["v_scale"][i])
                                     for i in range(case["layers"])])
    seqs, width = st["table"].shape
    c.dflash_kv8_evict(st["layers"], st["table"], st["kv_len"], st["weights"], st["budget"], st["kept"], st["source"],
                       _space(st, "evict_space", c.dflash_kv8_evict_workspace_bytes(seqs, width)), _err(st),
                       weights_out=st["weights_out"], dropped=st["dropped"], keep_first=case["first"],
                       keep_last=case["last"])
    return _cache_values(st) | {"source": st["source"], "weights_out": st["weights_out"], "kept": st["kept"],
                                "dropped": st["dropped"]}


def _run_own(st):
    c, case, op = _capi(), st["case"], st["case"]["op"]
    if op == "probs":
        c.dflash_probs(st["logits"], st["temperature"], st["out"], min_p=st["min_p"])
        return st["out"]
    if op == "verify":
        return _verify_own(c, st)
    if op == "weigh":
        c.dflash_kv8_weigh(st["q"], st["lse"], st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"],
                           st["kv_len"], st["row_start"], st["weights"], _err(st), count=st["count"],
                           observe=case["observe"], fresh=True, causal=case["causal"], window=case["window"])
        return st["weights"]
    if op == "evict":
        return _evict_own(c, st)
    got = _verify_own(c, st)
    c.dflash_pages_trim(st["kv_len"], st["new_len"], st["free"], st["n_free"], st["table"])
    got |= _evict_own(c, st)
    c.dflash_pages_trim(st["kv_len"], st["kept"], st["free"], st["n_free"], st["table"])
    c.dflash_pages_plan(st["kv_len"], st["q_len"], st["free"], st["n_free"], st["table"], st["row_start"],
                        st["positions"], st["slots"], st["kv_len"], st["n_free"])
    c.dflash_pages_shift(st["positions"], st["row_start"], st["dropped"], st["angles"])
    return got | _step_outputs(st)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ 64-bit definitions

def _exact_probs(st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for r in range(out.shape[0]):
        x, t = st["logits"][r].double(), float(st["temperature"][r])
        if t == 0:
            out[r, int(torch.nonzero(x == x.max())[0])] = 1.0
            continue
        y = x / t
        if st["min_p"] is not None:
            y = torch.where(x >= x.max() + t * math.log(float(st["min_p"][r])), y, -math.inf)
        out[r] = torch.softmax(y, 0)
    return out


def _exact_weigh(st):
    case, (rows, held) = st["case"], _lengths(st["case"])
    weights, group, at = st["weights"].double().clone(), case["heads"] // case["kv_heads"], 0
    for s, ((i0, i1), n, kv) in enumerate(zip(_counted(case), rows, held)):
        pages = st["table"][s, :-(-kv // PAGE)].long()
        k = st["k_codes"][pages].view(torch.float8_e4m3fn).double() * st["k_scale"][pages].double()[..., None, None]
        got = torch.zeros(kv, dtype=torch.float64, device="cuda")
        for i in range(i0, i1):
            p = kv - n + i
            lo, hi = 0, p + 1 if case["causal"] else kv
            if case["window"]:
                lo = max(0, (p + 1 if case["causal"] else kv - n) - case["window"])
            q = st["q"][at + i].double().view(case["kv_heads"], group, -1)
            x = torch.einsum("hgd,phkd->hgpk", q, k).flatten(2)[..., lo:hi] / math.sqrt(case["dim"])
            x = x - st["lse"][at + i].double().view(case["kv_heads"], group, 1)
            got[lo:hi] += x.exp().sum((0, 1))
        old = torch.cat([weights[p] for p in pages])[:kv]
        old[kv - n:] = 0.0
        for b, p in enumerate(pages.tolist()):
            e = min(PAGE, kv - b * PAGE)
            weights[p, :e] = (old + got)[b * PAGE:b * PAGE + e]
        at += n
    return weights


def _exact_round(y):
    """e4m3 of values within the format: three bits below the leading one, steps of 2^-9 at the least."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > y.abs(), e - 1, e).clamp(min=-6)
    unit = torch.exp2(e - 3)
    return torch.round(y / unit) * unit


def _exact_evict(st, held, table):
    """Sequence by sequence, page by page, all layers and heads at once.  Values stay e4m3 values: in 32 bits."""
    case = st["case"]
    weights, out = st["weights"].double().tolist(), st["weights_out"].double().clone()
    got = {}
    values = {n: st[n + "_codes"].view(torch.float8_e4m3fn).float() for n in "kv"}
    scales = {n: st[n + "_scale"].double().clone() for n in "kv"}
    for s, kv in enumerate(held):
        pages, b = table[s], case["budget"]
        w = [weights[pages[j // PAGE]][j % PAGE] for j in range(kv)]
        if kv <= b:
            keep = list(range(kv))
        else:
            last = min(case["last"], b)
            first = min(case["first"], b - last)
            middle = sorted(range(first, kv - last), key=lambda j: (-w[j], j))[:b - first - last]
            keep = sorted(list(range(first)) + middle + list(range(kv - last, kv)))
        for i, j in enumerate(keep):
            got[(pages[i // PAGE], i % PAGE)] = w[j]
        for n in "kv" if kv > b else "":
            for d in range(0, len(keep), PAGE):
                src = torch.tensor([pages[j // PAGE] * PAGE + j % PAGE for j in keep[d:d + PAGE]], device="cuda")
                old = scales[n][:, src // PAGE]                                        # [layers][positions][heads]
                unit = old.amax(1)
                x = values[n][:, src // PAGE, :, src % PAGE].double()                  # [positions][layers][heads][dim]
                x = _exact_round(x * (old / unit[:, None]).transpose(0, 1)[..., None])
                values[n][:, pages[d // PAGE], :, :len(src)] = x.permute(1, 2, 0, 3).float()
                scales[n][:, pages[d // PAGE]] = unit
    at = torch.tensor([p * PAGE + i for p, i in got], device="cuda")
    out.view(-1)[at] = torch.tensor(list(got.values()), dtype=torch.float64, device="cuda")
    return {"k": values["k"], "v": values["v"], "k_scale": scales["k"], "v_scale": scales["v"], "weights_out": out}


def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None          # tokens and counts alone
    st = prepare(case, seed)
    if op == "probs":
        return _exact_probs(st)
    if op == "weigh":
        return _exact_weigh(st)
    _, held = _lengths(case)
    table = st["table"].tolist()
    if op == "step":
        # what the verification leaves: drafts kept one by one
        start, ids, u = st["row_start"].tolist(), st["ids"].tolist(), st["uniform"].tolist()
        for s in range(case["seqs"]):
            r, stop = start[s] + 1, start[s + 1]
            while r < stop and u[r] * (float(st["draft_probs"][r, ids[r]]) if st["draft_probs"] is not None else 1.0) \
                    < float(st["probs"][r - 1, ids[r]]):
                r += 1
            held[s] -= stop - r
    return _exact_evict(st, held, table)
