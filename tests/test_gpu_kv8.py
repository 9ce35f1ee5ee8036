"""The 8-bit paged cache's operators on the GPU against their plain 64-bit
definitions (tests/kv8_plain.py).

Tolerances.
* Page plans, codes and scales: equal (scales are powers of two, so every
  value the append rounds is exact in fp32).
* Rotary positions: the angle is off by at most 2^-26 turns * 2 pi (the
  turn's fp32 rounding) plus the frequency
  table's 2^-53 relative, sine and cosine by 2 ulp of fp32 at most, products
  and sums by 3 roundings: |x|max * scale * (2 pi 2^-25 + 8 * 2^-24) for the
  pair, then half a step of the type.
* Attention.  A score is off by d = (dim + 10) 2^-24 sum |q k| scale (fp32
  accumulation of dim exact products, the factor, the running maximum) and by
  2^-25 max|q| sum |k| scale (elements of q 2^-14 below the row's largest,
  held as f16); ex2 by 2^-22.  A weight is therefore off by d' = d + 2^-22,
  relative; with P rounded to f16 (2^-11 relative, or 2^-25 of the largest
  weight per key where it is subnormal) an output is off by at most
  mag (2^-11 + 2 d' + 2^-20) + unit 2^-25, then half a step of its type;
  the log of the sum by d' + 2^-22 (1 + |lse|).
"""

import math

import numpy as np
import pytest
import torch

from tests import gpu_common as G
from tests import kv8_plain as P

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def capi():
    G.build_lib()
    from block_diffusion_speculative_gather_gb300 import capi as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def half_step(t):
    return torch.finfo(t).eps / 2


# ------------------------------------------------------------------ pages

def run_plan(capi, kv, q, free, n_free, table, rows, alias=False):
    S = len(kv)
    kv_t, n_t, tab = ints(kv), ints([n_free]), ints(table)
    after = kv_t if alias else ints([-7] * S)
    n_out = n_t if alias else ints([-7])
    start, pos, slot = ints([-7] * (S + 1)), ints([-7] * rows), ints([-7] * rows)
    capi.dflash_pages_plan(kv_t, ints(q), ints(free), n_t, tab, start, pos, slot, after, n_out)
    return (tab.tolist(), start.tolist(), pos.tolist(), slot.tolist(), after.tolist(), n_out.item())


def plan_case(seed, S, width, most, short=0):
    g = np.random.default_rng(seed)
    kv = g.integers(0, (width - 2) * 64, S).tolist()
    q = g.integers(0, most + 1, S).tolist()
    used = sum(-(-k // 64) for k in kv)
    need = sum(-(-(k + n) // 64) for k, n in zip(kv, q)) - used
    order = g.permutation(used + need + 5).tolist()
    table, at = [], 0
    for k in kv:
        n = -(-k // 64)
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    free = order[at:]
    return kv, q, free + [-1] * used, max(0, len(free) - short), table


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("S,width,most,pad", [(1, 3, 1, 0), (1, 4, 90, 3), (33, 5, 70, 0), (300, 4, 3, 1000),
                                              (1025, 3, 9, 7), (2100, 3, 2, 4000), (40, 9, 300, 50)])
def test_plan(capi, S, width, most, pad, alias):
    kv, q, free, n, table = plan_case(S, S, width, most)
    rows = sum(q) + pad
    assert run_plan(capi, kv, q, free, n, table, rows, alias) == P.plan(kv, q, free, n, table, rows)


def test_plan_admits_in_order_while_pages_and_rows_last(capi):
    kv, q, free, n, table = plan_case(5, 50, 6, 100, short=20)
    rows = sum(q)
    assert run_plan(capi, kv, q, free, n, table, rows) == P.plan(kv, q, free, n, table, rows)
    kv, q, free, n, table = plan_case(6, 50, 6, 100)
    for rows in (0, 1, sum(q) // 2):
        assert run_plan(capi, kv, q, free, n, table, rows) == P.plan(kv, q, free, n, table, rows)


def test_plan_gives_invalid_lengths_nothing(capi):
    table = [[3, 4, -1]] * 5
    for kv, q in (([-1, 70, 70, 130, 128], [3, -2, 5, 63, 64]),
                  ([2**31 - 1, 0, 128, 0, 128], [2**31 - 1, 0, 1, 2**31 - 1, 65])):
        free = list(range(9))
        assert run_plan(capi, kv, q, free, 9, table, 200) == P.plan(kv, q, free, 9, table, 200)
    # a count beyond the list is cut to it; a negative one hands out nothing
    assert run_plan(capi, [0], [64], [5, 6], 9, [[-1]], 64)[0] == [[6]]
    assert run_plan(capi, [0], [64], [5, 6], -3, [[-1]], 64)[1] == [0, 0]


@pytest.mark.parametrize("S", [1, 40, 1500])
def test_trim_and_plan_again(capi, S):
    kv, q, free, n, table = plan_case(S + 1, S, 6, 60)
    free += [-1] * 8
    to = [k if i % 3 == 0 else (-5 if i % 3 == 1 else k // 2) for i, k in enumerate(kv)]
    kv_t, free_t, n_t, tab = ints(kv), ints(free), ints([n]), ints(table)
    capi.dflash_pages_trim(kv_t, ints(to), free_t, n_t, tab)
    want = P.trim(kv, to, free, n, table)
    assert (kv_t.tolist(), free_t.tolist(), n_t.item(), tab.tolist()) == want
    kv, free, n, table = want
    rows = sum(q)
    assert run_plan(capi, kv, q, free, n, table, rows) == P.plan(kv, q, free, n, table, rows)


def test_trim_never_writes_behind_the_list(capi):
    free, n, tab, kv = ints([1, 2, -9, -9]), ints([2]), ints([[5, 6, 7, 8]]), ints([256])
    capi.dflash_pages_trim(kv, ints([0]), free[:3], n, tab)
    assert free.tolist() == [1, 2, 8, -9] and n.item() == 3 and kv.item() == 0


# ------------------------------------------------------------------ rotary positions

ROPE = [
    # dim, rotary, interleaved, settings
    (128, 128, False, dict(theta=1e6)),
    (128, 64, True, dict(theta=1e6, scaling="parts", factor=32.0, original_len=32768, scale=1.25)),
    (64, 64, True, dict(theta=1e4, scaling="linear", factor=4.0)),
    (80, 40, False, dict(theta=1e4)),
    (96, 24, False, dict(theta=1e4)),          # 12 pairs: no 16-byte unit of 8
    (72, 6, True, dict(theta=1e4)),
    (256, 256, False, dict(theta=1e6)),
    (1024, 1024, True, dict(theta=1e6)),
    (2, 2, False, dict(theta=1e4)),
]


@pytest.mark.parametrize("kind", [BF, F16, F32])
@pytest.mark.parametrize("dim,rotary,il,w", ROPE)
def test_rope(capi, dim, rotary, il, w, kind):
    g = torch.Generator().manual_seed(dim + rotary)
    pos = torch.tensor([0, 1, 5, 63, -1, 4095, 131071, 10**6, 2**31 - 1], dtype=torch.int32)
    x = torch.randn(len(pos), 5, dim, generator=g).to(kind)
    k = torch.randn(len(pos), 2, dim, generator=g).to(kind)
    cfg = capi.rope_config(rotary, interleaved=il, **w)
    turns = torch.empty(rotary // 2, dtype=torch.int64, device="cuda")
    capi.dflash_rope_turns(cfg, turns)
    scale = w.get("scale", 1.0)
    freq = P.frequencies(rotary, **{n: v for n, v in w.items() if n != "scale"})
    outs = [torch.full_like(t, 9.0, device="cuda") for t in (x, k)]
    capi.dflash_rope(cfg, turns, pos.cuda(), x.cuda(), outs[0], k.cuda(), outs[1])
    for t, o in zip((x, k), outs):
        want = P.rope(t, pos, rotary, il, freq, scale)
        want[4] = 9.0                                   # a negative position: not written
        big = t.abs().max().double() * scale
        # the frequency's own 2^-52 relative, at the largest position
        far = 2 * math.pi * 2.0 ** -25 + 2.0 ** -52 * 2.0 ** 31
        tol = big * 2 * (far + 8 * 2.0 ** -24) + half_step(kind) * want.abs() + 2.0 ** -25
        err = (o.cpu().double() - want).abs()
        assert (err <= tol).all(), float((err / tol).max())
        assert torch.equal(o.cpu()[..., rotary:][pos >= 0], t[..., rotary:][pos >= 0])
    # in place, q alone, the same bits
    y = x.cuda()
    capi.dflash_rope(cfg, turns, pos.cuda(), y, y)
    ref = outs[0].clone()
    ref[4] = x[4].cuda()
    assert torch.equal(y, ref)


def test_rope_strided_misaligned_and_empty(capi):
    cfg = capi.rope_config(64)
    turns = torch.empty(32, dtype=torch.int64, device="cuda")
    capi.dflash_rope_turns(cfg, turns)
    pos = ints([3, 4000, 77])
    base = torch.randn(3, 7, 131, device="cuda").to(BF)
    x = base[:, 1:5, 2:130]                              # rows of 131, heads at odd addresses
    out = torch.full((4, 3, 128), 7.0, device="cuda", dtype=BF).permute(1, 0, 2)   # heads outermost
    capi.dflash_rope(cfg, turns, pos, x, out)
    want = P.rope(x.cpu(), pos.cpu(), 64, False, P.frequencies(64, 1e6))
    assert ((out.cpu().double() - want).abs() <= half_step(BF) * want.abs() + 1e-5).all()
    wide = torch.empty_like(x.contiguous())
    capi.dflash_rope(cfg, turns, pos, x.contiguous(), wide)
    assert torch.equal(wide, out.contiguous())           # the aligned form gives the same bits
    none = torch.empty((0, 4, 128), device="cuda", dtype=BF)
    capi.dflash_rope(cfg, turns, ints([]), none, none)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [1, 16, 700, 5000])
def test_rope_rows_do_not_depend_on_the_others(capi, rows):
    cfg = capi.rope_config(128)
    turns = torch.empty(64, dtype=torch.int64, device="cuda")
    capi.dflash_rope_turns(cfg, turns)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, 6, 128, device="cuda", generator=g).to(BF)
    pos = torch.randint(0, 1 << 20, (rows,), device="cuda", generator=g, dtype=torch.int32)
    out, one = torch.empty_like(x), torch.empty_like(x[:1])
    capi.dflash_rope(cfg, turns, pos, x, out)
    for r in {0, rows // 2, rows - 1}:
        capi.dflash_rope(cfg, turns, pos[r:r + 1].contiguous(), x[r:r + 1], one)
        assert torch.equal(one[0], out[r])


# ------------------------------------------------------------------ append

def pool(pages, n_kv, dim, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes = [(torch.randn(pages, n_kv, 64, dim, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
             .view(torch.uint8).cuda() for _ in range(2)]
    scale = [torch.exp2(torch.randint(-8, -5, (pages, n_kv), generator=g).float()).cuda() for _ in range(2)]
    return codes + scale


def values(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def check_append(capi, k, v, slots, cache, err_want=(0, 0)):
    want = [(values(cache[i]).numpy().copy(), cache[2 + i].cpu().double().numpy().copy()) for i in range(2)]
    err = ints([0, 0])
    capi.dflash_kv8_append(k, v, ints(slots), *cache, err)
    assert tuple(err.tolist()) == err_want
    for i, x in enumerate((k, v)):
        vals, sc = want[i]
        P.append(x.cpu().double().numpy(), slots, vals, sc)
        assert np.array_equal(cache[2 + i].cpu().double().numpy(), sc)
        assert np.array_equal(values(cache[i]).numpy(), vals, equal_nan=True)


RUNS = {
    "one": [5],
    "page": list(range(128, 192)),
    "crossing": list(range(100, 300)),
    "decode": [63, 64 * 3 + 1, 64 * 5, 64 * 7 + 62, 64 * 9 + 33],
    "skips": [-1, 70, 71, -1, 73, -1, -1, 200, 201, -5],
    "first": [0, 1, 2],
    "repeats": [70, 70, 70, 75, 74, 64, 65, 64, -1, 64, 64 * 3 + 1, 64 * 3 + 1] + [64 * 5 + 9] * 150,
    "far apart": [130] + [-1] * 200 + [131, 130] + [-1] * 130 + [64 * 4],
    "many": [64 * i + (i * 7) % 64 for i in range(300)],        # 300 pages, a row each
    "prompts": list(range(64 * 3 + 17, 64 * 3 + 17 + 333)) + list(range(64 * 20, 64 * 20 + 130)),
    "mixed": [64 * 60 + i for i in range(64)] + [64 * (70 + i) + i for i in range(50)] +
             list(range(64 * 130 + 3, 64 * 133)) + [-1] * 9 + list(range(64 * 140, 64 * 141 + 1)),
}


@pytest.mark.parametrize("kind", [BF, F16, F32])
@pytest.mark.parametrize("dim,n_kv", [(128, 2), (64, 3)])
@pytest.mark.parametrize("runs", sorted(RUNS))
def test_append(capi, runs, dim, n_kv, kind):
    slots = RUNS[runs]
    cache = pool(max(8, max(slots) // 64 + 2), n_kv, dim, seed=len(slots))
    g = torch.Generator().manual_seed(7)
    kv = torch.randn(2, len(slots), n_kv, dim, generator=g) * torch.exp(torch.randn(len(slots), 1, 1, generator=g))
    k, v = (t.to(kind).cuda() for t in kv)
    check_append(capi, k, v, slots, cache)


def test_append_extremes(capi):
    """Rows of zeros, infinities, NaN, the type's largest and smallest values;
    a scale that grows past the codes' range and one that starts anew."""
    rows = torch.zeros(8, 1, 64)
    rows[1] = torch.linspace(-3e38, 3e38, 64)
    rows[2, 0, 3] = math.inf
    rows[3, 0, :4] = torch.tensor([math.nan, 1.0, -math.inf, -2.0])
    rows[4] = 1e-40
    rows[5] = 448.0
    rows[6, 0, 0] = 448.0001
    rows[7] = torch.linspace(0, 2.0 ** -9, 64)
    for kind in (F32, BF):
        for r in range(8):
            for slot in (64, 64 + 20):                     # a fresh page; behind 20 tokens
                cache = pool(3, 1, 64)
                x = rows[r:r + 1].to(kind).cuda()
                check_append(capi, x, -x, [slot], cache)
    cache = pool(3, 1, 64)
    for i, top in enumerate((1e-20, 1.0, 1e20, 3.0, 1e30)):   # the scale only grows inside a page ...
        x = torch.full((1, 1, 64), top).cuda()
        check_append(capi, x, x, [64 + i], cache)
    check_append(capi, torch.ones(1, 1, 64).cuda(), torch.ones(1, 1, 64).cuda(), [64], cache)
    assert cache[2][1, 0].item() == 2.0 ** -8                 # ... and starts again with it


def test_append_strides_alignment_and_other_layouts(capi):
    slots = list(range(70, 170)) + [-1, 3]
    n = len(slots)
    g = torch.Generator().manual_seed(1)
    big = torch.randn(n, 11, 130, generator=g).to(BF).cuda()
    check_append(capi, big[:, 1:3, 1:129], big[:, 5:7, 2:130], slots, pool(4, 2, 128))   # odd addresses
    fused = torch.randn(n, 2, 2, 128, generator=g).to(F16).cuda()
    check_append(capi, fused[:, 0], fused[:, 1], slots, pool(4, 2, 128))                 # one projection's rows
    run = torch.randn(2, 2, 256, 64, generator=g).to(F16).cuda()                         # [heads][positions]: a context's cache
    check_append(capi, run[0].transpose(0, 1)[:n], run[1].transpose(0, 1)[:n], slots, pool(4, 2, 64))
    one = torch.randn(1, 2, 128, generator=g).cuda().expand(n, 2, 128)                   # a broadcast row
    check_append(capi, one, one, slots, pool(4, 2, 128))


def test_append_reports_a_slot_outside_the_pool(capi):
    x = torch.randn(4, 2, 64).cuda()
    err, cache = ints([0, 0]), pool(3, 2, 64)
    before = [t.clone() for t in cache]
    capi.dflash_kv8_append(x, x, ints([64 * 3, 2**31 - 1, -1, -(2**31)]), *cache, err)
    assert err.tolist()[0] == 2 and err.tolist()[1] in (0, 1)
    assert all(torch.equal(a, b) for a, b in zip(before, cache))
    capi.dflash_kv8_append(x[:0], x[:0], ints([]), *cache, err)
    assert all(torch.equal(a, b) for a, b in zip(before, cache))


# ------------------------------------------------------------------ attention

def attn_state(n_q, n_kv, dim, rows, held, kind, seed=0, pad=2, q_scale=1.5, width=None):
    """Everything a call takes: the pool's pages shuffled among the sequences,
    stale codes (NaN among them) behind every sequence's length."""
    g = torch.Generator().manual_seed(seed)
    S = len(rows)
    need = [-(-kv // 64) for kv in held]
    pages = sum(need) + 3
    kc, vc, ks, vs = pool(pages, n_kv, dim, seed)
    order = torch.randperm(pages, generator=g).tolist()
    width = width or max(max(need), 1) + 1
    table, at = [], 0
    for n, kv in zip(need, held):
        own = order[at:at + n]
        table.append(own + [-1] * (width - n))
        at += n
        if n and kv % 64:
            for c in (kc, vc):
                c[own[-1], :, kv % 64:] = torch.randint(0, 256, (n_kv, 64 - kv % 64, dim), generator=g).to(torch.uint8).cuda()
                c[own[-1], :, kv % 64:, :3] = 0x7f
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    total = start[-1] + pad
    q = (q_scale * torch.randn(total, n_q, dim, generator=g)).to(kind).cuda()
    return dict(q=q, cache=[kc, vc, ks, vs], table=table, held=held, start=start,
                out=torch.full((total, n_q, dim), 3.0, dtype=kind, device="cuda"),
                lse=torch.full((total, n_q), 3.0, device="cuda"))


def attend(capi, st, causal=True, window=0, scale=None, lse=True, workspace=None, stream=None, want_err=(0, 0)):
    q, table = st["q"], ints(st["table"])
    S, width = table.shape
    rows, n_q, dim = q.shape
    if workspace is None:
        n = capi.dflash_kv8_workspace_bytes(rows, S, n_q, st["cache"][0].shape[1], dim, width)
        workspace = torch.zeros(n, dtype=torch.uint8, device="cuda")
    err = ints([0, 0])
    args = (ints(st["held"]), ints(st["start"]))
    capi.dflash_kv8_attention(q, *st["cache"], table, *args, st["out"], workspace, err,
                              lse=st["lse"] if lse else None, scale=scale, causal=causal, window=window,
                              stream=stream)
    torch.cuda.synchronize()
    assert tuple(err.tolist()) == want_err
    return workspace


def check_attend(st, causal=True, window=0, scale=None):
    q = st["q"].cpu().double()
    rows, n_q, dim = q.shape
    kind = st["q"].dtype
    scale = dim ** -0.5 if scale is None else scale
    kc, vc = (values(c) for c in st["cache"][:2])
    ks, vs = (s.cpu().double() for s in st["cache"][2:])
    r = P.attend(q, kc, vc, ks, vs, st["table"], st["held"], st["start"], causal, window, scale)
    out, lse = st["out"].cpu().double(), st["lse"].cpu().double()
    n = st["start"][-1]
    assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()      # rows behind the last sequence
    d = (dim + 10) * 2.0 ** -24 * r["terms"] + 2.0 ** -25 * r["qabs"] + 2.0 ** -22
    tol = r["mag"] * (2.0 ** -11 + 2 * d[..., None] + 2.0 ** -20) + r["unit"] * 2.0 ** -25
    tol = tol * (1 + half_step(kind)) + half_step(kind) * r["out"].abs() + 2.0 ** -25
    e = (out - r["out"]).abs()[:n]
    assert (e <= tol[:n]).all(), (float((e / tol[:n]).nan_to_num(9e9).max()), e.max())
    empty = torch.isinf(r["lse"][:n])
    assert torch.equal(torch.isinf(lse[:n]), empty)
    assert (lse[:n][empty] == -math.inf).all() and (out[:n][empty] == 0).all()
    le = (lse - r["lse"]).abs()[:n][~empty]
    lt = (d + 2.0 ** -22 * (1 + r["lse"].abs()))[:n][~empty]
    assert (le <= lt).all(), float((le / lt).max())
    return float((e / tol[:n].clamp(min=1e-300)).max())


SHAPES = [
    # n_q, n_kv, dim, rows, held
    (1, 1, 64, [1], [1]),
    (4, 1, 128, [1], [64]),
    (8, 2, 128, [1], [65]),
    (8, 2, 64, [1, 1, 1], [1, 63, 700]),
    (32, 8, 128, [1], [1088]),
    (5, 1, 64, [3, 1, 2], [3, 130, 64]),
    (14, 2, 128, [4, 16], [300, 16]),
    (16, 1, 64, [16, 7], [200, 129]),
    (32, 2, 128, [2, 3], [100, 513]),
    (3, 3, 128, [16, 0, 5, 0], [128, 50, 5, 0]),
    (6, 2, 64, [40, 17, 1], [100, 17, 2000]),
    (4, 2, 128, [130], [200]),
    (8, 2, 128, [70, 33, 129], [70, 400, 130]),
]


@pytest.mark.parametrize("kind", [BF, F16])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0), (False, 64), (True, 1)])
@pytest.mark.parametrize("n_q,n_kv,dim,rows,held", SHAPES)
def test_attention(capi, n_q, n_kv, dim, rows, held, causal, window, kind):
    st = attn_state(n_q, n_kv, dim, rows, held, kind, seed=sum(held))
    ws = attend(capi, st, causal, window)
    check_attend(st, causal, window)
    first = st["out"].clone(), st["lse"].clone()
    st["out"].fill_(3.0), st["lse"].fill_(3.0)
    attend(capi, st, causal, window, workspace=ws)                # the workspace is as it was: the same bits
    assert torch.equal(first[0], st["out"]) and torch.equal(first[1], st["lse"])


@pytest.mark.parametrize("rows,held", [([1], [9000]), ([16], [6000]), ([1] * 7, [1, 4000, 64, 0, 2500, 128, 1]),
                                       ([64], [3000])])
def test_attention_long_caches(capi, rows, held):
    st = attn_state(4, 1, 128, rows, held, BF, seed=3)
    attend(capi, st)
    check_attend(st)


def test_attention_rows_without_keys(capi):
    """A sequence shorter than its rows (its first rows have negative
    positions), an empty one, and a window of nothing but the row itself."""
    for n in (1, 16, 90):
        st = attn_state(8, 2, 64, [n, 3, 2], [max(0, n - 5), 0, 70], BF, seed=n)
        attend(capi, st)
        check_attend(st)
        attend(capi, st, causal=False)
        check_attend(st, causal=False)


def test_attention_strides_scale_and_no_lse(capi):
    st = attn_state(8, 2, 128, [5, 20], [90, 20], F16, seed=2)
    total = st["q"].shape[0]
    q = torch.zeros(total, 12, 192, dtype=F16, device="cuda")[:, 2:10, 32:160]
    q.copy_(st["q"])
    out = torch.full((8, total, 136), 3.0, dtype=F16, device="cuda").transpose(0, 1)[..., :128]
    plain = dict(st)
    attend(capi, plain, scale=0.05)
    check_attend(plain, scale=0.05)
    lse = st["lse"].clone()
    st = {**st, "q": q, "out": out}
    st["lse"].fill_(3.0)
    attend(capi, st, scale=0.05, lse=False)
    assert torch.equal(st["out"], plain["out"]) and (st["lse"] == 3.0).all() and not torch.equal(lse, st["lse"])


def test_attention_scales_far_apart(capi):
    """Pages whose K and V scales differ by many powers of two, large and
    small q rows: weights stay within f16 whatever the scales."""
    st = attn_state(4, 1, 64, [3], [300], BF, seed=4, q_scale=1.0)
    ks, vs = st["cache"][2:]
    pages = st["table"][0][:5]
    for i, p in enumerate(pages):
        ks[p] = 2.0 ** (-8 - 2 * i)
        vs[p] = 2.0 ** (20 - 11 * i)
    st["q"][0] *= 2.0 ** -60
    st["q"][1, :, ::2] *= 2.0 ** -20
    attend(capi, st)
    check_attend(st)


def test_attention_sequences_do_not_depend_on_each_other(capi):
    """The same sequence among others of other lengths and contents: the same
    bits (row, sequence and head counts being the same)."""
    for rows in ([1, 1, 1], [16, 16, 16], [40, 40, 40]):
        outs = []
        for others in ([100, 3000], [2000, 64]):
            held = [others[0], 777, others[1]]
            st = attn_state(8, 2, 128, rows, held, BF, seed=9)
            alone = attn_state(8, 2, 128, [rows[1]], [777], BF, seed=10)
            for c, a in zip(st["cache"], alone["cache"]):
                for i, p in enumerate(alone["table"][0][:13]):
                    c[st["table"][1][i]] = a[p]
            st["q"][rows[0]:2 * rows[0]] = alone["q"][:rows[1]]
            attend(capi, st)
            outs.append((st["out"][rows[0]:2 * rows[0]].clone(), st["lse"][rows[0]:2 * rows[0]].clone()))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_attention_many_sequences(capi):
    g = np.random.default_rng(1)
    held = g.integers(1, 200, 300).tolist()
    st = attn_state(4, 2, 64, [1] * 300, held, BF, seed=5, pad=0)
    attend(capi, st)
    check_attend(st)


def test_attention_impossible_lengths_and_pages_are_reported(capi):
    """An impossible length or page sets err and is left out; the other
    sequences are right and nothing outside the buffers is touched."""
    st = attn_state(4, 2, 64, [2, 1, 3], [100, 64, 200], BF, seed=6)
    good = {**st, "out": st["out"].clone(), "lse": st["lse"].clone()}
    attend(capi, good)
    for held in ([100, 10**6, 200], [100, -1, 200]):
        bad = {**st, "held": held, "out": st["out"].clone(), "lse": st["lse"].clone()}
        attend(capi, bad, want_err=(2, 304))
        assert torch.equal(bad["out"][:2], good["out"][:2]) and torch.equal(bad["out"][3:6], good["out"][3:6])
        assert (bad["out"][2] == 3.0).all()
    for page in (-1, 10**6, -(2**31)):
        table = [list(t) for t in st["table"]]
        table[2][1] = page
        bad = {**st, "table": table, "out": st["out"].clone(), "lse": st["lse"].clone()}
        attend(capi, bad, want_err=(2, 303))
        assert torch.equal(bad["out"][:3], good["out"][:3])
        # its keys are left out: as if they were masked
        assert torch.isfinite(bad["out"].float()).all()
    start = [0, 2, 1, 6]                                           # not increasing
    bad = {**st, "start": start, "out": st["out"].clone(), "lse": st["lse"].clone()}
    attend(capi, bad, want_err=(2, 304))
    assert torch.equal(bad["out"][:1], good["out"][:1])


def test_attention_refuses_a_small_workspace(capi):
    st = attn_state(4, 2, 64, [2], [5000], BF)
    with pytest.raises(capi.DFlashError) as e:
        attend(capi, st, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert "workspace" in str(e.value)


def test_attention_nothing_to_do(capi):
    st = attn_state(4, 2, 64, [0, 0], [70, 0], BF, pad=3)
    attend(capi, st)
    assert (st["out"] == 3.0).all() and (st["lse"] == 3.0).all()


def test_attention_a_pool_past_4_gib(capi):
    """Offsets past 32 bits: pages at the far end of a pool of 4.4 GiB."""
    n_kv, dim = 8, 128
    pages = (1 << 32) // (n_kv * 64 * dim) + 4000
    if torch.cuda.mem_get_info()[0] < 3 * pages * n_kv * 64 * dim:
        pytest.skip("not enough device memory")
    small = attn_state(16, n_kv, dim, [1, 3], [130, 200], BF, seed=8)
    attend(capi, small)
    kc = torch.zeros((pages, n_kv, 64, dim), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    sc = [torch.ones((pages, n_kv), device="cuda") for _ in range(2)]
    table = [[-1 if p < 0 else pages - 1 - 7 * p for p in t] for t in small["table"]]
    big = {**small, "cache": [kc, vc] + sc, "table": table, "out": torch.full_like(small["out"], 3.0),
           "lse": torch.full_like(small["lse"], 3.0)}
    for t, u in zip(small["table"], table):
        for a, b in zip(t, u):
            if a >= 0:
                for c, s in zip(big["cache"], small["cache"]):
                    c[b] = s[a]
    attend(capi, big)
    assert torch.equal(big["out"], small["out"]) and torch.equal(big["lse"], small["lse"])
    x = torch.randn(70, n_kv, dim, device="cuda").to(BF)
    slots = list(range((pages - 2) * 64 + 5, (pages - 2) * 64 + 75))
    other = pool(2, n_kv, dim)
    for c, s in zip(big["cache"], other):
        c[pages - 2:] = s
    err = ints([0, 0])
    capi.dflash_kv8_append(x, x, ints(slots), *big["cache"], err)
    capi.dflash_kv8_append(x, x, ints([s - (pages - 2) * 64 for s in slots]), *other, err)
    assert err.tolist() == [0, 0]
    assert all(torch.equal(c[pages - 2:], s) for c, s in zip(big["cache"], other))


# ------------------------------------------------------------------ together

class Loop:
    """One layer of a serving loop on the operators: plan, rotate, append,
    attend; the state stays on the device."""

    def __init__(self, capi, S, width, pages, n_q, n_kv, dim, rows):
        self.capi, self.shape = capi, (n_q, n_kv, dim)
        self.kv, self.q_len = ints([0] * S), ints([0] * S)
        self.free, self.n_free = ints(list(range(pages))), ints([pages])
        self.table = ints([[-1] * width] * S)
        self.start, self.pos, self.slots = ints([0] * (S + 1)), ints([0] * rows), ints([0] * rows)
        self.cache = [torch.zeros((pages, n_kv, 64, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.cache += [torch.ones((pages, n_kv), device="cuda") for _ in range(2)]
        self.qkv = torch.zeros((rows, n_q + 2 * n_kv, dim), dtype=BF, device="cuda")
        self.rot = torch.zeros((rows, n_q + n_kv, dim), dtype=BF, device="cuda")
        self.out = torch.zeros((rows, n_q, dim), dtype=BF, device="cuda")
        self.lse = torch.zeros((rows, n_q), device="cuda")
        self.cfg = capi.rope_config(dim, theta=1e4)
        self.turns = torch.empty(dim // 2, dtype=torch.int64, device="cuda")
        capi.dflash_rope_turns(self.cfg, self.turns)
        self.err = ints([0, 0])
        self.ws = torch.zeros(capi.dflash_kv8_workspace_bytes(rows, S, n_q, n_kv, dim, width),
                              dtype=torch.uint8, device="cuda")

    def step(self):
        c, (n_q, n_kv, _) = self.capi, self.shape
        n = n_q + n_kv
        c.dflash_pages_plan(self.kv, self.q_len, self.free, self.n_free, self.table, self.start, self.pos,
                            self.slots, self.kv, self.n_free)
        c.dflash_rope(self.cfg, self.turns, self.pos, self.qkv[:, :n_q], self.rot[:, :n_q],
                      self.qkv[:, n_q:n], self.rot[:, n_q:])
        c.dflash_kv8_append(self.rot[:, n_q:], self.qkv[:, n:], self.slots, *self.cache, self.err)
        c.dflash_kv8_attention(self.rot[:, :n_q], *self.cache, self.table, self.kv, self.start, self.out,
                               self.ws, self.err, lse=self.lse)

    def state(self):
        n = self.start[-1].item()
        return [self.kv, self.table, self.n_free, self.pos, self.slots, self.out[:n], self.lse[:n],
                self.free[:self.n_free.item()]] + [t[:] for t in self.cache]


STEPS = [[40, 3, 0], [1, 70, 5], [16, 16, 16], [1, 1, 1], [0, 30, 16], [90, 0, 1]]


def feed(loop, i):
    g = torch.Generator(device="cuda").manual_seed(i)
    loop.qkv.copy_(torch.randn(loop.qkv.shape, generator=g, device="cuda"))
    loop.q_len.copy_(ints(STEPS[i % len(STEPS)]))


def test_a_run_of_steps_against_dense_attention(capi):
    """Six ragged steps with rows taken back between them: every step's
    outputs against dense attention over the tokens' own rotated K and V, as
    the definitions quantise them."""
    n_q, n_kv, dim, S = 8, 2, 64, 3
    loop = Loop(capi, S, 6, 18, n_q, n_kv, dim, 128)
    freq = P.frequencies(dim, 1e4)
    vals = [np.zeros((18, n_kv, 64, dim)) for _ in range(2)]
    scl = [np.ones((18, n_kv)) for _ in range(2)]
    for i in range(len(STEPS)):
        feed(loop, i)
        before = (loop.kv.tolist(), loop.free.tolist(), loop.n_free.item(), loop.table.tolist())
        loop.step()
        want = P.plan(before[0], STEPS[i], before[1], before[2], before[3], 128)
        assert (loop.table.tolist(), loop.start.tolist(), loop.pos.tolist(), loop.slots.tolist(),
                loop.kv.tolist(), loop.n_free.item()) == want
        rot = loop.rot.cpu()
        pos = loop.pos.cpu()
        ref = P.rope(loop.qkv[:, :n_q + n_kv].cpu(), pos, dim, False, freq)
        ref = torch.where((pos >= 0)[:, None, None], ref, rot.double())
        assert ((rot.double() - ref).abs() <= half_step(BF) * ref.abs() + 1e-5).all()
        # from here the GPU's own rotated rows: their rounding is checked above
        for which, x in enumerate((rot[:, n_q:], loop.qkv[:, n_q + n_kv:].cpu())):
            P.append(x.double().numpy(), want[3], vals[which], scl[which])
            assert np.array_equal(values(loop.cache[which]).numpy(), vals[which])
            assert np.array_equal(loop.cache[2 + which].cpu().double().numpy(), scl[which])
        n = want[1][-1]
        st = dict(q=loop.rot[:n, :n_q], cache=loop.cache, table=want[0], held=want[4], start=want[1],
                  out=loop.out[:n], lse=loop.lse[:n])
        check_attend(st)
        # a verify's rejected rows: back to two thirds
        to = [k - k // 3 for k in want[4]]
        capi.dflash_pages_trim(loop.kv, ints(to), loop.free, loop.n_free, loop.table)
    assert loop.err.tolist() == [0, 0]


def test_captured_steps_advance_like_eager_ones(capi):
    """A graph of one step, replayed while an eager loop runs the same steps;
    and two graphs over one workspace, replayed in turn."""
    eager, cap = (Loop(capi, 3, 8, 24, 8, 2, 128, 160) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            cap.step()
        graphs.append(g)
    for i in range(5):
        feed(eager, i)
        eager.step()
        feed(cap, i)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.state(), cap.state()):
            assert torch.equal(a, b)
    assert cap.err.tolist() == [0, 0]


def test_another_stream(capi):
    st = attn_state(8, 2, 128, [16, 1], [500, 900], BF, seed=1)
    attend(capi, st)
    want = st["out"].clone(), st["lse"].clone()
    st["out"].fill_(3.0), st["lse"].fill_(3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    attend(capi, st, stream=s)
    assert torch.equal(want[0], st["out"]) and torch.equal(want[1], st["lse"])
    with torch.cuda.stream(s):
        st["out"].fill_(3.0)
        attend(capi, st)
    assert torch.equal(want[0], st["out"])


def test_two_calls_at_once_with_their_own_workspaces(capi):
    a = attn_state(8, 2, 128, [16] * 4, [3000] * 4, BF, seed=1)
    b = attn_state(8, 2, 128, [1] * 9, [2500] * 9, BF, seed=2)
    wa, wb = attend(capi, a), attend(capi, b)
    want = a["out"].clone(), b["out"].clone()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for x in (s, t):
        x.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        err = ints([0, 0])
        torch.cuda.synchronize()
        for st, ws, x in ((a, wa, s), (b, wb, t)):
            with torch.cuda.stream(x):
                capi.dflash_kv8_attention(st["q"], *st["cache"], ints(st["table"]), ints(st["held"]),
                                          ints(st["start"]), st["out"], ws, err, lse=st["lse"])
        torch.cuda.synchronize()
        assert err.tolist() == [0, 0]
        assert torch.equal(a["out"], want[0]) and torch.equal(b["out"], want[1])


@pytest.mark.parametrize("n_q,rows,keys,dim", [(8, [16] * 4, [3000] * 4, 128),             # 64 packed rows
                                               (8, [32] * 3, [2100] * 3, 128),             # 128
                                               (8, [70, 33, 129], [2000, 1400, 1130], 128),
                                               (8, [1] * 9, [2500] * 9, 128),
                                               (10, [16] * 12, [1500] * 12, 64)])
def test_repeats_have_the_same_bits(capi, n_q, rows, keys, dim):
    # pages are overwritten in shared memory as soon as they are given back
    st = attn_state(n_q, 2, dim, rows, keys, BF, seed=3)
    ws = attend(capi, st)
    want, lse, err = st["out"].clone(), st["lse"].clone(), ints([0, 0])
    tabs = ints(st["table"]), ints(st["held"]), ints(st["start"])
    other = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(400):
        st["out"].fill_(3.0)
        capi.dflash_kv8_attention(st["q"], *st["cache"], *tabs, st["out"], ws, err, lse=st["lse"])
        other |= (st["out"] != want).any() | (st["lse"] != lse).any()
    assert err.tolist() == [0, 0] and not other.item()


def seen_by(st, s, causal, window):
    """[rows of s][its keys]: which keys each row sees."""
    n, kv = st["start"][s + 1] - st["start"][s], st["held"][s]
    pos, key = kv - n + torch.arange(n)[:, None], torch.arange(kv)[None]
    if causal:
        see = key <= pos
        return see & (key > pos - window) if window else see
    see = torch.ones(n, kv, dtype=torch.bool)
    return see & (key >= kv - n - window) if window else see


@pytest.mark.parametrize("n_q,n_kv,dim,rows,held", [
    (4, 1, 128, [5, 3, 1], [300, 1000, 70]),           # 16-row tiles
    (4, 2, 64, [4, 8], [2000, 63]),
    (8, 2, 128, [16, 9], [1500, 64]),                  # 64-row tiles, rows held twice
    (8, 1, 64, [8, 8], [700, 129]),
    (8, 2, 128, [30, 20], [500, 2000]),                # 128-row tiles
    (6, 2, 64, [41, 1], [1000, 40]),
    (8, 2, 128, [150, 70], [400, 1000]),               # two 128-row tiles
    (4, 2, 64, [300], [310]),
])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 0), (False, 33)])
@pytest.mark.parametrize("where", ["v", "k", "q"])
def test_nan_stays_with_the_rows_that_see_it(capi, n_q, n_kv, dim, rows, held, causal, window, where):
    """Zeros in place of the NaNs must give the other rows the same bits."""
    st = attn_state(n_q, n_kv, dim, rows, held, BF, seed=9, pad=0)
    g = torch.Generator().manual_seed(1)
    bad = torch.zeros(st["q"].shape, dtype=torch.bool)      # results that are NaN
    spots, lost = [], []
    for s, kv in enumerate(held):
        see, r0, group = seen_by(st, s, causal, window), st["start"][s], n_q // n_kv
        edge = torch.nonzero(~see.all(0)).flatten().tolist()
        keys = sorted({kv - 1, max(kv - 2, 0), max(kv - 1 - window, 0), *([edge[0], edge[-1], edge[len(edge) // 2]] if edge else [])})
        for i, key in enumerate(keys):
            kh, d = i % n_kv, int(torch.randint(0, dim, (1,), generator=g))
            spots.append((st["table"][s][key // 64], kh, key % 64, d, 0x7f if i % 2 else 0xff))
            hit = torch.nonzero(see[:, key]).flatten()
            for r in hit.tolist():
                bad[r0 + r, kh * group:(kh + 1) * group, d if where == "v" else slice(None)] = True
        lost.append((r0 + rows[s] // 2, s % n_q))
    outs = []
    for nan in (False, True):
        if where == "q":
            for i, (r, h) in enumerate(lost):
                st["q"][r, h, 3 + i] = (math.nan if i % 2 else math.inf) if nan else 0.0
        else:
            for pg, kh, at, d, code in spots:
                st["cache"][where == "v"][pg, kh, at, d] = code if nan else 0
        attend(capi, st, causal, window)
        outs.append(st["out"].clone().cpu())
    if where == "q":
        bad[:] = False
        for r, h in lost:
            bad[r, h] = True
        assert torch.equal(outs[1][~bad], outs[0][~bad])
        return
    assert torch.equal(torch.isnan(outs[1]), bad)
    assert torch.equal(outs[1][~bad], outs[0][~bad])


@pytest.mark.parametrize("rows,held", [([3, 2], [2, 130]), ([20, 1], [7, 64]), ([200], [150])])
@pytest.mark.parametrize("causal", [True, False])
def test_largest_window_and_more_rows_than_positions(capi, rows, held, causal):
    st = attn_state(4, 1, 64, rows, held, BF, seed=4)
    attend(capi, st, causal, window=2 ** 31 - 1)
    check_attend(st, causal, window=2 ** 31 - 1)


def test_the_paged_cache_class_runs_the_operators(capi):
    """Two layers, three sequences, one of which does not fit at first: the
    class's outputs against dense attention over what it cached."""
    from block_diffusion_speculative_gather_gb300.runtime import PagedKV8
    n_q, n_kv, dim, S, rows = 8, 2, 128, 3, 96
    kv = PagedKV8(2, n_q, n_kv, dim, S, 5, 4, rows, rope=capi.rope_config(dim))
    g = torch.Generator(device="cuda").manual_seed(3)
    for q_len, given, back in (([70, 5, 200], [70, 5, 0], None), ([1, 16, 0], [1, 16, 0], [70, 12, 0]),
                               ([1, 1, 0], [1, 1, 0], [0, 13, 0]), ([0, 1, 80], [0, 1, 80], None)):
        had = kv.kv_len.tolist()
        kv.plan(q_len)
        start = kv.row_start.tolist()
        assert [b - a for a, b in zip(start, start[1:])] == given
        assert kv.kv_len.tolist() == [a + b for a, b in zip(had, given)]
        for layer in range(2):
            qkv = torch.randn((rows, n_q + 2 * n_kv, dim), generator=g, device="cuda").to(BF)
            q, k, v = qkv.split([n_q, n_kv, n_kv], 1)
            out, lse = torch.full_like(q, 3.0), torch.full((rows, n_q), 3.0, device="cuda")
            kv.rotate(q, k)
            assert kv.attend(layer, q, k, v, out=out, lse=lse, causal=layer == 0) is out
            check_attend(dict(q=q, cache=kv.caches[layer], table=kv.table.tolist(), held=kv.kv_len.tolist(),
                              start=start, out=out, lse=lse), causal=layer == 0)
        if back is not None:
            kv.trim(back)
    kv.check()
    assert kv.n_free.item() == 5 - 1 - 2
    kv.err.copy_(ints([2, 7]))
    with pytest.raises(capi.DFlashError):
        kv.check()
    kv.check()


@pytest.mark.parametrize("gap", [3, 31, 33, 70, 140, 700, 3000])
def test_append_over_long_gaps_of_skipped_rows(capi, gap):
    """Runs of one page with skipped rows between them, and a padded end."""
    skip = [-1] * gap
    slots = skip + [64, 65, 66] + skip + [67, 68] + skip + [69, -5, 70] + skip + [195, 196, 2, 3] + skip
    g = torch.Generator().manual_seed(gap)
    x = torch.randn(2, len(slots), 1, 64, generator=g) * torch.exp(3 * torch.randn(len(slots), 1, 1, generator=g))
    check_append(capi, x[0].to(BF).cuda(), x[1].to(BF).cuda(), slots, pool(4, 1, 64, seed=2))


@pytest.mark.parametrize("rows,held", [([2, 3, 1], [0, 0, 70]), ([20], [0]), ([160, 1], [0, 0])])
def test_sequences_without_positions(capi, rows, held):
    st = attn_state(4, 2, 64, rows, held, BF, seed=6)
    attend(capi, st)
    check_attend(st)


# Calls with enough heads or rows that larger tiles are chosen (152 SMs).
TILES = [
    # n_q, n_kv, dim, rows, held
    (32, 8, 128, [16], [300]),                              # 64 rows, held twice
    (40, 10, 64, [12, 3], [700, 65]),
    (8, 8, 64, [200], [260]),                               # several of 64
    (100, 20, 64, [16, 9], [700, 64]),                      # 128 rows
    (64, 16, 128, [30, 20, 5], [1000, 20, 333]),
    (16, 16, 128, [130], [200]),                            # several of 128
    (32, 16, 128, [90, 150, 130, 100, 70], [400, 150, 1000, 777, 64]),   # two tiles of 128
    (40, 20, 64, [300, 280], [310, 900]),
]


@pytest.mark.parametrize("n_q,n_kv,dim,rows,held", TILES)
@pytest.mark.parametrize("causal,window,kind", [(True, 0, BF), (True, 100, F16), (False, 0, F16), (False, 70, BF)])
def test_larger_tiles(capi, n_q, n_kv, dim, rows, held, causal, window, kind):
    st = attn_state(n_q, n_kv, dim, rows, held, kind, seed=12)
    attend(capi, st, causal, window)
    check_attend(st, causal, window)


@pytest.mark.parametrize("n_q,n_kv,dim,rows,held", TILES)
def test_larger_tiles_repeat_their_bits(capi, n_q, n_kv, dim, rows, held):
    st = attn_state(n_q, n_kv, dim, rows, [h + 900 for h in held], BF, seed=13)
    ws = attend(capi, st)
    want, lse, err = st["out"].clone(), st["lse"].clone(), ints([0, 0])
    tabs = ints(st["table"]), ints(st["held"]), ints(st["start"])
    other = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(200):
        st["out"].fill_(3.0)
        capi.dflash_kv8_attention(st["q"], *st["cache"], *tabs, st["out"], ws, err, lse=st["lse"])
        other |= (st["out"] != want).any() | (st["lse"] != lse).any()
    assert err.tolist() == [0, 0] and not other.item()


@pytest.mark.parametrize("n_q,n_kv,dim,rows,held", TILES)
@pytest.mark.parametrize("causal,window", [(True, 90), (False, 33)])
@pytest.mark.parametrize("where", ["v", "k"])
def test_larger_tiles_keep_nan_with_its_rows(capi, n_q, n_kv, dim, rows, held, causal, window, where):
    test_nan_stays_with_the_rows_that_see_it(capi, n_q, n_kv, dim, rows, held, causal, window, where)


@pytest.mark.parametrize("S", [33, 100, 1000, 4096])
def test_many_sequences(capi, S):
    """More sequences than a warp's lanes, lengths of zero among them."""
    g = torch.Generator().manual_seed(S)
    held = torch.randint(0, 200, (S,), generator=g).tolist()
    rows = [min(h, n) for h, n in zip(held, torch.randint(0, 4, (S,), generator=g).tolist())]
    st = attn_state(2, 1, 64, rows, held, BF, seed=S)
    ws = attend(capi, st)
    check_attend(st)
    first = st["out"].clone()
    attend(capi, st, workspace=ws)
    assert torch.equal(first, st["out"])


def test_one_workspace_for_calls_of_many_shapes(capi):
    """Counters stay apart from every shape's partial sums."""
    shapes = [(32, 8, 128, [1], [4000]), (8, 2, 128, [16] * 4, [3000] * 4), (16, 8, 64, [1] * 40, [9000] + [500] * 39),
              (8, 2, 128, [70, 33, 129], [2000, 1400, 1130]), (64, 16, 128, [30, 20, 5], [1000, 20, 333]),
              (8, 1, 64, [300], [5000]), (2, 1, 64, [1], [64])]
    states, size = [], 0
    for i, s in enumerate(shapes):
        st = attn_state(*s, BF, seed=i)
        ws = attend(capi, st)
        check_attend(st)
        states.append((st, st["out"].clone(), st["lse"].clone()))
        size = max(size, ws.numel())
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    order = [0, 1, 2, 3, 4, 5, 6, 5, 3, 1, 6, 4, 2, 0, 3, 0, 5, 1, 1, 2, 4]
    for i in order:
        st, out, lse = states[i]
        st["out"].fill_(3.0), st["lse"].fill_(3.0)
        attend(capi, st, workspace=ws)
        assert torch.equal(st["out"], out) and torch.equal(st["lse"], lse), i
