"""Attention over the 8-bit paged cache where its numbers spread far: scores
that rise by hundreds of powers of two, weights far below a row's largest, V
scales at both ends of their range, pages and scales that are not there, many
sequences; in each of the kernels' tile forms, against 64-bit definitions.

Tolerances are those stated in tests/test_gpu_kv8.py, but for the weights' f16
rounding: a weight is held relative to 2^-7 or less of the row's largest (weight *
V scale), so a small one is off by half a step, 2^-25, of that: 2^-32 a key
instead of 2^-25.  A sum of n weights is a
chain of at most n / 32 + 16 fp32 additions, each off by 2^-24 of it.  A score
is added to its page's log2 of the V scale and taken from a reference, two
roundings of 2^-24 of that sum: 2^-23 |log2 scale| beside the score's own.
"""

import math

import pytest
import torch

from tests.test_gpu_kv8 import BF, F16, attend, attn_state, capi, half_step, ints   # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

# n_q, n_kv, dim, rows: tiles of 16, 64, 128 and two times 128 packed rows (152 SMs)
FORMS = [
    (8, 2, 128, [1, 3]),
    (4, 2, 64, [7, 1]),
    (32, 8, 128, [16]),
    (40, 10, 64, [12, 3]),
    (64, 16, 128, [30, 20, 5]),
    (100, 20, 64, [16, 9]),
    (32, 16, 128, [80, 100, 90, 70, 80]),
    (40, 20, 64, [300, 280]),
    (16, 8, 64, [1] * 10),                 # 16, a sequence's pages in one item
]


def define(st, causal=True, window=0, scale=None, gone=()):
    """The definition in 64 bits, by whole matrices; the keys of pages in
    `gone` are masked.  Keys as in kv8_plain.attend."""
    q, dev = st["q"].double(), "cuda"
    kc, vc = (c.view(torch.float8_e4m3fn).double() for c in st["cache"][:2])
    k_scale, v_scale = (s.double() for s in st["cache"][2:])
    rows, n_q, dim = q.shape
    n_kv = kc.shape[1]
    group = n_q // n_kv
    scale = dim ** -0.5 if scale is None else scale
    kw = dict(dtype=torch.float64, device=dev)
    r = {"out": torch.zeros((rows, n_q, dim), **kw), "mag": torch.zeros((rows, n_q, dim), **kw),
         "lse": torch.full((rows, n_q), -math.inf, **kw), "unit": torch.zeros((rows, n_q, 1), **kw),
         "terms": torch.zeros((rows, n_q), **kw), "qabs": torch.zeros((rows, n_q), **kw),
         "chain": torch.zeros((rows, n_q), **kw), "far": torch.zeros((rows, n_q), **kw)}
    for s, kv in enumerate(st["held"]):
        r0, n = st["start"][s], st["start"][s + 1] - st["start"][s]
        if n == 0 or kv == 0:
            continue
        pages = torch.tensor(st["table"][s][:-(-kv // 64)], device=dev)
        there = torch.tensor([p not in gone for p in pages.tolist()], device=dev).repeat_interleave(64)[:kv]
        pages = pages.clamp(0, kc.shape[0] - 1)
        key, pos = torch.arange(kv, device=dev)[None], kv - n + torch.arange(n, device=dev)[:, None]
        see = (key <= pos if causal else key < kv) & there
        if window:
            see = see & (key > pos - window if causal else key >= kv - n - window)
        cached = lambda c, sc: (c[pages] * sc[pages][..., None, None]).transpose(0, 1).reshape(n_kv, -1, dim)[:, :kv]  # noqa: E731
        ks, vs = (torch.where(there[:, None], cached(c, x), 0.0) for c, x in ((kc, k_scale), (vc, v_scale)))
        sc = torch.where(there, v_scale[pages].repeat_interleave(64, 0)[:kv].T, 0.0)            # [n_kv][kv]
        qh = q[r0:r0 + n].view(n, n_kv, group, dim).permute(1, 2, 0, 3).reshape(n_kv, group * n, dim)
        hide = ~see.expand(n, kv).repeat(group, 1)
        x = (qh @ ks.mT * scale).masked_fill_(hide, -math.inf)
        w = torch.softmax(x, -1).nan_to_num_(0.0)                      # rows without keys: zeros

        def put(name, v):                                              # [n_kv][group * n]...
            r[name][r0:r0 + n] = v.unflatten(1, (group, n)).movedim(2, 0).flatten(1, 2)
        put("out", w @ vs)
        put("mag", w @ vs.abs())
        put("lse", torch.logsumexp(x, -1))
        put("unit", ((w * sc[:, None]).amax(-1) * 448 * (~hide).sum(-1))[..., None])
        put("terms", (qh.abs() @ ks.abs().mT).masked_fill_(hide, 0.0).amax(-1) * scale)
        put("qabs", qh.abs().amax(-1) * torch.where(see.any(0), ks.abs().sum(-1), 0.0).amax(-1, keepdim=True) * scale)
        put("far", torch.where(sc > 0, sc, 1.0).log2().abs().amax(-1, keepdim=True).expand(n_kv, group * n))
        r["chain"][r0:r0 + n] = kv / 32 + 16
    return r


def check(st, causal=True, window=0, scale=None, gone=()):
    r = define(st, causal, window, scale, gone)
    kind, dim, n = st["q"].dtype, st["q"].shape[2], st["start"][-1]
    out, lse = st["out"].double(), st["lse"].double()
    assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()          # rows behind the last sequence
    d = (dim + 10) * 2.0 ** -24 * r["terms"] + 2.0 ** -25 * r["qabs"] + 2.0 ** -22 + 2.0 ** -23 * r["far"]
    tol = r["mag"] * (2.0 ** -11 + 2 * d[..., None] + 2.0 ** -20) + r["unit"] * 2.0 ** -32
    tol = tol * (1 + half_step(kind)) + half_step(kind) * r["out"].abs() + 2.0 ** -25
    e = (out - r["out"]).abs()[:n]
    assert (e <= tol[:n]).all(), (float((e / tol[:n]).nan_to_num(9e9).max()), float(e.nan_to_num(9e9).max()))
    empty = torch.isinf(r["lse"][:n])
    assert torch.equal(torch.isinf(lse[:n]), empty)
    assert (lse[:n][empty] == -math.inf).all() and (out[:n][empty] == 0).all()
    le = (lse - r["lse"]).abs()[:n][~empty]
    lt = (d + 2.0 ** -22 * (1 + r["lse"].abs()) + 2.0 ** -24 * r["chain"])[:n][~empty]
    assert (le <= lt).all(), float((le / lt).max())


def codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def set_keys(st, level, bits, v=None, noise=0.05):
    """Scores of `bits` powers of two times level[key] of every sequence (and
    a little noise): dimension 0 of q is 16, of a key its level.  Values
    v[key] in every dimension where given (codes; scales stay).  Returns the
    softmax scale."""
    g = torch.Generator(device="cuda").manual_seed(5)
    q, (kc, vc, ks, _) = st["q"], st["cache"]
    q.copy_(noise * torch.randn(q.shape, generator=g, device="cuda"))
    q[..., 0] = 16.0
    ks.fill_(1.0)
    for s, kv in enumerate(st["held"]):
        pages = torch.tensor(st["table"][s][:-(-kv // 64)], device="cuda")
        n = 64 * len(pages)
        here = lambda x: torch.nn.functional.pad(x[:n].float().cuda(), (0, n - len(x[:n]))).view(-1, 1, 64)   # noqa: E731
        held = (torch.arange(n, device="cuda") < kv).view(-1, 1, 64, 1)
        k = 0.25 * torch.randn((len(pages), *kc.shape[1:]), generator=g, device="cuda")
        k[..., 0] = here(level)
        kc[pages] = torch.where(held, codes(k), kc[pages])
        if v is not None:
            vc[pages] = torch.where(held, codes(here(v)[..., None].expand_as(k)), vc[pages])
    return bits * math.log(2) / 16


# ------------------------------------------------------------------ scores that rise

# 32-key blocks before which scores rise: inside a page, between a step's
# pages, between steps; at an item's first step and behind it
RISES = [[1], [2], [4], [5, 9], [1, 2, 3, 6, 8, 12], [7, 16]]


@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
@pytest.mark.parametrize("bits", [3, 9, 20, 100, 130, 300])
def test_scores_that_rise(capi, n_q, n_kv, dim, rows, bits):       # noqa: F811
    """What came before weighs 2^-bits of what comes: below 2^-126 as nothing."""
    held = [max(n + 5, 700 + 37 * i) for i, n in enumerate(rows)]
    st = attn_state(n_q, n_kv, dim, rows, held, BF, seed=bits)
    for up in RISES:
        level = torch.zeros(max(held))
        for b in up:
            level[32 * b:] += 1
        scale = set_keys(st, level, bits)
        st["out"].fill_(3.0), st["lse"].fill_(3.0)
        attend(capi, st, scale=scale)
        check(st, scale=scale)
        attend(capi, st, causal=False, window=300, scale=scale)
        check(st, causal=False, window=300, scale=scale)


# ------------------------------------------------------------------ V scales far apart

@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
@pytest.mark.parametrize("e", [0, 27, 60, 119])
def test_pages_of_zeros_beside_large_ones(capi, n_q, n_kv, dim, rows, e):      # noqa: F811
    """Keys of pages whose values are zeros (V scale 2^-100) count in the sum
    like any others, whatever the other pages' scales; scores rise and fall."""
    held = [max(n + 5, 500 + 64 * i) for i, n in enumerate(rows)]
    st = attn_state(n_q, n_kv, dim, rows, held, BF, seed=e)
    v_codes = st["cache"][1].clone()
    for zeros in ([0], [1], [2, 4, 5], [-1]):
        for bits, ups in ((1, []), (40, [7]), (-20, [5, 8]), (-100, [4])):
            st["cache"][1].copy_(v_codes)
            st["out"].fill_(3.0), st["lse"].fill_(3.0)
            level = torch.zeros(max(held))
            for b in ups:
                level[32 * b:] += 1
            scale = set_keys(st, level, bits) * (1 if bits > 0 else -1)
            if bits < 0:
                st["q"][..., 0] = -16.0
            st["cache"][3].fill_(2.0 ** e)
            for s, t in enumerate(st["table"]):
                n = -(-held[s] // 64)
                for p in zeros:
                    st["cache"][1][t[p % n]] = 0
                    st["cache"][3][t[p % n]] = 2.0 ** -100
            attend(capi, st, scale=scale)
            check(st, scale=scale)


@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
@pytest.mark.parametrize("bits", [0, 13, 70, 200])
def test_v_scales_over_their_whole_range(capi, n_q, n_kv, dim, rows, bits):      # noqa: F811
    """Pages of all scales in turn, each larger one with the smaller weights."""
    held = [max(n + 5, 600 + 64 * i) for i, n in enumerate(rows)]
    st = attn_state(n_q, n_kv, dim, rows, held, BF, seed=bits)
    pages = -(-max(held) // 64)
    for scales in ((-100, 119), (119, -100), (-100, 0, 100), (60, -60), (-100,), (119,), (-50, -90, -10)):
        e = torch.tensor([scales[p % len(scales)] for p in range(pages)])
        order = torch.unique(e)
        level = -(e[:, None] == order).float().argmax(1).repeat_interleave(64).float()
        scale = set_keys(st, level, max(bits, 1))
        for s, t in enumerate(st["table"]):
            for p in range(-(-held[s] // 64)):
                st["cache"][3][t[p]] = 2.0 ** int(e[p])
        st["out"].fill_(3.0), st["lse"].fill_(3.0)
        attend(capi, st, scale=scale)
        check(st, scale=scale)


@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
def test_a_long_cache_of_zeros(capi, n_q, n_kv, dim, rows):      # noqa: F811
    """Values of zeros everywhere and scores that rise by less than a
    reference moves for: the sum stays within fp32."""
    rows = [min(rows[0], 40)]
    st = attn_state(n_q, n_kv, dim, rows, [40000], BF, seed=1)
    level = torch.ones(40000)
    level[:32] = 0
    st["cache"][1].zero_()
    st["cache"][3].fill_(2.0 ** -100)
    for bits in (3, 5.5, 13.9):
        scale = set_keys(st, level, bits, noise=0.01)
        attend(capi, st, scale=scale)
        check(st, scale=scale)


# ------------------------------------------------------------------ weights far below the largest

@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
@pytest.mark.parametrize("at", [0, 2990])
def test_a_long_tail_behind_one_key(capi, n_q, n_kv, dim, rows, at):      # noqa: F811
    """One key without values, of 2^bits the weight of each other one, in a
    page whose V scale is 2^above over the others': the values are the tail's."""
    held = [3000 + n for n in rows]
    st = attn_state(n_q, n_kv, dim, rows, held, F16, seed=at)
    for bits, above in ((15, 8), (17, 8), (20, 8), (12, 0), (22, 0)):
        level, v = torch.zeros(max(held)), torch.full((max(held),), 224.0)
        level[at] = 1.0
        v[64 * (at // 64):64 * (at // 64) + 64] = 224.0 * 2.0 ** -above
        v[at] = 0.0
        scale = set_keys(st, level, bits, v, noise=0.02)
        st["cache"][3].fill_(0.125)
        for t in st["table"]:
            st["cache"][3][t[at // 64]] = 0.125 * 2.0 ** above
        for causal in (True, False):
            st["out"].fill_(3.0), st["lse"].fill_(3.0)
            attend(capi, st, causal=causal, scale=scale)
            check(st, causal=causal, scale=scale)


# ------------------------------------------------------------------ pages and scales that are not there

GONE = [[0], [1], [0, 1], [2, 3], [3, 4], [5], [-1], list(range(64))]


def _spoil(st, which, change):
    """Applies change(table row, page index) to the pages `which` of every
    sequence and returns the page numbers as the table then has them."""
    gone = set()
    for s, t in enumerate(st["table"]):
        n = -(-st["held"][s] // 64)
        for p in {w % n for w in which if w < n}:
            change(t, p)
            gone.add(t[p])
    return gone


@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
@pytest.mark.parametrize("which", GONE)
def test_pages_that_are_not_there(capi, n_q, n_kv, dim, rows, which):      # noqa: F811
    """A page number out of range sets err; its keys are left out as if they
    were masked.  The codes that stand in shared memory instead are NaN."""
    held = [max(n + 5, 400 + 64 * i) for i, n in enumerate(rows)]
    st = attn_state(n_q, n_kv, dim, rows, held, BF, seed=3)
    stale = attn_state(n_q, n_kv, dim, rows, held, BF, seed=3)
    for c in stale["cache"][:2]:
        c.fill_(0x7f)
    pages = st["cache"][0].shape[0]
    for bad in (-1, pages, 2 ** 31 - 1, -(2 ** 31)):
        cut = {**st, "table": [list(t) for t in st["table"]]}

        def lose(t, p):
            t[p] = bad
        gone = _spoil(cut, which, lose)
        for causal, window in ((True, 0), (False, 0), (True, 130)):
            attend(capi, stale)                                        # fills the pages' places
            cut["out"].fill_(3.0), cut["lse"].fill_(3.0)
            # only pages that some row sees are looked up
            read = any(t[p] in gone for s, t in enumerate(cut["table"])
                       for p in range(max(0, held[s] - rows[s] + 1 - window) // 64 if window else 0, -(-held[s] // 64)))
            attend(capi, cut, causal, window, want_err=(2, 303) if read else (0, 0))
            check(cut, causal, window, gone=gone)


# ------------------------------------------------------------------ many sequences, far pools

@pytest.mark.parametrize("n_q,n_kv,dim,rows", [
    (8, 2, 64, [16] * 40),                                   # 64-row tiles
    (8, 1, 128, [5, 0, 8, 1] * 20 + [16]),
    (32, 2, 64, [8, 1, 16] * 15),                            # 128
    (8, 2, 64, [30, 40, 1] * 100),
    (4, 2, 64, [150, 40, 0] * 33 + [300]),                   # two times 128
])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 40)])
def test_larger_tiles_of_many_sequences(capi, n_q, n_kv, dim, rows, causal, window):      # noqa: F811
    """More sequences than a warp's lanes in the tcgen05 form."""
    g = torch.Generator().manual_seed(len(rows))
    past = torch.randint(0, 500, (len(rows),), generator=g).tolist()
    st = attn_state(n_q, n_kv, dim, rows, [n + p for n, p in zip(rows, past)], BF, seed=2, pad=0)
    ws = attend(capi, st, causal, window)
    check(st, causal, window)
    first = st["out"].clone(), st["lse"].clone()
    st["out"].fill_(3.0), st["lse"].fill_(3.0)
    attend(capi, st, causal, window, workspace=ws)
    assert torch.equal(first[0], st["out"]) and torch.equal(first[1], st["lse"])


def test_larger_tiles_over_a_pool_past_4_gib(capi):      # noqa: F811
    n_kv, dim = 8, 128
    pages = (1 << 32) // (n_kv * 64 * dim) + 4000
    if torch.cuda.mem_get_info()[0] < 3 * pages * n_kv * 64 * dim:
        pytest.skip("not enough device memory")
    kc = torch.zeros((pages, n_kv, 64, dim), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    sc = [torch.ones((pages, n_kv), device="cuda") for _ in range(2)]
    for rows in ([16] * 4, [40] * 6, [200] * 6):
        small = attn_state(32, n_kv, dim, rows, [260 + n for n in rows], BF, seed=8)
        attend(capi, small)
        check(small)
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


BAD_SCALES = [(3, 0.0), (3, -1.0), (3, math.nan), (3, math.inf), (2, -0.5), (2, math.nan), (2, math.inf)]


@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
@pytest.mark.parametrize("which", [[0], [1, 2], [5, 6, -1]])
def test_scales_that_no_append_writes(capi, n_q, n_kv, dim, rows, which):      # noqa: F811
    """A K scale that is negative, a V scale that is not above 0, one that is
    not finite: err, and the page's keys are left out."""
    held = [max(n + 5, 400 + 64 * i) for i, n in enumerate(rows)]
    st = attn_state(n_q, n_kv, dim, rows, held, BF, seed=4)
    good = st["cache"]
    for tensor, value in BAD_SCALES:
        bad = {**st, "cache": [c.clone() if i > 1 else c for i, c in enumerate(good)]}

        def spoil(t, p):
            bad["cache"][tensor][t[p]] = value
        gone = _spoil(bad, which, spoil)
        st["out"].fill_(3.0), st["lse"].fill_(3.0)
        attend(capi, bad, want_err=(2, 305))
        check(bad, gone=gone)


@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
def test_k_scales_of_zero(capi, n_q, n_kv, dim, rows):      # noqa: F811
    st = attn_state(n_q, n_kv, dim, rows, [max(n + 5, 300) for n in rows], BF, seed=4)
    for t in st["table"]:
        st["cache"][2][t[1]] = 0.0
    attend(capi, st)
    check(st)


# ------------------------------------------------------------------ row starts that overlap

@pytest.mark.parametrize("n_q,n_kv,dim,S,rows", [(8, 2, 64, 64, 96), (8, 2, 128, 40, 2000), (256, 256, 64, 4096, 65536)])
def test_overlapping_sequences_beyond_the_calls_rows(capi, n_q, n_kv, dim, S, rows):      # noqa: F811
    """Row starts 0, rows, 0, rows, ...: every other sequence claims all rows
    (at the largest more than 2^31 items).  err, and nothing is touched."""
    cache = [torch.zeros((2, n_kv, 64, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones((2, n_kv), device="cuda") for _ in range(2)]
    q = torch.zeros((rows, n_q, dim), dtype=BF, device="cuda")
    out, lse = torch.full_like(q, 3.0), torch.full((rows, n_q), 3.0, device="cuda")
    start = ints([0, rows] * (S // 2) + [0])
    ws = torch.zeros(capi.dflash_kv8_workspace_bytes(rows, S, n_q, n_kv, dim, 2), dtype=torch.uint8, device="cuda")
    err = ints([0, 0])
    capi.dflash_kv8_attention(q, *cache, ints([[0, 1]] * S), ints([100] * S), start, out, ws, err, lse=lse)
    assert err.tolist() == [2, 304]
    assert (out == 3.0).all() and (lse == 3.0).all() and (ws == 0).all()


# ------------------------------------------------------------------ rows and what they do not see

@pytest.mark.parametrize("n_q,n_kv,dim,rows", FORMS)
@pytest.mark.parametrize("window", [0, 200, 333])
def test_bits_do_not_follow_from_keys_a_row_does_not_see(capi, n_q, n_kv, dim, rows, window):      # noqa: F811
    """Scores rise by a few powers of two along the cache, so that references
    move; then the sequence's last key, which only the last row sees, and with
    a window the first row's first key, get scores of another size: the other
    rows keep their bits."""
    held = [max(n + 5, 900 + 50 * i) for i, n in enumerate(rows)]
    st = attn_state(n_q, n_kv, dim, rows, held, BF, seed=6)
    level = torch.arange(max(held)).float() / max(held)
    for bits in (6, 12, 25, 60):
        scale = set_keys(st, level, bits, noise=0.3)
        outs = []
        for odd in (0.0, 2.0, -2.0):
            for s, n in enumerate(rows):
                at = [held[s] - 1] + ([max(held[s] - n + 1 - window, 0)] if window and n > 1 else [])
                for key in at:
                    st["cache"][0][st["table"][s][key // 64], :, key % 64, 0] = codes(torch.tensor(odd, device="cuda"))
            attend(capi, st, window=window, scale=scale)
            outs.append((st["out"].clone(), st["lse"].clone()))
        keep = torch.ones(st["start"][-1], dtype=torch.bool)
        for s, n in enumerate(rows):
            keep[st["start"][s + 1] - 1] = False
            if window and held[s] - n + 1 > window:
                keep[st["start"][s]] = False
            elif window:
                keep[st["start"][s]:st["start"][s + 1]] = False
        keep = torch.nonzero(keep).flatten().cuda()
        for out, lse in outs[1:]:
            assert torch.equal(out[keep], outs[0][0][keep]) and torch.equal(lse[keep], outs[0][1][keep])


# ------------------------------------------------------------------ verify's schedule and single tokens'

@pytest.mark.parametrize("large", [1.0, 64.0, 2.0 ** 14])
@pytest.mark.parametrize("off", [0, 9])
def test_rejected_rows_leave_their_scale(capi, large, off):      # noqa: F811
    """A run of four rows of which the last, `large` times the others, is
    rejected, beside the first three appended one by one: each schedule's values
    are the rows' rounded to its scale, and the run's scale is the larger one."""
    g = torch.Generator().manual_seed(off)
    x = torch.randn(4, 2, 64, generator=g).cuda()
    x[3] *= large
    made = []
    for runs in ([range(4)], [[0], [1], [2]]):
        cache = [torch.zeros((2, 2, 64, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
        cache += [torch.full((2, 2), 2.0 ** -100, device="cuda") for _ in range(2)]
        err = ints([0, 0])
        for r in runs:
            rows = x[list(r)].contiguous()
            capi.dflash_kv8_append(rows, rows, ints([64 + off + i for i in r]), *cache, err)
        assert err.tolist() == [0, 0]
        sc = cache[2][1][None, :, None]
        made.append((cache[0][1, :, off:off + 3].view(torch.float8_e4m3fn).float().transpose(0, 1) * sc, cache[2][1].clone()))
        # later rows of the page can re-round earlier ones: twice half a step of the last scale
        assert ((made[-1][0] - x[:3]).abs() <= 2 * torch.maximum(x[:3].abs() * 2.0 ** -4, sc * 2.0 ** -10)).all()
    assert (made[0][1] >= made[1][1]).all()
    if large > 1:
        assert not torch.equal(made[0][1], made[1][1])
