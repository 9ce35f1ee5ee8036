"""Accumulated weights and eviction of the 8-bit paged cache on the GPU against
their plain 64-bit definitions (tests/sampling_plain.py).

Tolerances.
* Weights: a term exp(x - lse) is off by d relative, d made of the score's (dim
  + 10) 2^-24 sum |q k| scale and 2^-25 max|q| sum |k| scale (fp32 products
  and sums; elements of q far below the row's largest, held as f16), lse's 2^-23
  |lse| in base 2, the difference's 2^-24 (|x| + |lse|) and ex2's 2^-22; the sum
  of n terms by (n + 8) 2^-24 of itself.
* Codes, scales, chosen positions, lengths: equal (scales are powers of two).
"""

import math

import numpy as np
import pytest
import torch

from tests import gpu_common as G
from tests import kv8_plain as K
from tests import sampling_plain as P
from tests.test_gpu_kv8 import attend, attn_state, half_step, ints, pool, values

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def capi():
    G.build_lib()
    from block_diffusion_speculative_gather_gb300 import capi as m
    return m


# ------------------------------------------------------------------ weights

def weigh(capi, st, count=None, observe=0, fresh=False, causal=True, window=0, scale=None, seed=0, want_err=(0, 0),
          stream=None):
    """Runs the call; returns (weights before, after)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.rand(st["cache"][0].shape[0], 64, device="cuda", generator=g)
    before, err = w.clone(), ints([0, 0])
    capi.dflash_kv8_weigh(st["q"], st["lse"], *st["cache"], ints(st["table"]), ints(st["held"]), ints(st["start"]), w,
                          err, count=None if count is None else ints(count), observe=observe, fresh=fresh, scale=scale,
                          causal=causal, window=window, stream=stream)
    torch.cuda.synchronize()
    assert tuple(err.tolist()) == tuple(want_err)
    return before, w


def check_weigh(capi, st, **kw):
    before, w = weigh(capi, st, **kw)
    f = lambda t: t.double().cpu().numpy()      # noqa: E731
    kc = values(st["cache"][0]).numpy()
    args = {k: v for k, v in kw.items() if k in ("count", "observe", "fresh", "causal", "window")}
    dim = st["q"].shape[2]
    want, bound = P.weigh(f(st["q"]), f(st["lse"]), kc, f(st["cache"][2]), st["table"], st["held"], st["start"],
                          f(before), scale=kw.get("scale") or dim ** -0.5, **args)
    got = f(w)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    e = np.where(nan, 0.0, np.abs(got - want))
    b = np.where(nan, 0.0, bound)
    assert (e <= b).all(), (float((e / np.maximum(b, 1e-300)).max()), float(e.max()))
    return before, w


SHAPES = [
    # n_q, n_kv, dim, rows, held
    (1, 1, 64, [1], [1]),
    (4, 1, 128, [1], [64]),
    (8, 2, 128, [1], [65]),
    (8, 2, 64, [1, 1, 1], [1, 63, 300]),
    (32, 8, 128, [1], [200]),
    (5, 1, 64, [3, 1, 2], [3, 130, 64]),
    (14, 2, 128, [4, 16], [190, 16]),
    (16, 1, 64, [16, 7], [150, 129]),
    (3, 3, 128, [16, 0, 5, 0], [128, 50, 5, 0]),
    (4, 2, 128, [70], [140]),
    (12, 4, 64, [33, 1], [70, 257]),
    (20, 4, 128, [17, 2], [17, 66]),
    # many rows: the tcgen05 form, with groups that fill a tile and ones that do not
    (32, 8, 128, [64, 40], [300, 100]),
    (20, 4, 128, [64], [190]),
    (16, 1, 64, [33, 70], [200, 130]),
    (6, 2, 64, [70, 0, 3], [90, 64, 260]),
    (7, 1, 128, [129, 20, 64], [130, 20, 64]),
]


@pytest.mark.parametrize("kind", [BF, F16])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 40), (False, 0), (False, 30)])
@pytest.mark.parametrize("n_q,n_kv,dim,rows,held", SHAPES)
def test_weigh(capi, n_q, n_kv, dim, rows, held, causal, window, kind):
    st = attn_state(n_q, n_kv, dim, rows, held, kind, seed=len(held))
    attend(capi, st, causal=causal, window=window)
    check_weigh(capi, st, causal=causal, window=window, fresh=causal)


def test_weigh_many_rows_counted(capi):
    """The tcgen05 form: counted and observed rows, a window, sequences without rows."""
    st = attn_state(16, 4, 128, [90, 0, 64, 5, 33], [200, 70, 64, 300, 129], BF, seed=21)
    for kw in (dict(), dict(window=50)):
        attend(capi, st, **kw)
        for more in (dict(observe=32, fresh=True), dict(count=[0, 0, 40, 5, 33], fresh=True),
                     dict(count=[90, 9, 64, -1, 12], observe=20)):
            check_weigh(capi, st, **kw, **more)


def test_weigh_many_rows_strides_nan_and_pages(capi):
    st = attn_state(8, 2, 64, [64, 50], [140, 300], F16, seed=22)
    attend(capi, st)
    big = torch.full((st["q"].shape[0] + 3, 3, 8, 72), NAN, dtype=F16, device="cuda")
    view = big[1:-2, 1, :, :64]
    view.copy_(st["q"])
    st["q"] = view
    check_weigh(capi, st)
    st["q"][5] = NAN                                  # a row that adds nothing
    st["q"][9, :, 3] = INF
    st["lse"][5], st["lse"][9] = NAN, INF
    st["cache"][0][st["table"][1][1], 1, 5, 7] = 0x7f
    check_weigh(capi, st)
    _, good = weigh(capi, st)
    table = [list(t) for t in st["table"]]
    table[1][0] = -1
    _, w = weigh(capi, dict(st, table=table), want_err=(2, 303))
    for p in st["table"][0][:3] + st["table"][1][1:5]:
        assert torch.equal(w[p], good[p])
    _, w = weigh(capi, dict(st, held=[140, 10 ** 6]), want_err=(2, 304))
    assert torch.equal(w[st["table"][0][:3]], good[st["table"][0][:3]])
    st["cache"][2][st["table"][1][0], 0] = -1.0       # a scale that no append writes: nothing from that head
    _, w = weigh(capi, st, want_err=(2, 305))
    assert torch.equal(w[st["table"][1][1:5]], good[st["table"][1][1:5]])


@pytest.mark.parametrize("n_q,n_kv,dim,S,n,kv", [(32, 8, 128, 40, 16, 3000), (8, 8, 64, 9, 40, 5000), (40, 8, 128, 3, 200, 2000)])
def test_weigh_many_rows_repeat_their_bits(capi, n_q, n_kv, dim, S, n, kv):
    st = attn_state(n_q, n_kv, dim, [n - s % 3 for s in range(S)], [kv - 37 * s for s in range(S)], BF, seed=23)
    attend(capi, st)
    before, w = weigh(capi, st, fresh=True)
    for _ in range(10):
        assert torch.equal(weigh(capi, st, fresh=True)[1], w)
    for s in range(S):
        pages = st["table"][s][:-(-st["held"][s] // 64)]
        got = (w[pages].double().flatten()[:st["held"][s]].sum() -
               before[pages].double().flatten()[:st["held"][s] - (n - s % 3)].sum()).item()
        assert abs(got - (n - s % 3) * n_q) < (n - s % 3) * n_q * 1e-4


@pytest.mark.parametrize("count,observe,fresh", [([3, 0, 16, 1], 0, True), ([16, -4, 99, 2], 5, True), (None, 4, False),
                                                 ([0, 0, 0, 0], 3, True), (None, 1000, True)])
def test_weigh_counted_rows(capi, count, observe, fresh):
    st = attn_state(8, 2, 128, [16, 3, 16, 1], [100, 3, 130, 65], BF, seed=3)
    attend(capi, st)
    check_weigh(capi, st, count=count, observe=observe, fresh=fresh)


def test_weigh_sums_to_the_rows(capi):
    """Every counted row gives each of its heads' weight 1 in all."""
    st = attn_state(32, 8, 128, [16, 1, 64], [3000, 5000, 1500], BF, seed=5)
    attend(capi, st)
    before, w = weigh(capi, st)
    for s, (n, kv) in enumerate(zip([16, 1, 64], st["held"])):
        pages = st["table"][s][:-(-kv // 64)]
        got = (w - before)[pages].double().sum().item()
        assert abs(got - n * 32) < n * 32 * 1e-4
    others = [p for p in range(w.shape[0]) if p not in {x for t in st["table"] for x in t}]
    assert torch.equal(w[others], before[others])
    for s, kv in enumerate(st["held"]):           # positions behind the length
        if kv % 64:
            p = st["table"][s][kv // 64]
            assert torch.equal(w[p, kv % 64:], before[p, kv % 64:])


def test_weigh_strides_scale_and_layers(capi):
    st = attn_state(8, 2, 64, [5, 9], [140, 80], F16, seed=6)
    attend(capi, st, scale=0.3)
    big = torch.full((st["q"].shape[0], 3, 8, 64), NAN, dtype=F16, device="cuda")
    big[:, 1] = st["q"]
    st["q"] = big[:, 1]
    check_weigh(capi, st, scale=0.3)
    # two layers' calls add up, the first starts the step's own positions anew
    _, one = weigh(capi, st, scale=0.3, fresh=True)
    two = one.clone()
    err = ints([0, 0])
    capi.dflash_kv8_weigh(st["q"], st["lse"], *st["cache"], ints(st["table"]), ints(st["held"]), ints(st["start"]), two,
                          err, scale=0.3)
    before, _ = weigh(capi, st, scale=0.3)
    assert ((two - one) - (_ - before)).abs().max() < 1e-4


@pytest.mark.parametrize("n", [2, 40])
def test_weigh_rows_that_share_their_memory(capi, n):
    """A row stride of 0, and weights at an odd place."""
    st = attn_state(4, 2, 64, [n], [100], BF, seed=6)
    st["q"] = st["q"][:1].expand(n + 2, -1, -1)
    attend(capi, dict(st, q=st["q"].contiguous()))
    check_weigh(capi, st)
    before, want = weigh(capi, st)
    held = torch.zeros(before.numel() + 1, device="cuda")
    w = held[1:].view_as(before)
    w.copy_(before)
    capi.dflash_kv8_weigh(st["q"], st["lse"], *st["cache"], ints(st["table"]), ints(st["held"]), ints(st["start"]), w,
                          ints([0, 0]))
    assert torch.equal(w, want) and held[0] == 0


def test_weigh_rows_without_keys_and_with_nan(capi):
    """More rows than positions; NaN codes add nothing, to their own position
    alone, and rows that saw one (an lse of NaN) none at all."""
    st = attn_state(4, 2, 64, [9], [4], BF, seed=7)
    attend(capi, st)
    check_weigh(capi, st)
    st = attn_state(4, 2, 64, [3], [100], BF, seed=8)
    attend(capi, st)
    page = st["table"][0][0]
    st["cache"][0][page, 1, 5, 7] = 0x7f
    before, w = check_weigh(capi, st)
    assert w[page, 5] > before[page, 5] and w[page, 4] > before[page, 4]      # the other kv head's
    attend(capi, st)
    assert torch.isnan(st["lse"][:3, 2:]).all() and not torch.isnan(st["lse"][:3, :2]).any()
    check_weigh(capi, st)


def test_weigh_scales_far_apart(capi):
    st = attn_state(4, 2, 128, [4, 1], [200, 130], BF, seed=9)
    st["cache"][2][st["table"][0][1]] = 2.0 ** -60
    st["cache"][2][st["table"][1][0]] = 0.0
    st["cache"][2][st["table"][0][0]] = 2.0 ** -3
    attend(capi, st)
    check_weigh(capi, st)


def test_weigh_extreme_rows(capi):
    """Rows of q at both ends of the type, and zeros."""
    st = attn_state(4, 2, 64, [6], [150], BF, seed=10)
    st["q"][0] = 0
    st["q"][1] *= 1e-30
    st["q"][2] *= 30
    st["q"][3, :, 1:] *= 1e-6
    attend(capi, st)
    check_weigh(capi, st)


def test_weigh_sequences_do_not_depend_on_each_other(capi):
    rows, held = [16, 1, 40, 7], [700, 1300, 90, 64]
    st = attn_state(8, 2, 128, rows, held, BF, seed=11)
    attend(capi, st)
    before, w = weigh(capi, st)
    _, again = weigh(capi, st)
    assert torch.equal(w, again)
    for s in range(4):
        other = dict(st, held=[kv if i == s else 0 for i, kv in enumerate(held)])
        other["start"] = st["start"]
        # the others' rows see nothing: their lengths are 0
        b, o = weigh(capi, other)
        pages = [p for p in st["table"][s] if p >= 0]
        assert torch.equal(o[pages], w[pages])


def test_weigh_reports_impossible_lengths_and_pages(capi):
    st = attn_state(4, 2, 64, [2, 2, 2], [100, 100, 100], BF, seed=12)
    attend(capi, st)
    _, good = weigh(capi, st)
    for change, site in ((dict(held=[100, 10 ** 6, 100]), 304), (dict(held=[100, -1, 100]), 304),
                         (dict(start=[0, 2, 9, 6]), 304)):
        _, w = weigh(capi, dict(st, **change), want_err=(2, site))
        pages = [p for p in st["table"][0] if p >= 0]
        assert torch.equal(w[pages], good[pages])
    for bad in (-1, 10 ** 6):
        table = [list(t) for t in st["table"]]
        table[1][0] = bad
        _, w = weigh(capi, dict(st, table=table), want_err=(2, 303))
        for p in [x for x in st["table"][0] + st["table"][2] if x >= 0] + [st["table"][1][1]]:
            assert torch.equal(w[p], good[p])


@pytest.mark.parametrize("S", [70, 400])
def test_weigh_many_sequences(capi, S):
    r = np.random.RandomState(S)
    st = attn_state(2, 1, 64, r.randint(0, 4, S).tolist(), r.randint(4, 90, S).tolist(), BF, seed=13)
    attend(capi, st)
    check_weigh(capi, st)


def test_weigh_long_rows_of_a_prompt(capi):
    """Many counted rows: against sums by torch in 64 bits."""
    st = attn_state(32, 8, 128, [600, 64], [1000, 2500], F16, seed=14, q_scale=1.0)
    attend(capi, st)
    before, w = weigh(capi, st, fresh=True)
    for s, (n, kv) in enumerate(zip([600, 64], st["held"])):
        pages = st["table"][s][:-(-kv // 64)]
        k = (values(st["cache"][0])[pages] * st["cache"][2].cpu().double()[pages][..., None, None]).cuda()
        k = k.transpose(0, 1).flatten(1, 2)[:, :kv]
        r0 = st["start"][s]
        q = st["q"][r0:r0 + n].double().view(n, 8, 4, 128)
        x = torch.einsum("nhgd,hkd->nhgk", q, k) * 128 ** -0.5 - st["lse"][r0:r0 + n].double().view(n, 8, 4, 1)
        seen = torch.arange(kv, device="cuda") <= torch.arange(kv - n, kv, device="cuda")[:, None]
        t = torch.where(seen[:, None, None], x.exp(), 0.0).sum((0, 1, 2))
        old = before[pages].flatten()[:kv].double()
        old[kv - n:] = 0
        got = w[pages].flatten()[:kv].double()
        # d by the terms' own bounds, at most; n_q n + 8 roundings of the sum
        terms = torch.einsum("nhgd,hkd->nhgk", q.abs(), k.abs()).amax((0, 1, 2)) * 128 ** -0.5
        d = 138 * 2.0 ** -24 * terms + 2.0 ** -22 + 2.0 ** -22 * (x.abs().amax() + 30)
        assert ((got - old - t).abs() <= t * (d + (32 * n + 8) * 2.0 ** -24) + 2.0 ** -24 * got.abs() + 1e-12).all()


def test_weigh_nothing_to_do(capi):
    st = attn_state(4, 2, 64, [2], [100], BF)
    w, err = torch.ones(st["cache"][0].shape[0], 64, device="cuda"), ints([0, 0])
    capi.dflash_kv8_weigh(st["q"][:0], st["lse"][:0], *st["cache"], ints(st["table"]), ints(st["held"]), ints([0, 0]), w,
                          err)
    assert (w == 1).all() and err.tolist() == [0, 0]


# ------------------------------------------------------------------ eviction

def weights_of(pages, seed, ties=False):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(pages, 64, generator=g) ** 4
    if ties:
        w = (w * 6).floor()
    return w


class Evict:
    def __init__(self, capi, held, n_kv=2, dim=64, layers=2, seed=0, ties=False, spread=3):
        g = torch.Generator().manual_seed(seed)
        need = [-(-kv // 64) for kv in held]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g).tolist()
        width = max(max(need), 1) + 1
        self.table, at = [], 0
        for n in need:
            self.table.append(order[at:at + n] + [-1] * (width - n))
            at += n
        self.caches = []
        for i in range(layers):
            kc, vc, ks, vs = pool(pages, n_kv, dim, seed + i)
            for x in (ks, vs):
                x.copy_(torch.exp2(torch.randint(-9 - spread, -8, x.shape, generator=g).float()))
            self.caches.append([kc, vc, ks, vs])
        self.held, self.w = held, weights_of(pages, seed + 9, ties).cuda()
        self.err, self.S, self.width = ints([0, 0]), len(held), width
        self.ws = torch.full((capi.dflash_kv8_evict_workspace_bytes(self.S, width),), 0xa5, dtype=torch.uint8, device="cuda")
        self.source = torch.full((self.S, width * 64), -7, dtype=torch.int32, device="cuda")
        self.new, self.dropped = ints([-7] * self.S), ints(list(range(self.S)))

    def snapshot(self):
        f = lambda t: t.double().cpu().numpy().copy()      # noqa: E731
        return [(values(c[0]).numpy().copy(), values(c[1]).numpy().copy(), f(c[2]), f(c[3])) for c in self.caches], f(self.w)

    def run(self, capi, budget, first=0, last=0, out=None, stream=None):
        capi.dflash_kv8_evict(capi.kv8_layers(self.caches), ints(self.table), ints(self.held), self.w, ints(budget),
                              self.new, self.source, self.ws, self.err, weights_out=out, dropped=self.dropped,
                              keep_first=first, keep_last=last, stream=stream)
        torch.cuda.synchronize()
        return self

    def check(self, capi, budget, first=0, last=0, out=None, err=(0, 0), bad=()):
        layers, w = self.snapshot()
        held = [0 if s in bad else kv for s, kv in enumerate(self.held)]
        kept_out = None if out is None else out.double().cpu().numpy().copy()
        self.run(capi, budget, first, last, out)
        before = w.copy()
        new, source, gone = P.evict(layers, self.table, held, w, budget, first, last)
        for s in bad:
            new[s], source[s] = self.held[s], []
        assert tuple(self.err.tolist()) == tuple(err)
        assert self.new.tolist() == new
        assert self.dropped.tolist() == [s + x for s, x in enumerate(gone)]
        for s in range(self.S):
            n = len(source[s])
            assert self.source[s, :n].tolist() == source[s]
            assert (self.source[s, n:] == -7).all()
        after = self.snapshot()
        for (a, b) in zip(after[0], layers):
            for which in range(2):
                assert np.array_equal(a[which], b[which], equal_nan=True)
                assert np.array_equal(a[2 + which], b[2 + which])
        if out is None:
            assert np.array_equal(after[1], w, equal_nan=True)
        else:
            assert np.array_equal(after[1], before, equal_nan=True)
            for s in range(self.S):
                for i in range(len(source[s])):
                    p = self.table[s][i // 64]
                    kept_out[p, i % 64] = w[p, i % 64]
            assert np.array_equal(out.double().cpu().numpy(), kept_out, equal_nan=True)
        return new


@pytest.mark.parametrize("held,budget,first,last", [
    ([1], [1], 0, 0), ([2], [1], 0, 0), ([2], [1], 1, 0), ([2], [1], 0, 5), ([64], [63], 2, 2), ([65], [64], 0, 0),
    ([65], [1], 9, 9), ([130, 64, 200], [64, 64, 128], 4, 16), ([300], [100], 4, 32), ([300], [299], 0, 0),
    ([300, 0, 5, 1000], [0, 0, -3, 512], 1, 100), ([700, 129], [333, 70], 0, 0), ([1000], [40], 100, 30),
    ([1000], [40], 3, 300), ([2500, 2500], [1500, 2400], 4, 256)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(capi, held, budget, first, last, ties):
    Evict(capi, held, seed=len(held) + budget[0], ties=ties).check(capi, budget, first, last)


@pytest.mark.parametrize("n_kv,dim,layers", [(1, 64, 1), (3, 128, 2), (8, 128, 1), (2, 64, 33), (1, 128, 70)])
def test_evict_shapes(capi, n_kv, dim, layers):
    e = Evict(capi, [260, 190], n_kv, dim, layers, seed=layers)
    e.check(capi, [150, 100], 2, 20)


def test_evict_more_pools_than_run_at_once(capi):
    """Chains of pages in a little more than one round: two CTAs each."""
    Evict(capi, [1200], 8, 64, 31, seed=12).check(capi, [700], 4, 64)
    Evict(capi, [500, 80], 4, 128, 31, seed=13).check(capi, [130, 70], 4, 64)


def test_evict_clusters_repeat_their_bits(capi):
    """Few chains: clusters of 2, 4 and 8 CTAs share the pages of a turn, over many
    turns.  Neighbouring pages' scales differ, so a scale of another turn would show."""
    for held, budget, n_kv, dim, layers in (([6000], [5000], 1, 128, 2), ([5000], [4500], 4, 128, 5),
                                            ([7000, 3000], [6000, 2900], 8, 64, 4), ([9000], [8500], 2, 64, 1)):
        make = lambda: Evict(capi, held, n_kv, dim, layers, seed=layers, spread=6)      # noqa: E731
        first = make()
        first.check(capi, budget, 4, 64)
        for _ in range(5):
            again = make().run(capi, budget, 4, 64)
            assert torch.equal(again.w, first.w) and torch.equal(again.source, first.source)
            for a, b in zip(again.caches, first.caches):
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_evict_special_weights(capi):
    e = Evict(capi, [400], seed=3)
    w = e.w.view(-1)
    r = torch.randperm(w.numel(), generator=torch.Generator().manual_seed(1)).cuda()
    w[r[:60]] = NAN
    w[r[60:90]] = INF
    w[r[90:120]] = -INF
    w[r[120:200]] = 0.0
    w[r[200:260]] = -0.0
    w[r[260:290]] = -1.5
    w[r[290:300]] = 1e-42
    e.check(capi, [333], 3, 5)
    e = Evict(capi, [200], seed=4)
    e.w.fill_(NAN)
    e.check(capi, [100])
    e = Evict(capi, [200], seed=5)
    e.w.fill_(0.0)
    e.w[e.table[0][1], 7] = -0.0
    e.check(capi, [100], 10, 10)


def test_evict_scales_far_apart_and_nan_codes(capi):
    e = Evict(capi, [500], 2, 128, 2, seed=6)
    for c in e.caches:
        for x in c[2:]:
            x.copy_(torch.exp2(torch.randint(-100, 120, x.shape, generator=torch.Generator().manual_seed(2)).float()))
        c[0][:, :, ::7, 3] = 0x7f
        c[1][:, :, ::5, 9] = 0xff
    e.caches[0][2][e.table[0][0]] = 0.0
    e.caches[0][2][e.table[0][1]] = 0.0
    e.check(capi, [250], 1, 1)


def test_evict_into_other_weights(capi):
    e = Evict(capi, [300, 100, 500], seed=7)
    e.check(capi, [128, 200, 300], 4, 30, out=torch.full_like(e.w, 5.0))


def test_evict_leaves_impossible_sequences_alone(capi):
    e = Evict(capi, [300, 300, 300], seed=8)
    e.table[1][2] = -1
    e.check(capi, [100, 100, 100], 4, 30, err=(2, 303), bad=[1])
    e = Evict(capi, [300, 300, 300], seed=8)
    e.table[2][0] = 10 ** 6
    e.check(capi, [100, 100, 100], 4, 30, err=(2, 303), bad=[2])
    for kv in (-1, 10 ** 6):
        e = Evict(capi, [300, 300, 300], seed=8)
        e.held = [300, kv, 300]
        e.check(capi, [100, 100, 100], 4, 30, err=(2, 304), bad=[1])


def test_evict_long_and_many(capi):
    Evict(capi, [70000], 1, 64, 1, seed=9).check(capi, [40000], 4, 1000)
    Evict(capi, [70000], 1, 64, 1, seed=9, ties=True).check(capi, [4000], 4, 1000)
    r = np.random.RandomState(3)
    held = r.randint(0, 200, 200).tolist()
    Evict(capi, held, 1, 64, 1, seed=10).check(capi, r.randint(-20, 200, 200).tolist(), 2, 9)


def test_evict_again_and_again(capi):
    """Each call's result is the next one's start."""
    e = Evict(capi, [900, 700], seed=11)
    for b in (800, 640, 639, 500, 64, 3):
        new = e.check(capi, [b, b], 2, 20 if b > 100 else 1)
        e.held = new
        e.source.fill_(-7)
        e.dropped.copy_(ints([0, 1]))


def test_evict_streams_and_graphs(capi):
    """On another stream, and captured: two graphs over one workspace."""
    want, got = (Evict(capi, [900, 700, 64], 2, 128, 3, seed=12) for _ in range(2))
    want.run(capi, [300, 800, 50], 4, 40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got.run(capi, [300, 800, 50], 4, 40, stream=s)
    same = lambda a, b: all(torch.equal(x, y) for c, d in zip(a.caches, b.caches) for x, y in zip(c, d)) and \
        torch.equal(a.w, b.w) and torch.equal(a.source, b.source) and torch.equal(a.new, b.new)     # noqa: E731
    assert same(want, got)
    a, b = (Evict(capi, [900, 700, 64], 2, 128, 3, seed=12) for _ in range(2))
    layers, table, held, budget = capi.kv8_layers(a.caches), ints(a.table), ints(a.held), ints([0, 0, 0])
    graphs = []
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            capi.dflash_kv8_evict(layers, table, held, a.w, budget, a.new, a.source, a.ws, a.err, dropped=a.dropped,
                                  keep_first=4, keep_last=40)
        graphs.append(g)
    for i, bud in enumerate(([300, 800, 50], [200, 0, 0], [0, 300, 7])):
        budget.copy_(ints(bud))
        graphs[i % 2].replay()
        b.run(capi, bud, 4, 40)
        assert same(a, b)
        held.copy_(a.new)
        b.held = b.new.tolist()


# ------------------------------------------------------------------ positions

@pytest.mark.parametrize("S,pad", [(1, 0), (5, 3), (300, 100)])
def test_shift(capi, S, pad):
    r = np.random.RandomState(S)
    n, first, dropped = r.randint(0, 6, S), r.randint(0, 3, S) * 50, r.randint(0, 99, S).tolist()
    start = [0] + np.cumsum(n).tolist()
    pos, want = [], []
    for s in range(S):
        for i in range(n[s]):
            pos.append(int(first[s] + i))
            want.append(int(first[s] + i + (dropped[s] if first[s] else 0)))
    left = [0 if n[s] and first[s] == 0 else dropped[s] for s in range(S)]
    pos += [-1] * pad
    want += [-1] * pad
    p, d = ints(pos), ints(dropped)
    for out in (torch.full_like(p, -9), p):
        d.copy_(ints(dropped))
        capi.dflash_pages_shift(p, ints(start), d, out)
        assert out.tolist() == want and d.tolist() == left


# ------------------------------------------------------------------ together

def test_a_run_of_steps(capi):
    """Prompts, then steps of draft rows over a cache that is kept at its budget:
    plan, rotary at true positions, attention, weights, verification, trim,
    eviction.  Every step's attention is checked against the definitions over a
    model of the cache that holds true positions, and every weight against its
    own sum."""
    from block_diffusion_speculative_gather_gb300.runtime import PagedKV8
    n_q, n_kv, dim, S, V, layers, bud = 8, 2, 64, 3, 501, 2, 150
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = PagedKV8(layers, n_q, n_kv, dim, S=S, pages=40, max_pages=12, rows=700, rope=capi.rope_config(dim, theta=1e4),
                  vocab=V, evict=True)
    freq = K.frequencies(dim, 1e4)
    model = [[] for _ in range(S)]        # true positions of the cached ones
    lens = [0] * S                        # true lengths
    f = lambda t: t.double().cpu().numpy()      # noqa: E731
    steps = [[400, 31, 200], [5, 5, 5], [8, 1, 0], [6, 6, 6], [16, 16, 16], [3, 150, 2], [4, 4, 4]]
    for i, n in enumerate(steps):
        if i == 4:                        # the second sequence ends, another takes its place
            kv.trim([10 ** 6, 0, 10 ** 6])
            model[1], lens[1] = [], 0
        kv.plan(n)
        start = kv.row_start.tolist()
        assert start == [0] + np.cumsum(n).tolist()
        rows, total = kv.rows, start[-1]
        want = [lens[s] + j for s in range(S) for j in range(n[s])] + [-1] * (rows - total)
        assert kv.angles.tolist() == want
        qkv = torch.randn(rows, n_q + 2 * n_kv, dim, device="cuda", generator=g).to(BF)
        lse = torch.zeros(rows, n_q, device="cuda")
        before = f(kv.weights)
        bound = np.zeros_like(before)
        for layer in range(layers):
            x = qkv.roll(layer, 0).clone()
            q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
            raw = x[:total, :n_q + n_kv].cpu()
            kv.rotate(q, k)
            ref = K.rope(raw, torch.tensor(want[:total]), dim, False, freq)
            assert ((x[:total, :n_q + n_kv].cpu().double() - ref).abs() <= half_step(BF) * ref.abs() + 1e-4).all()
            out = kv.attend(layer, q, k, v, lse=lse)
            kv.weigh(layer, q, lse, observe=32)
            c = kv.caches[layer]
            table, held = kv.table.tolist(), kv.kv_len.tolist()
            st = dict(q=q[:total].contiguous(), cache=c, table=table, held=held, start=start, out=out[:total], lse=lse[:total])
            if i:
                from tests.test_gpu_kv8 import check_attend
                check_attend(st)
            before, b = P.weigh(f(q), f(lse), values(c[0]).numpy(), f(c[2]), table, held, start, before,
                                observe=32, fresh=layer == 0, scale=dim ** -0.5)
            bound += b
        e = np.abs(f(kv.weights) - before)
        for s in range(S):
            model[s] += [lens[s] + j for j in range(n[s])]
            assert len(model[s]) == held[s]
            for p in table[s][:-(-held[s] // 64)]:
                assert (e[p] <= bound[p] + 1e-30).all()
        probs = torch.softmax(3 * torch.randn(rows, V, device="cuda", generator=g), 1)
        q_probs = torch.softmax(probs.roll(1, 0).log() + torch.randn(rows, V, device="cuda", generator=g), 1)
        ids = q_probs.argmax(1).int()
        u = torch.rand(rows, device="cuda", generator=g)
        if not i:
            u.zero_()                     # a prompt's rows all stay
            q_probs[:, :] = probs.roll(1, 0)
        tok, got = kv.accept(probs, ids, u, q_probs)
        t, cnt, new = P.verify(f(probs)[:total], ids.tolist(), u.tolist(), start, f(q_probs), kv.kv_len.tolist())
        assert got.tolist() == cnt and kv.new_len.tolist() == new
        assert tok[:total].tolist() == [t[r] for r in range(total)]
        kv.trim()
        for s in range(S):
            gone = held[s] - new[s]
            model[s] = model[s][:len(model[s]) - gone]
            lens[s] += n[s] - gone
        w = f(kv.weights)
        pools = [(values(c[0]).numpy().copy(), values(c[1]).numpy().copy(), f(c[2]), f(c[3])) for c in kv.caches]
        table = kv.table.tolist()
        want_new, source, _ = P.evict(pools, table, new, w, [bud] * S, 4, 40)
        kv.evict([bud] * S, keep_first=4, keep_last=40)
        assert kv.kv_len.tolist() == want_new
        for s in range(S):
            model[s] = [model[s][j] for j in source[s]]
            assert lens[s] - len(model[s]) == kv.dropped.tolist()[s]
            for p in table[s][:-(-want_new[s] // 64)]:
                for c, want_c in zip(kv.caches, pools):
                    assert np.array_equal(values(c[0])[p].numpy(), want_c[0][p])
                    assert np.array_equal(f(c[3])[p], want_c[3][p])
        kv.check()
    assert sorted(kv.free[:kv.n_free.item()].tolist() + [p for t in kv.table.tolist() for p in t if p >= 0]) == list(range(40))


def test_captured_steps_advance_like_eager_ones(capi):
    """A graph of a whole step (plan to eviction), replayed beside an eager run."""
    from block_diffusion_speculative_gather_gb300.runtime import PagedKV8
    n_q, n_kv, dim, S, V, bud = 8, 2, 128, 3, 1000, 100
    make = lambda: PagedKV8(1, n_q, n_kv, dim, S=S, pages=30, max_pages=8, rows=48, rope=capi.rope_config(dim),  # noqa: E731
                            vocab=V, evict=True)
    eager, cap = make(), make()
    qkv = torch.zeros(48, n_q + 2 * n_kv, dim, dtype=BF, device="cuda")
    probs, q_probs = torch.zeros(48, V, device="cuda"), torch.zeros(48, V, device="cuda")
    ids, u = torch.zeros(48, dtype=torch.int32, device="cuda"), torch.zeros(48, device="cuda")
    spaces = [dict(lse=torch.zeros(48, n_q, device="cuda"), x=torch.empty_like(qkv), out=torch.zeros_like(qkv[:, :n_q]))
              for _ in range(2)]

    def step(kv, space):
        kv.plan()
        x = space["x"]
        x.copy_(qkv)
        q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
        kv.rotate(q, k)
        kv.attend(0, q, k, v, out=space["out"], lse=space["lse"])
        kv.weigh(0, q, space["lse"])
        kv.accept(probs, ids, u, q_probs)
        kv.trim()
        kv.evict(keep_first=2, keep_last=20)

    for kv in (eager, cap):
        kv.q_len.copy_(ints([16, 16, 16]))
        kv.budget.copy_(ints([bud, bud, 0]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            step(cap, spaces[1])
        graphs.append(gr)
    for i in range(16):
        qkv.copy_(torch.randn(qkv.shape, device="cuda"))
        probs.copy_(torch.softmax(2 * torch.randn(48, V, device="cuda"), 1))
        q_probs.copy_(probs.roll(1, 0))
        ids.copy_(q_probs.argmax(1))
        u.copy_(torch.rand(48, device="cuda") * 1.1)
        step(eager, spaces[0])
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        n = eager.row_start[-1].item()
        for name in ("kv_len", "table", "free", "n_free", "row_start", "positions", "slots", "angles", "dropped", "kept",
                     "tokens", "n_tokens", "new_len"):
            assert torch.equal(getattr(eager, name), getattr(cap, name)), name
        assert torch.equal(spaces[0]["out"][:n], spaces[1]["out"][:n])
        for a, b in zip(eager.caches[0], cap.caches[0]):
            assert torch.equal(a, b)
        assert torch.equal(eager.weights, cap.weights)
    assert eager.dropped.tolist()[0] > 0 and eager.dropped.tolist()[2] == 0
    eager.check()
    cap.check()


@pytest.mark.parametrize("layers,order", [(2, [1]), (2, [1, 0]), (3, [2, 1]), (2, [0, 1])])
def test_weights_of_reused_pages_start_anew_whatever_the_layers(capi, layers, order):
    """Any of the layers weighed, in any order: a sequence's positions have what its own
    rows gave them, n_q a row and layer, not what a page held for another one; eager
    and where the layers' calls are captured without the plan."""
    from block_diffusion_speculative_gather_gb300.runtime import PagedKV8
    n_q, n_kv, dim, rows = 4, 2, 64, 200
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = PagedKV8(layers, n_q, n_kv, dim, S=2, pages=8, max_pages=4, rows=rows, evict=True)
    x = torch.randn(rows, n_q + 2 * n_kv, dim, device="cuda", generator=g).to(BF)
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    lse, out = torch.zeros(rows, n_q, device="cuda"), torch.zeros(rows, n_q, dim, dtype=BF, device="cuda")

    def step():
        for i in order:
            kv.attend(i, q, k, v, out=out, lse=lse)
            kv.weigh(i, q, lse)

    def check(held, n):
        for s in range(2):
            pages = kv.table[s, :-(-held[s] // 64)].long()
            got = kv.weights[pages].flatten()[:held[s]].double().sum().item()
            want = n[s] * n_q * len(order)
            assert abs(got - want) < 1e-4 * want, (s, got, want)

    kv.plan([100, 60])
    step()
    check([100, 60], [100, 60])
    kv.trim([0, 0])
    kv.plan([60, 100])
    step()
    check([60, 100], [60, 100])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    kv.trim([0, 0])
    kv.plan([90, 70])
    graph.replay()
    check([90, 70], [90, 70])
    kv.check()


def test_steps_whose_refused_rows_do_not_count(capi):
    """Layers' rows and lse kept until verification: weights of the rows that stay alone
    (count = n_tokens, before the trim), against the definitions; eviction in their
    order; and the same steps captured."""
    from block_diffusion_speculative_gather_gb300.runtime import PagedKV8
    n_q, n_kv, dim, S, V, layers, rows, bud = 8, 2, 64, 3, 300, 2, 30, 90
    g = torch.Generator(device="cuda").manual_seed(8)
    f = lambda t: t.double().cpu().numpy()      # noqa: E731
    make = lambda: PagedKV8(layers, n_q, n_kv, dim, S=S, pages=16, max_pages=4, rows=rows,      # noqa: E731
                            rope=capi.rope_config(dim), vocab=V, evict=True)
    x = torch.zeros(layers, rows, n_q + 2 * n_kv, dim, dtype=BF, device="cuda")
    probs, q_probs = torch.zeros(rows, V, device="cuda"), torch.zeros(rows, V, device="cuda")
    ids, u = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")

    class Side:
        def __init__(self):
            self.kv, self.x = make(), torch.empty_like(x)
            self.out, self.lse = torch.zeros_like(x[0, :, :n_q]), torch.zeros(layers, rows, n_q, device="cuda")

        def forward(self):
            self.x.copy_(x)
            self.kv.plan()
            for i in range(layers):
                q, k, v = self.x[i, :, :n_q], self.x[i, :, n_q:n_q + n_kv], self.x[i, :, n_q + n_kv:]
                self.kv.rotate(q, k)
                self.kv.attend(i, q, k, v, out=self.out, lse=self.lse[i])

        def choose(self):
            _, n = self.kv.accept(probs, ids, u, q_probs)
            for i in range(layers):
                self.kv.weigh(i, self.x[i, :, :n_q], self.lse[i], count=n)

        def cut(self):
            self.kv.trim()
            self.kv.evict(keep_first=2, keep_last=20)

    eager, cap = Side(), Side()
    for a in (eager, cap):
        a.kv.budget.copy_(ints([bud, bud, 0]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cap.forward(), cap.choose(), cap.cut()
    refused = 0
    for i in range(14):
        n = [10, 10, 10] if i % 3 else [10, 4, 7]
        for a in (eager, cap):
            a.kv.q_len.copy_(ints(n))
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        probs.copy_(torch.softmax(2 * torch.randn(rows, V, device="cuda", generator=g), 1))
        q_probs.copy_(probs.roll(1, 0))
        ids.copy_(q_probs.argmax(1))
        u.copy_(torch.rand(rows, device="cuda", generator=g) * 1.1)      # an eleventh of the drafts is refused
        eager.forward()
        kv = eager.kv
        before, table, held, start = f(kv.weights), kv.table.tolist(), kv.kv_len.tolist(), kv.row_start.tolist()
        eager.choose()
        count = kv.n_tokens.tolist()
        refused += sum(n) - sum(count)
        bound = np.zeros_like(before)
        for layer in range(layers):
            c = kv.caches[layer]
            before, b = P.weigh(f(eager.x[layer, :, :n_q]), f(eager.lse[layer]), values(c[0]).numpy(), f(c[2]), table, held, start,
                                before, count=count, fresh=layer == 0, scale=dim ** -0.5)
            bound += b
        e = np.abs(f(kv.weights) - before)
        for s in range(S):
            for p in table[s][:-(-held[s] // 64)]:
                assert (e[p] <= bound[p] + 1e-30).all()
        pools = [(values(c[0]).numpy().copy(), values(c[1]).numpy().copy(), f(c[2]), f(c[3])) for c in kv.caches]
        new, source, _ = P.evict(pools, table, kv.new_len.tolist(), f(kv.weights), [bud, bud, 0], 2, 20)
        eager.cut()
        assert kv.kv_len.tolist() == new
        for s in range(S):
            if kv.dropped[s] > 0:
                assert kv.source[s, :new[s]].tolist() == source[s]
        graph.replay()
        torch.cuda.synchronize()
        for name in ("kv_len", "table", "n_free", "dropped", "kept", "n_tokens", "new_len", "weights"):
            assert torch.equal(getattr(eager.kv, name), getattr(cap.kv, name)), name
        for a, b in zip(eager.kv.caches, cap.kv.caches):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert refused > 20 and eager.kv.dropped.tolist()[0] > 0 and eager.kv.dropped.tolist()[2] == 0
    eager.kv.check()
    cap.kv.check()
