"""Sampled decoding and eviction without a GPU: structs as the header lays
them out, argument checks of the C ABI and of the binding (each call is refused
before anything is enqueued), workspace sizes, and the plain definitions
themselves."""

import ctypes as C

import numpy as np
import pytest
import torch

from tests import sampling_plain as P
from tests.test_kv8_host import ARG, CONFIG, PTR, _cache, _query, capi   # noqa: F401 (a fixture)

BIG = 1 << 40


def test_struct_sizes(capi):      # noqa: F811
    assert C.sizeof(capi.dflash_drafts) == 9 * 8 + 2 * 8 + 4 * 4 == capi._DRAFTS.size
    assert C.sizeof(capi.dflash_evict) == 8 * 8 + 4 * 4 == capi._EVICT.size


def test_probs_guards(capi):      # noqa: F811
    call = capi.lib.dflash_probs
    ok = [PTR, 100, 0, PTR, None, 3, 100, PTR + 4096, 100, None]
    for at, bad in ((0, None), (0, PTR + 2), (2, 2), (2, 9), (3, None), (3, PTR + 2), (4, PTR + 2), (5, -1),
                    (5, (1 << 30) + 1), (6, 0), (6, (1 << 30) + 1), (7, None), (7, PTR + 4098), (8, 99), (1, -1)):
        a = list(ok)
        a[at] = bad
        assert call(*a) == ARG, (at, bad)
    # in place: the same type and rows
    assert call(PTR, 100, 1, PTR, None, 3, 100, PTR, 100, None) == ARG
    assert call(PTR, 101, 0, PTR, None, 3, 100, PTR, 100, None) == ARG
    assert call(None, 100, 0, None, None, 0, 100, None, 100, None) == 0      # no rows


def test_selftest_exchange_guards(capi):      # noqa: F811
    ok = [PTR, PTR, 3, 100, PTR + 4096, 0, 0, 0, 1000, None]
    for at, bad in ((0, None), (0, PTR + 4), (1, None), (1, PTR + 2), (2, 0), (2, 4097), (3, 0), (3, 98), (3, 4100), (4, None),
                    (4, PTR + 8), (6, -1), (6, 2), (7, -1), (8, 0), (8, 10 ** 9 + 1)):
        a = list(ok)
        a[at] = bad
        assert capi.lib.dflash_selftest_exchange(*a) == ARG, (at, bad)


def _drafts(capi, **kw):      # noqa: F811
    d = dict(probs=PTR, draft_probs=PTR, ids=PTR, uniform=PTR, row_start=PTR, kv_len=PTR, tokens=PTR + 64, n_tokens=PTR,
             new_len=PTR, probs_row=100, draft_row=100, rows=3, vocab=100, S=2, pad_=0)
    d.update(kw)
    return capi.dflash_drafts(*(d[n] for n, _ in capi.dflash_drafts._fields_))


@pytest.mark.parametrize("kw,code", [
    (dict(probs=None), ARG), (dict(probs=PTR + 2), ARG), (dict(draft_probs=PTR + 1), ARG), (dict(ids=None), ARG),
    (dict(uniform=None), ARG), (dict(row_start=None), ARG), (dict(kv_len=None), ARG), (dict(new_len=None), ARG),
    (dict(tokens=None), ARG), (dict(tokens=PTR), ARG), (dict(n_tokens=None), ARG), (dict(probs_row=-1), ARG), (dict(draft_row=-1), ARG),
    (dict(rows=-1), ARG), (dict(rows=(1 << 30) + 1), ARG), (dict(vocab=0), CONFIG), (dict(vocab=(1 << 24) + 1), CONFIG),
    (dict(S=0), CONFIG), (dict(S=65536), CONFIG)])
def test_verify_guards(capi, kw, code):      # noqa: F811
    d = _drafts(capi, **kw)
    assert capi.lib.dflash_verify_drafts(C.byref(d), PTR, BIG, PTR, None) == code


def test_verify_other_guards(capi):      # noqa: F811
    call, d = capi.lib.dflash_verify_drafts, _drafts(capi)
    need = capi.dflash_verify_workspace_bytes(2, 100)
    assert need > 0
    assert call(None, PTR, BIG, PTR, None) == ARG
    assert call(C.byref(d), None, BIG, PTR, None) == ARG
    assert call(C.byref(d), PTR + 16, BIG, PTR, None) == ARG
    assert call(C.byref(d), PTR, need - 1, PTR, None) == ARG
    assert call(C.byref(d), PTR, BIG, None, None) == ARG
    assert call(C.byref(d), PTR, BIG, PTR + 4, None) == ARG
    for S, vocab in ((0, 10), (65536, 10), (4, 0), (4, (1 << 24) + 1)):
        assert capi.dflash_verify_workspace_bytes(S, vocab) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(n_q=3), CONFIG), (dict(S=4097), CONFIG), (dict(rows=-1), ARG), (dict(max_pages=0), ARG), (dict(dtype=0), ARG),
    (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG), (dict(window=-1), ARG), (dict(q=PTR + 2), ARG),
    (dict(q_row=513), ARG), (dict(q_head=4), ARG), (dict(table=None), ARG), (dict(lse=None), ARG), (dict(q=None), ARG),
    (dict(kv_len=None), ARG), (dict(row_start=None), ARG), (dict(lse=PTR + 2), ARG), (dict(rows=1 << 30, n_q=32), CONFIG)])
def test_weigh_guards(capi, kw, code):      # noqa: F811
    c, q = _cache(capi), _query(capi, **{"lse": PTR, "out": None, **kw})
    assert capi.lib.dflash_kv8_weigh(C.byref(c), C.byref(q), PTR, None, 0, 0, PTR, None) == code, kw


def test_weigh_other_guards(capi):      # noqa: F811
    c, q = _cache(capi), _query(capi, lse=PTR)
    ok = [C.byref(c), C.byref(q), PTR, None, 0, 0, PTR, None]
    for at, bad in ((0, None), (1, None), (2, None), (2, PTR + 2), (4, -1), (6, None), (6, PTR + 4)):
        a = list(ok)
        a[at] = bad
        assert capi.lib.dflash_kv8_weigh(*a) == ARG, (at, bad)
    bad = _cache(capi, head_dim=96)
    assert capi.lib.dflash_kv8_weigh(C.byref(bad), *ok[1:]) == CONFIG


def _evict(capi, **kw):      # noqa: F811
    d = dict(table=PTR, kv_len=PTR, weights=PTR, weights_out=PTR, budget=PTR, new_len=PTR + 64, dropped=None, source=PTR,
             S=2, max_pages=4, keep_first=0, keep_last=0)
    d.update(kw)
    return capi.dflash_evict(*(d[n] for n, _ in capi.dflash_evict._fields_))


@pytest.mark.parametrize("kw,code", [
    *((dict([(n, None)]), ARG) for n in ("table", "kv_len", "weights", "weights_out", "budget", "new_len", "source")),
    (dict(new_len=PTR), ARG), (dict(keep_first=-1), ARG), (dict(keep_last=-1), ARG), (dict(S=0), CONFIG),
    (dict(S=4097), CONFIG), (dict(max_pages=0), CONFIG), (dict(max_pages=(1 << 24) + 1), CONFIG)])
def test_evict_guards(capi, kw, code):      # noqa: F811
    c, e = _cache(capi), _evict(capi, **kw)
    assert capi.lib.dflash_kv8_evict(C.byref(c), 1, C.byref(e), PTR, BIG, PTR, None) == code


def test_evict_other_guards(capi):      # noqa: F811
    call, e = capi.lib.dflash_kv8_evict, _evict(capi)
    two = (capi.dflash_kv8_cache * 2)(_cache(capi), _cache(capi, n_pages=9))
    need = capi.dflash_kv8_evict_workspace_bytes(2, 4)
    ok = [two, 1, C.byref(e), PTR, need - 1, PTR, None]
    assert need > 0 and call(*ok) == ARG
    ok[4] = need
    for at, bad, code in ((0, None, ARG), (1, 0, ARG), (1, 1025, ARG), (1, 2, CONFIG), (2, None, ARG), (3, None, ARG),
                          (3, PTR + 16, ARG), (5, None, ARG), (5, PTR + 4, ARG)):
        a = list(ok)
        a[at] = bad
        assert call(*a) == code, (at, bad)
    for S, pages in ((0, 4), (4097, 4), (2, 0), (2, (1 << 24) + 1)):
        assert capi.dflash_kv8_evict_workspace_bytes(S, pages) == 0


@pytest.mark.parametrize("n", [1, 2, 5, 1024])
def test_evict_refuses_pools_that_overlap(capi, n):      # noqa: F811
    """One pool as two layers or as K's and V's, or the end of one as the start of another."""
    codes, scales = 8 * 2 * 64 * 128, 8 * 2 * 4          # bytes of _cache's pools
    base = 1 << 40

    def call(change=None):
        layers = (capi.dflash_kv8_cache * n)()
        for i in range(n):
            at = base + (n - 1 - i) * (2 * codes + 2 * scales)
            layers[i] = _cache(capi, k_codes=at, v_codes=at + codes, k_scale=at + 2 * codes, v_scale=at + 2 * codes + scales)
        if change:
            change(layers)
        e = _evict(capi)
        assert capi.lib.dflash_kv8_evict(layers, n, C.byref(e), PTR, 1, PTR, None) == ARG
        return capi.lib.dflash_last_error()

    last = n - 1

    def same(a, b):
        return lambda x: setattr(x[last], a, getattr(x[0], b))

    assert b"workspace" in call()                        # the next thing that is refused
    for change in ([same(p, p) for p in ("k_codes", "v_codes", "k_scale", "v_scale")] if n > 1 else []) + [
            same("v_codes", "k_codes"), same("v_scale", "k_scale"),
            lambda x: setattr(x[last], "v_codes", x[last].k_codes + codes - 16),
            lambda x: setattr(x[last], "v_scale", x[last].k_scale - 4)]:
        assert b"overlap" in call(change)


def test_shift_guards(capi):      # noqa: F811
    ok = [PTR, PTR, PTR, 3, 2, PTR, None]
    for at, bad in ((0, None), (1, None), (2, None), (3, -1), (3, (1 << 30) + 1), (4, 0), (4, (1 << 30) + 1), (5, None)):
        a = list(ok)
        a[at] = bad
        assert capi.lib.dflash_pages_shift(*a) == ARG, (at, bad)


# ------------------------------------------------------------------ the binding

def _i32(*n):
    return torch.zeros(n, dtype=torch.int32)


def test_binding_names_what_is_wrong(capi, monkeypatch):      # noqa: F811
    """On host tensors: refused before the library is called."""
    c = capi
    x, p, t = torch.zeros(3, 10), torch.zeros(3, 10), torch.ones(3)

    def refused(word, f, *a, **kw):
        with pytest.raises(c.DFlashError) as e:
            f(*a, **kw)
        assert e.value.code == ARG and word in str(e.value), (word, str(e.value))

    refused("CUDA", c.dflash_probs, x, t, p)
    refused("out", c.dflash_probs, x, t, torch.zeros(3, 11))
    refused("out", c.dflash_probs, x, t, p.half())
    refused("logits", c.dflash_probs, x.double(), t, p)
    refused("logits", c.dflash_probs, torch.zeros(10, 3).t(), t, p)
    refused("temperature", c.dflash_probs, x, torch.ones(2), p)
    refused("min_p", c.dflash_probs, x, t, p, min_p=torch.ones(3, dtype=torch.float64))

    ids, u, start, tok, n, ws, err = _i32(3), torch.zeros(3), _i32(3), _i32(3), _i32(2), torch.zeros(1 << 20), _i32(2)
    v = c.dflash_verify_drafts
    refused("CUDA", v, p, ids, u, start, tok, n, ws, err)
    refused("ids", v, p, ids.long(), u, start, tok, n, ws, err)
    refused("uniform", v, p, ids, u.double(), start, tok, n, ws, err)
    refused("row_start", v, p, ids, u, _i32(2), tok, n, ws, err)
    refused("tokens", v, p, ids, u, start, _i32(4), n, ws, err)
    refused("draft_probs", v, p, ids, u, start, tok, n, ws, err, draft_probs=torch.zeros(3, 9))
    refused("together", v, p, ids, u, start, tok, n, ws, err, kv_len=_i32(2))
    refused("new_len", v, p, ids, u, start, tok, n, ws, err, kv_len=_i32(2), new_len=_i32(3))

    codes, scales = torch.zeros((4, 2, 64, 64), dtype=torch.uint8), torch.ones(4, 2)
    cache = (codes, codes, scales, scales)
    q, lse, w = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 4), torch.zeros(4, 64)
    g = c.dflash_kv8_weigh
    rest = (_i32(2, 4), _i32(2), _i32(3), w, err)
    refused("CUDA", g, q, lse, *cache, *rest)
    refused("lse", g, q, lse.t(), *cache, *rest)
    refused("weights", g, q, lse, *cache, *rest[:3], torch.zeros(3, 64), err)
    refused("count", g, q, lse, *cache, *rest, count=_i32(3))
    refused("q:", g, q.float(), lse, *cache, *rest)
    monkeypatch.setattr(c, "_here", lambda **tensors: None)
    refused("observe", g, q, lse, *cache, *rest, observe=-1, stream=0)
    refused("window", g, q, lse, *cache, *rest, window=2 ** 31, stream=0)
    monkeypatch.undo()

    refused("at least one", c.kv8_layers, [])
    refused("CUDA", c.kv8_layers, [cache])
    refused("v_codes", c.kv8_layers, [(codes, codes[:3], scales, scales)])
    monkeypatch.setattr(c, "_on_gpu", lambda **tensors: None)
    refused("shapes", c.kv8_layers, [cache, (codes[:3], codes[:3], scales[:3], scales[:3])])
    layers = c.kv8_layers([cache, cache])
    monkeypatch.undo()
    e = c.dflash_kv8_evict
    rest = [_i32(2, 4), _i32(2), w, _i32(2), _i32(2), _i32(2, 256), ws, err]
    refused("kv8_layers", e, [cache], *rest)
    refused("CUDA", e, layers, *rest)
    for at, bad, word in ((0, _i32(2, 4).long(), "table"), (1, _i32(3), "kv_len"), (2, torch.zeros(5, 64), "weights"),
                          (3, _i32(1), "budget"), (4, _i32(1), "new_len"), (5, _i32(2, 255), "source"),
                          (7, _i32(3), "err")):
        a = list(rest)
        a[at] = bad
        refused(word, e, layers, *a)
    refused("weights_out", e, layers, *rest, weights_out=w[:2])
    refused("dropped", e, layers, *rest, dropped=_i32(1))

    s = c.dflash_pages_shift
    refused("CUDA", s, _i32(3), _i32(3), _i32(2), _i32(3))
    refused("out", s, _i32(3), _i32(3), _i32(2), _i32(2))
    refused("row_start", s, _i32(3), _i32(2), _i32(2), _i32(3))


def test_the_paged_cache_class_says_what_it_was_made_without(capi):      # noqa: F811
    from block_diffusion_speculative_gather_gb300.runtime import PagedKV8
    kv = PagedKV8.__new__(PagedKV8)         # without its device buffers
    kv.tokens = kv.weights = None
    for call, word in ((lambda: kv.accept(None, None, None), "vocab"), (lambda: kv.evict(), "evict"),
                       (lambda: kv.weigh(0, None, None), "evict")):
        with pytest.raises(capi.DFlashError) as e:
            call()
        assert word in str(e.value)


# ------------------------------------------------------------------ the definitions

def test_plain_probs():
    p, _ = P.probs(np.array([0.0, 1.0, -np.inf, np.nan]), 1.0)
    e = np.e / (1 + np.e)
    assert np.allclose(p, [1 - e, e, 0, 0])
    assert P.probs(np.array([3.0, 5.0, 5.0]), 0.0)[0].tolist() == [0, 1, 0]
    assert P.probs(np.array([-np.inf, np.nan]), 1.0)[0].tolist() == [0, 0]
    assert P.probs(np.array([np.inf, 1.0, np.inf]), 2.0)[0].tolist() == [0.5, 0, 0.5]
    p, _ = P.probs(np.log([8.0, 4.0, 2.0, 1.0]).astype(np.float32).astype(float), 1.0, 0.4)
    assert np.allclose(p, [2 / 3, 1 / 3, 0, 0])


def test_plain_verification_has_the_targets_distribution():
    """Over a grid of uniform numbers, each emitted first token as often as p says."""
    p = np.array([[0.5, 0.25, 0.25], [0.25, 0.5, 0.25]])
    q = np.array([[0.0, 0.0, 0.0], [0.25, 0.5, 0.25]])
    n, count = 64, np.zeros(3)
    for d in range(3):
        for i in range(n):
            for j in range(n):
                u = [(j + 0.5) / n, (i + 0.5) / n]
                tok, _, _ = P.verify(p, [0, d], u, [0, 2], q)
                count[tok[0]] += q[1, d] / n / n
    assert np.allclose(count, p[0])


def test_plain_pick():
    w = np.array([0.0, 0.25, 0.0, 0.75, 0.0])
    got = [P.pick(w, u) for u in (-1.0, 0.0, 0.2, 0.25, 0.9, 1.0, 2.0, float("nan"))]
    assert got == [1, 1, 1, 3, 3, 3, 3, 3]
    assert P.pick(np.zeros(3), 0.5) == -1


def test_plain_evict():
    k = np.arange(2 * 64, dtype=float).reshape(2, 1, 64, 1) % 16
    v, ks, vs = k.copy(), np.array([[1.0], [2.0]]), np.array([[1.0], [1.0]])
    w = np.zeros((2, 64))
    w[0, 5], w[1, 3] = 2.0, 1.0
    new, src, gone = P.evict([(k, v, ks, vs)], [[1, 0]], [70], w, [4], 1, 1)
    # page 1 holds positions 0 .. 63, page 0 positions 64 .. 69; of equal weights the lowest position stays
    assert (new, src, gone) == ([4], [[0, 1, 3, 69]], [66])
    assert k[1, 0, :4, 0].tolist() == [0.0, 1.0, 3.0, 2.5]      # 0, 1, 3 of scale 2; 5 of scale 1
    assert ks[1, 0] == 2.0 and w[1, :4].tolist() == [0.0, 0.0, 1.0, 2.0]
