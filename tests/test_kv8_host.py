"""The 8-bit paged cache and rotary positions without a GPU: structs as the
header lays them out, argument checks of the C ABI and of the binding (each
call is refused before anything is enqueued), workspace sizes, and the plain
definitions themselves."""

import ctypes as C

import numpy as np
import pytest
import torch

from tests import kv8_plain as P


@pytest.fixture(scope="module")
def capi():
    from block_diffusion_speculative_gather_gb300 import build
    build.build()
    from block_diffusion_speculative_gather_gb300 import capi as m
    return m


PTR = 1 << 20      # aligned, never dereferenced: every call below is refused
CONFIG, ARG = -1, -3


def test_struct_sizes(capi):
    assert C.sizeof(capi.dflash_kv8_cache) == 4 * 8 + 4 * 4
    assert C.sizeof(capi.dflash_kv8_query) == 6 * 8 + 4 * 8 + 8 * 4
    assert C.sizeof(capi.dflash_rope_config) == 4 * 4 + 4 * 8 + 8
    assert C.sizeof(capi.dflash_heads) == 2 * 8 + 8 + 4 * 8


def _cache(capi, **kw):
    d = dict(k_codes=PTR, v_codes=PTR, k_scale=PTR, v_scale=PTR, n_pages=8, n_kv=2, head_dim=128, pad_=0)
    d.update(kw)
    return capi.dflash_kv8_cache(*(d[n] for n, _ in capi.dflash_kv8_cache._fields_))


def _query(capi, **kw):
    d = dict(q=PTR, out=PTR, lse=None, table=PTR, kv_len=PTR, row_start=PTR, q_row=512, q_head=128,
             out_row=512, out_head=128, rows=3, n_q=4, S=2, max_pages=4, dtype=1, causal=1, window=0,
             scale=0.1)
    d.update(kw)
    return capi.dflash_kv8_query(*(d[n] for n, _ in capi.dflash_kv8_query._fields_))


@pytest.mark.parametrize("kw,code", [
    (dict(k_codes=None), ARG), (dict(v_scale=None), ARG), (dict(head_dim=96), CONFIG),
    (dict(head_dim=256), CONFIG), (dict(n_kv=0), CONFIG), (dict(n_pages=0), CONFIG),
    (dict(n_pages=1 << 24, n_kv=2), CONFIG), (dict(k_codes=PTR + 8), ARG), (dict(k_scale=PTR + 2), ARG)])
def test_cache_guards(capi, kw, code):
    c, q = _cache(capi, **kw), _query(capi)
    big = 1 << 40
    assert capi.lib.dflash_kv8_attention(C.byref(c), C.byref(q), PTR, big, PTR, None) == code
    assert capi.lib.dflash_kv8_append(C.byref(c), PTR, 256, 128, PTR, 256, 128, 1, 3, PTR, PTR, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_q=3), CONFIG), (dict(n_q=34), CONFIG), (dict(n_q=0), CONFIG), (dict(S=0), CONFIG),
    (dict(S=4097), CONFIG), (dict(rows=-1), ARG), (dict(max_pages=0), ARG), (dict(dtype=0), ARG),
    (dict(dtype=2), ARG), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(scale=3e38), ARG), (dict(window=-1), ARG), (dict(q=PTR + 2), ARG),
    (dict(q_row=513), ARG), (dict(out_head=4), ARG), (dict(table=None), ARG), (dict(out=None), ARG),
    (dict(rows=1 << 30, n_q=32), CONFIG)])
def test_query_guards(capi, kw, code):
    c, q = _cache(capi), _query(capi, **kw)
    assert capi.lib.dflash_kv8_attention(C.byref(c), C.byref(q), PTR, 1 << 40, PTR, None) == code, kw


def test_attention_other_guards(capi):
    c, q = _cache(capi), _query(capi)
    call = capi.lib.dflash_kv8_attention
    assert call(None, C.byref(q), PTR, 1 << 40, PTR, None) == ARG
    assert call(C.byref(c), None, PTR, 1 << 40, PTR, None) == ARG
    assert call(C.byref(c), C.byref(q), None, 1 << 40, PTR, None) == ARG
    assert call(C.byref(c), C.byref(q), PTR, 1 << 40, None, None) == ARG
    assert call(C.byref(c), C.byref(q), PTR, 1 << 40, PTR + 4, None) == ARG


def test_append_guards(capi):
    c = _cache(capi)
    call = capi.lib.dflash_kv8_append
    ok = [C.byref(c), PTR, 256, 128, PTR, 256, 128, 1, 3, PTR, PTR, None]
    for at, bad in ((1, None), (4, None), (7, 2), (8, -1), (9, None), (10, None), (1, PTR + 1), (10, PTR + 4)):
        a = list(ok)
        a[at] = bad
        assert call(*a) == ARG, (at, bad)


def test_plan_guards(capi):
    ok = [PTR, PTR, 2, PTR, 8, PTR, PTR, 4, 16, PTR, PTR, PTR, PTR, PTR, None]
    for at, bad in ((0, None), (1, None), (2, 0), (3, None), (4, -1), (5, None), (6, None), (7, 0),
                    (7, 1 << 25), (8, -1), (9, None), (10, None), (11, None), (12, None), (13, None)):
        a = list(ok)
        a[at] = bad
        assert capi.lib.dflash_pages_plan(*a) == ARG, (at, bad)
    ok = [PTR, PTR, 2, PTR, 8, PTR, PTR, 4, None]
    for at, bad in ((0, None), (1, None), (2, 0), (3, None), (4, -1), (5, None), (6, None), (7, 0)):
        a = list(ok)
        a[at] = bad
        assert capi.lib.dflash_pages_trim(*a) == ARG, (at, bad)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=2048), dict(theta=1.0), dict(theta=float("nan")),
    dict(scaling="linear", factor=0.5), dict(scaling="parts", factor=2.0, original_len=0),
    dict(scaling="parts", factor=2.0, original_len=64, alpha=4.0, beta=4.0), dict(scale=float("inf"))])
def test_rope_config_guards(capi, kw):
    cfg = capi.rope_config(**{"rotary_dim": 64, **kw})
    h = capi.dflash_heads(PTR, PTR, 2, 0, 256, 128, 256, 128)
    assert capi.lib.dflash_rope_turns(C.byref(cfg), PTR, None) == CONFIG
    assert capi.lib.dflash_rope(C.byref(cfg), PTR, PTR, 3, 128, 1, C.byref(h), None, None) == CONFIG


def test_rope_guards(capi):
    cfg = capi.rope_config(64)
    h = capi.dflash_heads(PTR, PTR, 2, 0, 256, 128, 256, 128)
    call = capi.lib.dflash_rope
    assert call(None, PTR, PTR, 3, 128, 1, C.byref(h), None, None) == ARG
    assert call(C.byref(cfg), None, PTR, 3, 128, 1, C.byref(h), None, None) == ARG
    assert call(C.byref(cfg), PTR, None, 3, 128, 1, C.byref(h), None, None) == ARG
    assert call(C.byref(cfg), PTR, PTR, 3, 128, 2, C.byref(h), None, None) == ARG
    assert call(C.byref(cfg), PTR, PTR, 3, 32, 1, C.byref(h), None, None) == ARG      # rotary 64 of 32
    assert call(C.byref(cfg), PTR, PTR, -1, 128, 1, C.byref(h), None, None) == ARG
    for bad in (capi.dflash_heads(None, PTR, 2, 0, 256, 128, 256, 128),
                capi.dflash_heads(PTR + 1, PTR, 2, 0, 256, 128, 256, 128),
                capi.dflash_heads(PTR, PTR, -1, 0, 256, 128, 256, 128),
                capi.dflash_heads(PTR, PTR, 2, 0, 256, 128, 512, 128)):               # in place, other strides
        assert call(C.byref(cfg), PTR, PTR, 3, 128, 1, C.byref(bad), None, None) == ARG
    with pytest.raises(capi.DFlashError):
        capi.rope_config(64, scaling="cubic")


def test_workspace_sizes(capi):
    ws = capi.dflash_kv8_workspace_bytes
    assert ws(16, 1, 32, 8, 128, 17) > 0
    assert ws(0, 1, 32, 8, 128, 17) > 0
    assert ws(16, 1, 32, 8, 96, 17) == 0 and ws(16, 0, 32, 8, 128, 17) == 0 and ws(16, 1, 31, 8, 128, 17) == 0
    # long prompts need no splits: the workspace stays far below the rows' own bytes
    assert ws(16384, 4, 32, 8, 128, 256) < 256 << 20


def test_binding_refuses_on_the_host(capi):
    """dtype, shape, contiguity and device are checked before the library is
    called; host tensors are refused."""
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    codes = lambda hd=128: torch.zeros((4, 2, 64, hd), dtype=torch.uint8)
    sc = lambda: torch.zeros(4, 2)
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16)
    cfg = capi.rope_config(64)

    def plan(**kw):
        a = dict(kv_len=i32(2), q_len=i32(2), free_pages=i32(8), n_free=i32(1), table=i32(2, 4),
                 row_start=i32(3), positions=i32(5), slots=i32(5), kv_after=i32(2), n_free_out=i32(1))
        return lambda: capi.dflash_pages_plan(**{**a, **kw})

    def app(**kw):
        a = dict(k=bf(3, 2, 128), v=bf(3, 2, 128), slots=i32(3), k_codes=codes(), v_codes=codes(),
                 k_scale=sc(), v_scale=sc(), err=i32(2))
        return lambda: capi.dflash_kv8_append(**{**a, **kw})

    def att(**kw):
        a = dict(q=bf(3, 4, 128), k_codes=codes(), v_codes=codes(), k_scale=sc(), v_scale=sc(),
                 table=i32(2, 4), kv_len=i32(2), row_start=i32(3), out=bf(3, 4, 128),
                 workspace=torch.zeros(1 << 20, dtype=torch.uint8), err=i32(2))
        return lambda: capi.dflash_kv8_attention(**{**a, **kw})

    def rot(**kw):
        a = dict(cfg=cfg, turns=torch.zeros(32, dtype=torch.int64), positions=i32(3), x=bf(3, 4, 128),
                 out=bf(3, 4, 128))
        return lambda: capi.dflash_rope(**{**a, **kw})

    cases = [("q_len", plan(q_len=i32(3))), ("slots", plan(slots=i32(4))), ("table", plan(table=i32(8))),
             ("row_start", plan(row_start=i32(2))), ("n_free", plan(n_free=i32(2))),
             ("kv_len", plan(kv_len=torch.zeros(2))), ("CUDA", plan()),
             ("v", app(v=bf(3, 2, 64))), ("v", app(v=torch.zeros(3, 2, 128))), ("k", app(k=bf(3, 2, 256)[..., ::2])),
             ("k_codes", app(k_codes=torch.zeros((4, 2, 32, 128), dtype=torch.uint8))),
             ("v_codes", app(v_codes=codes(64))), ("k_scale", app(k_scale=torch.zeros(4, 3))),
             ("err", app(err=i32(1))), ("CUDA", app()),
             ("q", att(q=bf(3, 4, 64))), ("q", att(q=torch.zeros(3, 4, 128))),
             ("out", att(out=torch.zeros(3, 4, 128, dtype=torch.float16))), ("kv_len", att(kv_len=i32(3))),
             ("row_start", att(row_start=i32(2))), ("lse", att(lse=torch.zeros(3, 3))), ("CUDA", att()),
             ("turns", rot(turns=torch.zeros(64, dtype=torch.int64))), ("x", rot(x=bf(2, 4, 128))),
             ("out", rot(out=bf(3, 4, 64))), ("x2", rot(x2=bf(3, 1, 128))),
             ("x2", rot(x2=bf(3, 1, 64), out2=bf(3, 1, 64))), ("CUDA", rot())]
    for word, call in cases:
        with pytest.raises(capi.DFlashError) as e:
            call()
        assert word in str(e.value), (word, str(e.value))


def test_plain_rounding_is_the_formats():
    """The definition's e4m3 rounding against torch's conversion, over every
    code and the midpoints between neighbours."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    fine = codes[~codes.isnan()].sort().values.double()
    mid = (fine[1:] + fine[:-1]) / 2
    y = torch.cat((fine, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)))
    want = y.float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.round_e4m3(y.float().double().numpy()), want)
    assert P.round_e4m3(1e9) == 448.0 and np.isnan(P.round_e4m3(float("nan")))


def test_plain_scale_brackets_the_largest_magnitude():
    for top in (1e-30, 0.5, 447.0, 448.0, 448.0001, 896.0, 3.0e38):
        s = P.scale_for([top, -top / 2])
        assert top <= 448 * s or s == 2.0 ** 119
        assert s == 2.0 ** -100 or top > 448 * s / 2
    assert P.scale_for([0.0]) == 2.0 ** -100 and P.scale_for([np.inf, 1.0]) == P.scale_for([1.0])


def test_plain_rope_is_a_rotation_by_the_position():
    x = torch.randn(5, 2, 16, dtype=torch.float64)
    f = P.frequencies(16, 1e4)
    p = torch.tensor([0, 1, 7, 100, -1])
    for il in (False, True):
        y = P.rope(x, p, 16, il, f)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
        assert torch.equal(y[0], x[0]) and torch.equal(y[4], x[4])
        # q . k depends on the distance alone
        u = P.rope(x, p + 3, 16, il, f)
        a, b = P.rope(x, torch.full((5,), 9), 16, il, f), P.rope(x, torch.full((5,), 12), 16, il, f)
        assert torch.allclose((y[1:4] * a[1:4]).sum(-1), (u[1:4] * b[1:4]).sum(-1))
