"""Limits of the 8-bit paged cache's calls, without a GPU (each call is
refused before anything is enqueued)."""

import ctypes as C

import pytest
import torch

from tests.test_kv8_host import ARG, CONFIG, PTR, _cache, _query, capi   # noqa: F401 (a fixture)

OVER = [(1 << 30) + 1, 2 ** 31 - 1]


@pytest.mark.parametrize("n", OVER)
def test_counts_whose_sums_leave_int32(capi, n):      # noqa: F811
    lib = capi.lib
    assert lib.dflash_pages_plan(PTR, PTR, n, PTR, 8, PTR, PTR, 4, 16, PTR, PTR, PTR, PTR, PTR, None) == ARG
    assert lib.dflash_pages_plan(PTR, PTR, 2, PTR, 8, PTR, PTR, 4, n, PTR, PTR, PTR, PTR, PTR, None) == ARG
    assert lib.dflash_pages_trim(PTR, PTR, n, PTR, 8, PTR, PTR, 4, None) == ARG
    c = _cache(capi)
    assert lib.dflash_kv8_append(C.byref(c), PTR, 0, 0, PTR, 0, 0, 1, n, PTR, PTR, None) == ARG
    q = _query(capi, rows=n, n_q=2)
    assert lib.dflash_kv8_attention(C.byref(c), C.byref(q), PTR, 1 << 40, PTR, None) == CONFIG
    cfg, h = capi.rope_config(64), capi.dflash_heads(PTR, PTR, 2, 0, 0, 0, 0, 0)
    assert lib.dflash_rope(C.byref(cfg), PTR, PTR, n, 128, 1, C.byref(h), None, None) == ARG


def test_extents_beyond_int32_do_not_wrap(capi):      # noqa: F811
    capi._counts(rows=2 ** 31 - 1, S=0)
    for n in (2 ** 31, 2 ** 32 + 5):
        with pytest.raises(capi.DFlashError) as e:
            capi._counts(S=1, rows=n)
        assert "rows" in str(e.value)


@pytest.mark.parametrize("kw,word", [(dict(window=2 ** 31), "window"), (dict(window=-2 ** 31 - 1), "window"),
                                     (dict(window=1.5), "window"), (dict(scale="x"), "scale")])
def test_window_and_scale_outside_their_types(capi, monkeypatch, kw, word):      # noqa: F811
    """The library's error, not the one of packing its struct."""
    monkeypatch.setattr(capi, "_here", lambda **tensors: None)      # host tensors: refused before the call
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    q, out = (torch.zeros((3, 4, 64), dtype=torch.bfloat16) for _ in range(2))
    codes, scales = torch.zeros((4, 2, 64, 64), dtype=torch.uint8), torch.ones(4, 2)
    with pytest.raises(capi.DFlashError) as e:
        capi.dflash_kv8_attention(q, codes, codes, scales, scales, i32(2, 4), i32(2), i32(3), out,
                                  torch.zeros(1 << 20, dtype=torch.uint8), i32(2), stream=0, **kw)
    assert e.value.code == ARG and word in str(e.value)


def test_rotating_without_rotary_settings(capi):      # noqa: F811
    c = capi
    from block_diffusion_speculative_gather_gb300.runtime import PagedKV8
    kv = PagedKV8.__new__(PagedKV8)         # without its device buffers
    kv.rope = None
    with pytest.raises(c.DFlashError) as e:
        kv.rotate(torch.zeros(3, 4, 64), torch.zeros(3, 2, 64))
    assert "rope" in str(e.value)
