"""Rotary positions on the GPU: how far the angles are off, position by position.

The table holds each pair's frequency within 2^-52 of a turn (its fp64
arithmetic), position * frequency modulo a turn is exact, and the remainder of
at most an eighth of a turn is rounded to fp32: 2^-28 turns.  The definition's
own angle, a product in fp64, is off by position * 2^-51 radians.  Sine, cosine,
products and sums then by 8 * 2^-24 of the pair.
"""

import math

import pytest
import torch

from tests import kv8_plain as P
from tests.test_gpu_kv8 import F32, ROPE, capi   # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, 2, 5, 63, 1000, 4095, 16383, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 27 - 1, 2 ** 31 - 1]


@pytest.mark.parametrize("dim,rotary,il,w", ROPE)
def test_angles_by_position(capi, dim, rotary, il, w):      # noqa: F811
    g = torch.Generator().manual_seed(dim)
    pos = torch.tensor(POSITIONS, dtype=torch.int32)
    x = torch.randn(len(pos), 3, dim, generator=g)
    cfg = capi.rope_config(rotary, interleaved=il, **w)
    turns = torch.empty(rotary // 2, dtype=torch.int64, device="cuda")
    capi.dflash_rope_turns(cfg, turns)
    out = torch.empty_like(x, device="cuda")
    capi.dflash_rope(cfg, turns, pos.cuda(), x.cuda(), out)
    scale = w.get("scale", 1.0)
    want = P.rope(x, pos, rotary, il, P.frequencies(rotary, **{n: v for n, v in w.items() if n != "scale"}), scale)
    p = pos.double()[:, None, None]
    angle = 2 * math.pi * (2.0 ** -28 + p * 2.0 ** -52) + p * 2.0 ** -51
    tol = 2 * x.abs().max().double() * scale * (angle + 8 * 2.0 ** -24) + torch.finfo(F32).eps / 2 * want.abs()
    err = (out.cpu().double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dim,rotary,il,w", ROPE)
def test_the_table_itself(capi, dim, rotary, il, w):      # noqa: F811
    turns = torch.empty(rotary // 2, dtype=torch.int64, device="cuda")
    capi.dflash_rope_turns(capi.rope_config(rotary, interleaved=il, **w), turns)
    freq = P.frequencies(rotary, **{n: v for n, v in w.items() if n != "scale"})
    for t, f in zip(turns.tolist(), freq):
        off = t / 2.0 ** 64 - f / (2 * math.pi)
        assert abs(off - round(off)) <= 2.0 ** -51           # 2^-52 of either side
