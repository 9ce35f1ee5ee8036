"""Probabilities and verification on the GPU against their plain 64-bit
definitions (tests/sampling_plain.py).

Tolerances.
* Probabilities: with y = (x - m) / T, a weight's exponent y log2(e) is off by
  the difference's rounding (2^-24), log2(e) / T's two (2^-23) and the
  product's (2^-24), 2^-22 |y| together relative to the weight, and ex2 by
  2^-22; the sum has at most vocab / 512 + 16 roundings of a thread's terms and
  the tree, 2^-24 each; the quotient two.  The sum's own error is the average
  of its terms' errors.  Weights below 2^-126 of the largest are 0.
* Tokens, counts and lengths: equal.  The kernel's sums are exact to 2^-46 or so, and
  the plain ones to 2^-63; cases on a border have exact sums.
"""

import math

import numpy as np
import pytest
import torch

from tests import gpu_common as G
from tests import sampling_plain as P

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def capi():
    G.build_lib()
    from block_diffusion_speculative_gather_gb300 import capi as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def floats(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


# ------------------------------------------------------------------ probabilities

def check_probs(x, t, out, min_p=None, rows=None):
    """x, t, min_p, out as the call had them (out after it)."""
    xs, ps = x.double().cpu().numpy(), out.double().cpu().numpy()
    V = xs.shape[1]
    for r in range(xs.shape[0]) if rows is None else rows:
        want, d = P.probs(xs[r], float(t[r]), float(min_p[r]) if min_p is not None else 0.0)
        if float(t[r]) == 0:
            assert np.array_equal(ps[r], want), r
            continue
        y = np.abs(d)
        tol = want * ((y + (want * y).sum()) * 2.0 ** -22 + 2.0 ** -21 + (V / 512 + 16) * 2.0 ** -24 + 2.0 ** -23)
        tol += 2.0 ** -126
        e = np.abs(ps[r] - want)
        assert (e <= tol).all(), (r, float((e / tol).max()), int((e / tol).argmax()))
        assert (ps[r][want == 0] == 0).all()


def logits(rows, V, kind, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (spread * torch.randn(rows, V, device="cuda", generator=g)).to(kind)


@pytest.mark.parametrize("kind", [F32, BF, F16])
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (2, 7), (5, 255), (3, 1024), (2, 4099), (7, 8192), (3, 32003),
                                    (2, 65537), (2, 151936), (1, 163841), (1, 200001), (1, 524291)])
def test_probs(capi, rows, V, kind):
    x = logits(rows, V, kind, V)
    t = floats([0.7, 1.0, 0.0, 1.9, 0.31, 1e-3, 50.0][:rows])
    for min_p in (None, floats([0.1, 0.0, 0.5, 1.0, -1.0, 2.0, NAN][:rows])):
        out = torch.full((rows, V), 7.0, device="cuda")
        capi.dflash_probs(x, t, out, min_p=min_p)
        check_probs(x, t, out, min_p)


@pytest.mark.parametrize("kind", [F32, BF, F16])
@pytest.mark.parametrize("V,y", [(400003, 1.0), (400003, 3.0), ((1 << 24) + 5, 1.0), ((1 << 24) + 5, 0.5)])
def test_probs_of_long_flat_rows(capi, V, y, kind):
    """One likely token and V - 1 equal ones, whose roundings all go one way.  Weights e^-y are
    off by 2^-22 y + 2^-21 relative; their sum by that, and as none of its fp32 parts has more
    than 40 terms in a row and 16 levels above them, by 56 roundings of 2^-24; the quotient by
    two more."""
    x = torch.zeros(1, V, dtype=kind, device="cuda")
    x[0, V // 2] = y
    out = torch.empty(1, V, device="cuda")
    capi.dflash_probs(x, floats([1.0]), out)
    w = math.exp(-y)
    tol = 2 * (y * 2.0 ** -22 + 2.0 ** -21) + 58 * 2.0 ** -24
    top = out[0, V // 2].item()
    out[0, V // 2] = w * top
    for got, want in ((top, 1 / (1 + (V - 1) * w)), (out.min().item(), w / (1 + (V - 1) * w)), (out.max().item(), w / (1 + (V - 1) * w))):
        assert abs(got - want) <= tol * want, (got / want - 1, tol)


@pytest.mark.parametrize("V", [5, 4099, 151936])
def test_probs_of_special_logits(capi, V):
    """Masked tokens, NaN and infinities, rows without a logit, zeros of both
    signs, equal maxima far apart, the extremes of the type and of temperature."""
    x = logits(12, V, F32, 1)
    x[0, : V - 1] = -INF
    x[1] = -INF
    x[2] = NAN
    x[3, 1::2] = NAN
    x[4, [0, V - 1]] = INF
    x[5] = 0.0
    x[5, ::2] = -0.0
    x[6, [1, V - 1]] = 100.0
    x[7, 2], x[7, 3] = 3e38, -3e38
    x[8] = -3.4e38
    x[9, 1], x[9, 4] = INF, NAN
    t = floats([1.0, 1.0, 0.0, 0.5, 1.0, 0.0, 0.0, 1.0, 2.0, 0.0, 1e-45, 3e38])
    out = torch.full((12, V), 7.0, device="cuda")
    for min_p in (None, torch.full((12,), 0.3, device="cuda")):
        capi.dflash_probs(x, t, out, min_p=min_p)
        check_probs(x, t, out, min_p)
    assert (out[1:3] == 0).all()
    assert out[5, 0] == 1 and out[6, 1] == 1 and out[9, 1] == 1


def test_probs_leaves_rows_without_a_temperature(capi):
    x = logits(5, 1000, F32)
    out = torch.full((5, 1000), 7.0, device="cuda")
    t = floats([-1.0, NAN, INF, -INF, 1.0])
    capi.dflash_probs(x, t, out)
    assert (out[:4] == 7.0).all()
    check_probs(x, t, out, rows=[4])


def test_probs_cuts_exactly_at_the_border(capi):
    """Logits on the border and the fp32 values beside it."""
    t, min_p = 0.8, 0.05
    border = np.float64(2.5) + np.float64(np.float32(t)) * math.log(float(np.float32(min_p)))
    f = np.float32(border)
    near = [f]
    for way in (-np.inf, np.inf):
        v = f
        for _ in range(3):
            v = np.nextafter(v, np.float32(way))
            near.append(v)
    x = torch.tensor([[2.5] + [float(v) for v in near]], device="cuda")
    out = torch.empty_like(x)
    capi.dflash_probs(x, floats([t]), out, min_p=floats([min_p]))
    assert ((out[0, 1:] > 0).cpu().numpy() == (np.array(near, dtype=np.float64) >= border)).all()


@pytest.mark.parametrize("kind", [F32, BF])
@pytest.mark.parametrize("V,stride,shift,out_stride,out_shift", [
    (1000, 1003, 1, 1000, 0), (4097, 4100, 4, 4099, 3), (32000, 32000, 8, 32004, 2), (513, 520, 0, 513, 1),
    (151936, 151940, 4, 151936, 0), (151936, 151937, 3, 151939, 1)])
def test_probs_strides_and_alignment(capi, kind, V, stride, shift, out_stride, out_shift):
    rows = 4
    base = torch.full((rows * stride + 16,), NAN, dtype=kind, device="cuda")
    x = base[shift:shift + rows * stride].view(rows, stride)[:, :V]
    x.copy_(logits(rows, V, kind, 3))
    held = torch.full((rows * out_stride + 16,), 7.0, device="cuda")
    out = held[out_shift:out_shift + rows * out_stride].view(rows, out_stride)[:, :V]
    t, min_p = floats([0.5, 1.0, 0.0, 2.0]), floats([0.0, 0.01, 0.0, 0.2])
    capi.dflash_probs(x, t, out, min_p=min_p)
    check_probs(x, t, out, min_p)
    again = held.clone()
    held.view(-1)[out_shift:out_shift + rows * out_stride].view(rows, out_stride)[:, :V] = 7.0
    assert (held == 7.0).all()          # nothing beside the rows was written
    capi.dflash_probs(x, t, out, min_p=min_p)
    assert torch.equal(held, again)


def test_probs_in_place_and_row_shared_by_all(capi):
    x = logits(6, 10007, F32, 4)
    t = floats([0.5, 0.7, 1.0, 0.0, 2.0, 1.0])
    want = torch.empty_like(x)
    capi.dflash_probs(x, t, want)
    got = x.clone()
    capi.dflash_probs(got, t, got)
    assert torch.equal(got, want)
    one = x[:1].expand(6, -1)           # stride 0: one row at six temperatures
    capi.dflash_probs(one, t, got)
    check_probs(one, t, got)


@pytest.mark.parametrize("rows", [1, 7, 40, 300])
def test_probs_rows_do_not_depend_on_the_others(capi, rows):
    x, t = logits(rows, 20001, BF, 5), torch.rand(rows, device="cuda") + 0.3
    out, one = torch.empty(rows, 20001, device="cuda"), torch.empty(1, 20001, device="cuda")
    capi.dflash_probs(x, t, out)
    for r in (0, rows // 2, rows - 1):
        # a row alone may be dealt to more CTAs: equal within the tolerance, and the same on every run
        capi.dflash_probs(x[r:r + 1], t[r:r + 1], one)
        check_probs(x[r:r + 1], t[r:r + 1], one)
    check_probs(x, t, out, rows=[0, rows - 1])
    again = torch.empty_like(out)
    capi.dflash_probs(x, t, again)
    assert torch.equal(out, again)


MANY = [(700, 16000, F32), (700, 16003, F32), (1300, 20000, BF), (640, 20001, F16), (1240, 20001, F16),
        (330, 40000, F32), (90, 151936, F32), (100, 151936, BF), (170, 151936, BF), (45, 210000, F32), (45, 210001, F32),
        (50, 300000, BF), (50, 300001, BF)]


def many_rows(rows, V, kind):
    """More rows than run at once, with temperatures, cuts and logits of every kind among them."""
    x = logits(rows, V, kind, rows)
    x[3] = -INF
    x[5, 1::2] = NAN
    x[7, [2, V - 1]] = INF
    x[rows - 2, : V - 1] = -INF
    t = 0.3 + torch.rand(rows, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows))
    t[::7] = 0.0
    t[4], t[rows - 1], t[rows // 2] = -1.0, NAN, INF
    min_p = torch.where(torch.arange(rows, device="cuda") % 3 == 0, 0.05, 0.0)
    left = [4, rows // 2, rows - 1]
    some = sorted(set(list(range(12)) + list(range(0, rows, 37)) + [rows - 3, rows - 2]) - set(left))
    return x, t, min_p, left, some


@pytest.mark.parametrize("rows,V,kind", MANY)
def test_probs_many_rows(capi, rows, V, kind):
    x, t, min_p, left, some = many_rows(rows, V, kind)
    out = torch.full((rows, V), 7.0, device="cuda")
    capi.dflash_probs(x, t, out, min_p=min_p)
    check_probs(x, t, out, min_p, rows=some)
    assert (out[left] == 7.0).all()
    sums = out.double().sum(1)
    ok = torch.ones(rows, dtype=torch.bool, device="cuda")
    ok[left], ok[3] = False, False
    assert ((sums - 1).abs()[ok] < 1e-4).all()
    for _ in range(3):
        again = torch.full_like(out, 7.0)
        capi.dflash_probs(x, t, again, min_p=min_p)
        assert torch.equal(out, again)
    # outputs that are not 16-byte aligned, with gaps between their rows
    held = torch.full((rows * (V + 3) + 1,), 7.0, device="cuda")
    view = held[1:].view(rows, V + 3)[:, :V]
    capi.dflash_probs(x, t, view, min_p=min_p)
    check_probs(x, t, view, min_p, rows=some[:20])
    assert (held[1:].view(rows, V + 3)[:, V:] == 7.0).all() and held[0] == 7.0 and (view[left] == 7.0).all()
    if kind is F32:
        same = x.clone()
        capi.dflash_probs(same, t, same, min_p=min_p)
        keep = [r for r in range(rows) if r not in left]
        assert torch.equal(same[keep], out[keep])
        assert torch.equal(same[left].nan_to_num(1.5), x[left].nan_to_num(1.5))


def test_probs_many_rows_captured_and_side_by_side(capi):
    """The clusters that stay, in a graph, and two calls at once on two streams."""
    x, t, min_p, left, some = many_rows(700, 16000, F32)
    y, u, cut, _, other = many_rows(1300, 20000, BF)
    a, b = torch.full((700, 16000), 7.0, device="cuda"), torch.full((1300, 20000), 7.0, device="cuda")
    capi.dflash_probs(x, t, a, min_p=min_p)
    capi.dflash_probs(y, u, b, min_p=cut)
    want = a.clone(), b.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        capi.dflash_probs(x, t, a, min_p=min_p)
        capi.dflash_probs(y, u, b, min_p=cut)
    for _ in range(3):
        a.fill_(7.0), b.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    s = torch.cuda.Stream()
    for _ in range(10):
        a.fill_(7.0), b.fill_(7.0)
        torch.cuda.synchronize()
        capi.dflash_probs(x, t, a, min_p=min_p, stream=s)
        capi.dflash_probs(y, u, b, min_p=cut, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("word", [0, 1])
@pytest.mark.parametrize("stays", [False, True])
def test_probs_whose_exchange_does_not_come_about(capi, stays, word):
    """A CTA that hears nothing of the others within its limit (5 ms here): what it
    writes is NaN, and so is every later row of its cluster; rows before are right,
    rows without a temperature as they were, and the next call works."""
    rows, V, at = 9, 2004, 3
    x = logits(rows, V, F32, 2)
    x[5] = -INF
    x[4, 7] = INF
    for greedy in (False, True):
        t = floats([0.7, 0.0, 1.0, 0.0 if greedy else 0.9, 1.0, 2.0, -1.0, 0.0, 1.5])
        out = torch.full((rows, V), 7.0, device="cuda")
        # where clusters have a row each, all of them have but one, their first
        capi.dflash_selftest_exchange(x, t, out, stays, word, at if stays else 0, 5_000_000)
        torch.cuda.synchronize()
        assert (out[6] == 7.0).all()
        good, lost = ([0, 1, 2], [3, 4, 5, 7, 8]) if stays else ([], [0, 1, 2, 3, 4, 5, 7, 8])
        check_probs(x, t, out, rows=good)
        assert torch.isnan(out[lost]).all()
        # a row that no cluster has: nothing is withheld
        capi.dflash_selftest_exchange(x, t, out, stays, word, 100, 5_000_000)
        check_probs(x, t, out, rows=[r for r in range(rows) if r != 6])
        assert (out[6] == 7.0).all()
    capi.dflash_probs(x, t, out)
    check_probs(x, t, out, rows=[r for r in range(rows) if r != 6])


# ------------------------------------------------------------------ verification

class Call:
    def __init__(self, capi, rows, V, seed=0, q=True, pad=2, sharp=3.0, stride=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        start = [0]
        for n in rows:
            start.append(start[-1] + n)
        self.S, self.total, self.V, self.start = len(rows), start[-1] + pad, V, start
        x = sharp * torch.randn(self.total, V, device="cuda", generator=g)
        y = torch.roll(x, 1, 0) + 0.7 * torch.randn(self.total, V, device="cuda", generator=g)
        self.p, self.q = (self._rows(torch.softmax(z, 1), stride) for z in (x, y))
        race = torch.empty(self.total, V, device="cuda").exponential_(generator=g)
        self.ids = torch.argmax(self.q / race if q else self.q, 1).int()
        if not q:
            self.q = None
        self.u = torch.rand(self.total, device="cuda", generator=g)
        self.row_start, self.kv = ints(start), ints([100 + 7 * s + n for s, n in enumerate(rows)])
        self.ws = torch.zeros(capi.dflash_verify_workspace_bytes(self.S, V), dtype=torch.uint8, device="cuda")
        self.err = ints([0, 0])
        self.clear()

    @staticmethod
    def _rows(x, stride):
        if stride is None:
            return x
        held = torch.full((x.shape[0], stride), NAN, device="cuda")
        held[:, 1:1 + x.shape[1]] = x
        return held[:, 1:1 + x.shape[1]]

    def clear(self):
        self.tokens, self.n = torch.full((self.total,), -7, dtype=torch.int32, device="cuda"), ints([-7] * self.S)
        self.new = ints([-7] * self.S)

    def run(self, capi, stream=None):
        capi.dflash_verify_drafts(self.p, self.ids, self.u, self.row_start, self.tokens, self.n, self.ws, self.err,
                                  draft_probs=self.q, kv_len=self.kv, new_len=self.new, stream=stream)
        return self

    def check(self, err=(0, 0)):
        f = lambda t: t.double().cpu().numpy()      # noqa: E731
        tok, n, new = P.verify(f(self.p), self.ids.tolist(), self.u.tolist(), self.row_start.tolist(),
                               None if self.q is None else f(self.q), self.kv.tolist())
        got = self.tokens.tolist()
        assert self.n.tolist() == n
        assert self.new.tolist() == new
        assert [got[r] for r in sorted(tok)] == [tok[r] for r in sorted(tok)]
        assert all(v == -7 for r, v in enumerate(got) if r not in tok)
        assert tuple(self.err.tolist()) == tuple(err)
        assert (self.ws[:65536 * 4] == 0).all()     # its counters
        return tok, n


@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("rows,V", [([1], 1), ([3], 2), ([2, 5], 7), ([16], 255), ([4, 1, 16, 0, 9], 4096),
                                    ([16, 3], 4097), ([7, 16], 32003), ([40, 33, 65], 300), ([16, 16, 16], 151936),
                                    ([1] * 9, 8195), ([5] * 40, 1000)])
def test_verify(capi, rows, V, q):
    for seed in range(3):
        c = Call(capi, rows, V, seed, q)
        c.run(capi).check()


def test_verify_accepts_all_some_and_none(capi):
    """The accepted counts of a call spread over the whole range."""
    c = Call(capi, [16] * 60, 2000, 1, sharp=2.0)
    _, n = c.run(capi).check()
    assert min(n) == 1 and max(n) >= 8
    c.u.zero_()
    c.clear()
    _, n = c.run(capi).check()
    assert n == [16] * 60


@pytest.mark.parametrize("q", [True, False])
def test_verify_greedy_rows(capi, q):
    """Probabilities of 0 and 1: first-mismatch acceptance and its argmax."""
    V, rows = 50, [6, 6, 6]
    c = Call(capi, rows, V, 2, q)
    best = torch.randint(0, V, (c.total,), device="cuda")
    c.p = torch.nn.functional.one_hot(best, V).float()
    c.ids[1:] = best[:-1].int()
    c.ids[3], c.ids[7] = (best[2] + 1) % V, (best[6] + 1) % V
    if q:
        c.q = torch.nn.functional.one_hot(c.ids.long(), V).float()
    tok, n = c.run(capi).check()
    assert n == [3, 1, 6]
    assert all(tok[r] == int(best[r]) for r in (0, 1, 2, 6, 12, 13, 14, 15, 16, 17))


def test_verify_on_the_borders_of_running_sums(capi):
    """Multiples of 2^-12 with exact sums: a uniform number on a border takes the next token."""
    V, n = 4096 + 512, 4097
    c = Call(capi, [1] * n, V, 3, False, pad=0)
    w = torch.zeros(V)
    at = torch.randperm(V, generator=torch.Generator().manual_seed(5))[:600].sort().values
    w[at] = 1.0
    w[at[::3]] = 7.0
    left = 4096 - int(w.sum())
    w[at[300]] += left
    c.p = (w / 4096).cuda()[None].expand(n, V)
    c.u = (torch.arange(n, device="cuda") / 4096).float()      # 0 .. 1, both ends
    c.run(capi).check()


def test_verify_special_numbers(capi):
    """Probabilities that do not count, rows without weight, uniform numbers outside [0, 1)."""
    V, rows = 4100, [1] * 12 + [3] * 4 + [1] * 4
    c = Call(capi, rows, V, 4)
    c.p[0] = 0
    c.p[1] = NAN
    c.p[2, ::2] = INF
    c.p[3, 1::2] = -1.0
    c.u[4:9] = floats([-0.5, 1.0, 2.0, NAN, 0.0])
    c.u[24:28] = floats([-3e38, 3e38, -INF, INF])
    c.p[9], c.p[10] = 0, 0
    c.p[9, V - 1] = 1e-42                        # one token with a subnormal weight
    c.p[10, 0] = 1e30                            # the largest that count, and one above
    c.p[10, 1] = 1.2e30
    c.p[10, 2] = 1.3e30
    c.p[11] *= 1e-30
    # a refused draft where p is nowhere above q: drawn from p
    c.q[13] = c.p[12]
    c.u[13] = 1.0
    c.ids[13] = int(c.p[12].argmax())
    # nothing left at all
    c.p[15], c.q[16] = 0, 0
    # q without weight at the draft, p without
    c.q[19, c.ids[19].item()] = 0
    c.p[21, c.ids[22].item()] = 0
    c.q[22, c.ids[22].item()] = 0
    tok, n = c.run(capi).check()
    assert n[0] == n[1] == 0 and tok[0] == -1 and tok[9] == V - 1
    assert n[13] == 0 and tok[15] == -1


def test_verify_rows_without_a_draft(capi):
    c = Call(capi, [4, 4, 4], 300, 5)
    c.u.fill_(0.5)
    c.q[:] = c.p.roll(1, 0)             # every draft would be accepted
    c.ids[2] = -1
    c.ids[7] = -5
    tok, n = c.run(capi).check()
    assert n[0] == 2 and n[1] == 3 and n[2] == 4


def test_verify_reports_impossible_ids_and_rows(capi):
    c = Call(capi, [4, 4], 300, 6)
    c.u.fill_(0.5)
    c.q[:] = c.p.roll(1, 0)
    c.ids[2] = 300
    _, n = c.run(capi).check(err=(2, 2))
    assert n[0] == 2
    for start, bad in (([0, 4, 11], 1), ([-1, 4, 8], 0), ([0, 5, 4], 1), ([0, 5, -2 ** 31], 1), ([-2 ** 31, 0, 4], 0)):
        c = Call(capi, [4, 4], 300, 6)
        c.row_start = ints(start)
        c.run(capi)
        torch.cuda.synchronize()
        assert c.err.tolist() == [2, bad]
        assert c.n[bad].item() == 0 and c.new[bad].item() == c.kv[bad].item() and c.n[1 - bad].item() > 0


@pytest.mark.parametrize("V,stride", [(1000, 1003), (4099, 4100), (8192, 8200)])
def test_verify_strides_and_alignment(capi, V, stride):
    c = Call(capi, [5, 1, 16], V, 7, stride=stride)
    assert c.p.stride(0) == stride
    c.run(capi).check()


def test_verify_without_lengths_and_in_place(capi):
    c = Call(capi, [5, 1, 0, 16], 1000, 8)
    c.run(capi).check()
    want = c.tokens.clone(), c.n.clone(), c.new.clone()
    c.clear()
    capi.dflash_verify_drafts(c.p, c.ids, c.u, c.row_start, c.tokens, c.n, c.ws, c.err, draft_probs=c.q)
    assert torch.equal(c.tokens, want[0]) and torch.equal(c.n, want[1])
    kv = c.kv.clone()
    capi.dflash_verify_drafts(c.p, c.ids, c.u, c.row_start, c.tokens, c.n, c.ws, c.err, draft_probs=c.q, kv_len=kv,
                              new_len=kv)
    assert torch.equal(kv, want[2])


def test_verify_past_4_gib_of_probabilities(capi):
    """Row offsets past 32 bits."""
    V, rows = 151936, 14500
    p = torch.zeros(rows, V, device="cuda")
    hot = torch.randint(0, V, (rows,), device="cuda")
    p.scatter_(1, hot[:, None], 1.0)
    tok, n = torch.full((rows,), -7, dtype=torch.int32, device="cuda"), ints([0] * 3)
    ids = torch.cat((hot[:1], hot[:-1])).int()
    ids[rows - 5] = (hot[rows - 6] + 1) % V
    ws = torch.zeros(capi.dflash_verify_workspace_bytes(3, V), dtype=torch.uint8, device="cuda")
    start = ints([0, 1, rows - 9, rows])
    err = ints([0, 0])
    capi.dflash_verify_drafts(p, ids, torch.full((rows,), 0.5, device="cuda"), start, tok, n, ws, err)
    assert n.tolist() == [1, rows - 10, 5 - 1] and err.tolist() == [0, 0]
    assert tok[rows - 9:].tolist() == hot[rows - 9:rows - 5].int().tolist() + [-1] * 5
    assert torch.equal(tok[1:rows - 9], hot[1:rows - 9].int())


def test_many_sequences_and_one_workspace_for_all_shapes(capi):
    """Small and large shapes in turn over one workspace."""
    ws = torch.zeros(capi.dflash_verify_workspace_bytes(3000, 40000), dtype=torch.uint8, device="cuda")
    for seed, (rows, V) in enumerate([([1] * 3000, 50), ([16] * 3, 40000), ([2] * 700, 4097), ([1], 40000),
                                      ([3] * 100, 9000), ([1] * 3000, 50)]):
        c = Call(capi, rows, V, seed)
        c.ws = ws
        c.run(capi).check()


def test_repeats_streams_and_two_calls_at_once(capi):
    a, b = Call(capi, [16] * 8, 151936, 1), Call(capi, [3] * 50, 32003, 2, False)
    want = [[t.clone() for t in (c.run(capi).tokens, c.n, c.new)] for c in (a, b)]
    a.check()
    b.check()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        torch.cuda.synchronize()
        for c, x in ((a, s), (b, t)):
            c.run(capi, stream=x)
        torch.cuda.synchronize()
        for c, w in zip((a, b), want):
            assert all(torch.equal(x, y) for x, y in zip((c.tokens, c.n, c.new), w))


def test_captured_calls(capi):
    """Probabilities and verification in a graph, replayed with other inputs;
    two graphs share a workspace."""
    V, n = 32003, 12
    x, t = torch.zeros(n, V, dtype=BF, device="cuda"), torch.full((n,), 0.8, device="cuda")
    min_p = torch.full((n,), 0.02, device="cuda")
    c = Call(capi, [4, 4, 4], V, 1, pad=0)
    c.p = torch.zeros(n, V, device="cuda")

    def step():
        capi.dflash_probs(x, t, c.p, min_p=min_p)
        c.run(capi)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        graphs.append(g)
    for i in range(6):
        x.copy_(logits(n, V, BF, 20 + i))
        c.u.copy_(torch.rand(n, device="cuda"))
        c.ids.random_(0, V)
        c.ids[1:] = torch.where(torch.rand(n - 1, device="cuda") < 0.7, x[:-1].argmax(1).int(), c.ids[1:])
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        check_probs(x, t, c.p, min_p, rows=[0, 5, 11])
        c.check()


def test_nothing_to_do(capi):
    e = torch.empty
    capi.dflash_probs(e(0, 100, device="cuda"), e(0, device="cuda"), e(0, 100, device="cuda"))
    c = Call(capi, [0, 0], 100, 1, pad=3)
    c.run(capi)
    assert c.n.tolist() == [0, 0] and c.new.tolist() == c.kv.tolist() and (c.tokens == -7).all()
    c = Call(capi, [0, 0], 100, 1, pad=0)
    c.run(capi)
    assert c.n.tolist() == [0, 0] and c.new.tolist() == c.kv.tolist()


def test_tokens_over_ids_are_refused(capi):
    c = Call(capi, [3, 3], 500, 1)
    c.tokens = c.ids
    with pytest.raises(capi.DFlashError) as e:
        c.run(capi)
    assert e.value.code == -3 and "ids" in str(e.value)


def test_a_small_workspace_is_refused(capi):
    c = Call(capi, [3, 3], 5000, 1)
    c.ws = c.ws[:-256]
    with pytest.raises(capi.DFlashError) as e:
        c.run(capi)
    assert e.value.code == -3 and "workspace" in str(e.value)
