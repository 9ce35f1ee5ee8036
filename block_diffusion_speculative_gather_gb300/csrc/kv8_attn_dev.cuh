// Work items of the attention over the 8-bit paged cache and the small
// device helpers its two kernels share.
#pragma once

#include "gemm.cuh"
#include "kv8.cuh"

namespace dfl {
namespace kv8 {

// Sites of err words.
constexpr int SITE_FULL = 301, SITE_EMPTY = 302, SITE_PAGE = 303, SITE_LEN = 304, SITE_SCALE = 305;

__device__ __forceinline__ void report(int* err, int code, int info) {
    if (err && atomicCAS(err, 0, code) == 0) err[1] = info;
}

// Bounded mbarrier wait, about two seconds by the SM's clock: reading the
// global timer between polls took a wait 1600 cycles to end instead of 700.
constexpr long long WAIT_CYCLES = 4000000000ll;
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > WAIT_CYCLES) return false;
    }
}

// Items are handed out one by one, as sequences differ in length: a CTA's
// first is its index, the others come from a counter in the workspace.  The
// last CTA to be refused one puts the counters back to zero.
// `ask` has the answer on its way while the caller goes on; `settle` reads it.
__device__ __forceinline__ int ask_item(const Kv8AttnArgs& a, int total) {
    return total > (int)gridDim.x ? atomicAdd(a.queue, 1) : 0;
}
__device__ __forceinline__ int settle_item(const Kv8AttnArgs& a, int total, int asked) {
    if (total <= (int)gridDim.x) return -1;      // each has had its only one
    const int item = (int)gridDim.x + asked;
    if (item < total) return item;
    if (atomicAdd(a.queue + 1, 1) == (int)gridDim.x - 1) {
        a.queue[0] = 0;
        a.queue[1] = 0;
    }
    return -1;
}

// One sequence of the call: its rows, keys and how they are cut.
struct Seq {
    int r0, n;          // rows r0 .. r0 + n - 1
    int kv, first;      // cached tokens; position of the first row (may be negative: rows without keys)
    int page_lo, page_hi;
    int tiles, splits, len;   // row tiles, splits of the pages, pages of a split
};

__device__ __forceinline__ Seq seq_of(const Kv8AttnArgs& a, int s) {
    Seq q;
    const int r0 = a.row_start[s], r1 = a.row_start[s + 1];
    q.r0 = r0;
    q.n = r1 - r0;
    int kv = a.kv_len[s];
    const long long cap = (long long)a.max_pages * KV8_PAGE;
    if (r0 < 0 || r1 < r0 || r1 > a.rows || kv < 0 || kv > cap) {
        report(a.err, DERR_INDEX, SITE_LEN);   // such a sequence is skipped
        q.n = 0;
        q.r0 = 0;
        kv = 0;
    }
    q.kv = kv;
    q.first = kv - q.n;
    int lo = 0;
    if (a.window > 0) {
        const int end = q.first + (a.causal ? 1 : 0);
        lo = end > a.window ? end - a.window : 0;
    }
    q.page_lo = lo / KV8_PAGE;
    q.page_hi = (kv + KV8_PAGE - 1) / KV8_PAGE;
    const int pages = q.page_hi > q.page_lo ? q.page_hi - q.page_lo : 0;
    q.tiles = (int)(((long long)q.n * a.group + a.tile - 1) >> a.tile_log2);
    const int most = a.caps[31 - __clz(pages | 1)];
    q.len = (pages + most - 1) / most;
    if (q.len < 1) q.len = 1;
    q.splits = (pages + q.len - 1) / q.len;
    if (q.splits < 1) q.splits = 1;
    return q;
}

// One unit of work: a row tile, a kv head and a split of the tile's pages.
struct Item {
    int s, tile, kh, split;
    int p0, p1;         // pages [p0, p1)
    int lo, hi;         // keys that some row of the tile sees: [lo, hi)
    int in_lo, in_hi;   // keys that every row of the tile sees: [in_lo, in_hi)
};

__device__ __forceinline__ void row_keys(const Kv8AttnArgs& a, const Seq& q, int i, int* lo, int* hi) {
    const int pos = q.first + i;
    *lo = 0;
    if (a.causal) {
        *hi = pos + 1;
        if (a.window > 0 && pos + 1 > a.window) *lo = pos + 1 - a.window;
    } else {
        *hi = q.kv;
        if (a.window > 0 && q.first > a.window) *lo = q.first - a.window;
    }
    if (*hi < 0) *hi = 0;
}

__device__ __forceinline__ Item item_of(const Kv8AttnArgs& a, const Seq& q, int s, int idx) {
    Item it;
    it.s = s;
    const unsigned rest = (unsigned)idx / (unsigned)q.splits, top = rest / (unsigned)a.n_kv;
    it.split = idx - (int)rest * q.splits;
    it.kh = (int)(rest - top * (unsigned)a.n_kv);
    // under the causal mask the last rows have the most keys: they go first
    it.tile = q.tiles - 1 - (int)top;
    const int i0 = (int)((unsigned)(it.tile * a.tile) / (unsigned)a.group);
    int i1 = (int)((unsigned)(it.tile * a.tile + a.tile - 1) / (unsigned)a.group);
    if (i1 > q.n - 1) i1 = q.n - 1;
    int lo0, hi0, lo1, hi1;
    row_keys(a, q, i0, &lo0, &hi0);
    row_keys(a, q, i1, &lo1, &hi1);
    it.lo = lo0;
    it.hi = hi1;
    it.in_lo = lo1;
    it.in_hi = hi0;
    int p0 = q.page_lo + it.split * q.len, p1 = p0 + q.len;
    if (p1 > q.page_hi) p1 = q.page_hi;
    const int tp0 = it.lo / KV8_PAGE, tp1 = (it.hi + KV8_PAGE - 1) / KV8_PAGE;
    it.p0 = p0 > tp0 ? p0 : tp0;
    it.p1 = p1 < tp1 ? p1 : tp1;
    if (it.p1 < it.p0) it.p1 = it.p0;
    return it;
}

// What a CTA's warps need of an item; one warp finds it for all.
struct Work {
    Seq q;
    Item w;
    int item;           // -1: no more
};

// The finding warp's state: lane i holds the items before the i-th group of
// `per` sequences.
struct Finder {
    int per, cum, total;
    Seq q;              // of this lane's sequence where per is 1,
    int s;              // and its index
};

__device__ __forceinline__ int items_of(const Kv8AttnArgs& a, const Seq& q) { return q.tiles * a.n_kv * q.splits; }

// Sums of counts that stay at the largest int: row starts may be anything.
__device__ __forceinline__ int add_counts(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); }

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = add_counts(v, u);
    }
    return v;
}

__device__ __forceinline__ Finder make_finder(const Kv8AttnArgs& a, int lane) {
    Finder f;
    f.per = (a.S + 31) / 32;
    int mine = 0;
    f.q = Seq{};
    for (int s = lane * f.per; s < a.S && s < (lane + 1) * f.per; ++s) {
        f.q = seq_of(a, s);
        mine = add_counts(mine, items_of(a, f.q));
    }
    f.s = lane;
    if (f.per == 1 && a.S > 1) {
        // up to 32 sequences: those with the longest items go first, so that no
        // long one is begun at the end (a bitonic sort; equal ones in order)
        uint32_t key = (uint32_t)f.q.len << 5 | (uint32_t)(31 - lane);
#pragma unroll
        for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
            for (int j = k >> 1; j > 0; j >>= 1) {
                const uint32_t o = __shfl_xor_sync(0xffffffffu, key, j);
                key = ((lane & k) == 0) == ((lane & j) == 0) ? max(key, o) : min(key, o);
            }
        const int from = 31 - (int)(key & 31);
        int* d = reinterpret_cast<int*>(&f.q);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Seq) / 4); ++i) d[i] = __shfl_sync(0xffffffffu, d[i], from);
        mine = __shfl_sync(0xffffffffu, mine, from);
        f.s = from;
    }
    const int inc = warp_inclusive(mine, lane);
    f.cum = inc - mine;
    f.total = __shfl_sync(0xffffffffu, inc, 31);
    // sequences whose rows overlap can ask for any number of items: above what
    // the call's rows can make nothing is done
    if (f.total > a.ticket_cap * a.split_cap) {
        report(a.err, DERR_INDEX, SITE_LEN);
        f.total = 0;
    }
    return f;
}

// By the whole warp: item `item` (below the total), the same in all lanes.
__device__ __forceinline__ Work find_item(const Kv8AttnArgs& a, const Finder& f, int item, int lane) {
    // the last group that begins at or before it
    const int group = __popc(__ballot_sync(0xffffffffu, f.cum <= item)) - 1;
    int idx = item - __shfl_sync(0xffffffffu, f.cum, group);
    int s0 = group * f.per;
    const int end = s0 + f.per < a.S ? s0 + f.per : a.S;
    Work k;
    k.item = item;
    if (f.per == 1) {              // the group's only sequence
        int* d = reinterpret_cast<int*>(&k.q);
        const int* src = reinterpret_cast<const int*>(&f.q);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Seq) / 4); ++i) d[i] = __shfl_sync(0xffffffffu, src[i], group);
        k.w = item_of(a, k.q, __shfl_sync(0xffffffffu, f.s, group), idx);
        return k;
    }
    while (true) {
        Seq q{};
        int n = 0;
        if (s0 + lane < end) {
            q = seq_of(a, s0 + lane);
            n = items_of(a, q);
        }
        const int inc = warp_inclusive(n, lane);
        const unsigned at = __ballot_sync(0xffffffffu, idx < inc);
        if (at || s0 + 32 >= end) {
            const int l = at ? __ffs(at) - 1 : 0;
            idx -= __shfl_sync(0xffffffffu, inc - n, l);
            int* d = reinterpret_cast<int*>(&k.q);
            const int* src = reinterpret_cast<const int*>(&q);
#pragma unroll
            for (int i = 0; i < (int)(sizeof(Seq) / 4); ++i) d[i] = __shfl_sync(0xffffffffu, src[i], l);
            k.w = item_of(a, k.q, s0 + l, idx);
            return k;
        }
        idx -= __shfl_sync(0xffffffffu, inc, 31);
        s0 += 32;
    }
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What a part of a row's keys leaves (kv8_attn.cu): outputs relative to 2^M, -inf
// without keys, and the sum l of the softmax relative to 2^Z.  Any Z near the
// part's largest score does; a NaN sum stays one.
__device__ __forceinline__ float sum_ref(float M, float Z) { return M == -INFINITY ? -INFINITY : Z; }
__device__ __forceinline__ float part_of(float l, float Z, float z) { return l == 0.f ? 0.f : l * ex2(Z - z); }
// The factor of outputs relative to 2^M: zeros for a row that sees no key.
__device__ __forceinline__ float out_factor(float M, float Z, float l) { return l == 0.f ? 0.f : ex2(M - Z) / l; }
__device__ __forceinline__ float row_lse(float Z, float l) {
    return l == 0.f ? -INFINITY : (Z + log2f(l)) * 0.6931471805599453f;
}

// Scales that a page can have (the append's are powers of two from 2^-100 to
// 2^119; K's may be 0, which makes all its scores 0).
__device__ __forceinline__ bool scales_fit(float k, float v) { return k >= 0.f && k < INFINITY && v > 0.f && v < INFINITY; }
// V scales that let outputs and sum share one reference.
__device__ __forceinline__ bool near(float scale) { return scale >= 0x1p-32f && scale <= 0x1p32f; }
// From this factor between weights on values and the sum's on, the former are zeros in f16.
constexpr float FAR_PAGE = 0x1p40f;

// Two e4m3 codes (the low 16 bits) to a pair of f16, exactly.
__device__ __forceinline__ uint32_t f16_of_codes(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(two));
    return h;
}

// Four codes with NaN ones as zeros; `seen` collects that there were some.
__device__ __forceinline__ uint32_t drop_nan(uint32_t w, uint32_t* seen) {
    const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // codes 0x7f and 0xff
    *seen |= m;
    return w & ~((m >> 7) * 0xffu);
}

// Byte offset of 16-byte chunk c of key row r in a tile that TMA wrote with
// the 128-byte (head_dim 128) or 64-byte (head_dim 64) swizzle.
template <int HD>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return HD == 128 ? swz128(r, c) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Which of dims d0 .. d0 + n - 1 (bits, n <= 32) have a NaN code in V among the
// keys that row qi of the idx-th item of sequence s sees, in the pages that not
// all of the item's rows see whole.  Rarely called: the item is found again, so
// that its numbers need not stay in registers.
template <int HD>
__device__ __noinline__ uint32_t nan_dims(const Kv8AttnArgs& a, int s, int idx, int qi, int d0, int n) {
    const Seq q = seq_of(a, s);
    const Item w = item_of(a, q, s, idx);
    if (qi >= q.n) return 0;
    int klo, khi;
    row_keys(a, q, qi, &klo, &khi);
    uint32_t m = 0;
#pragma unroll 1
    for (int p = w.p0; p < w.p1; ++p) {
        const int key0 = p * KV8_PAGE, pg = a.table[(size_t)s * a.max_pages + p];
        if ((key0 >= w.in_lo && key0 + KV8_PAGE <= w.in_hi) || pg < 0 || pg >= a.n_pages) continue;
        const size_t at = (size_t)pg * a.n_kv + w.kh;
        if (!scales_fit(a.k_scale[at], a.v_scale[at])) continue;
        const int k1 = khi - key0 < KV8_PAGE ? khi - key0 : KV8_PAGE;
#pragma unroll 1
        for (int k = klo > key0 ? klo - key0 : 0; k < k1; ++k)
            for (int d = 0; d < n; ++d)
                m |= (uint32_t)((a.v_codes[(at * KV8_PAGE + k) * HD + d0 + d] & 0x7f) == 0x7f) << d;
    }
    return m;
}

// A row of q's power-of-two factor: `inv` brings its largest finite element
// into [1, 2), `back` undoes it.
__device__ __forceinline__ void row_factor(float top, float* inv, float* back) {
    uint32_t e = __float_as_uint(top) >> 23;       // biased exponent
    e = e < 1 ? 1 : (e > 253 ? 253 : e);
    *inv = top > 0.f ? __uint_as_float((254 - e) << 23) : 1.f;
    *back = top > 0.f ? __uint_as_float(e << 23) : 1.f;
}

}  // namespace kv8
}  // namespace dfl
