// Attention over the 8-bit paged KV cache.
//
//   o[r] = sum_j w_rj v_j / sum_j w_rj,  w_rj = exp(scale * q_r . k_j)
// over the keys j that row r sees, k_j and v_j = code * (their page's scale).
//
// Rows of one kv head's q heads share its keys, so a tile's rows are (row,
// q head of the group) pairs, packed row-major.  Scores are kept in base 2.
// With page scales kp, vp (vp = 2^e for the cache's own scales) a page adds
//   P = 2^(t + log2 vp - M),  O += P * vcode,  l += (sum P) / vp
// with t the scores times kp and M the running maximum of t + log2 vp less 15: P
// is the key's weight on the value codes, at most 2^15, so it fits f16 whatever
// the scales; l carries the plain softmax sum relative to 2^M in fp32.
// A page with a small scale (of zeros: 2^-100) counts in l however little it
// adds to O, so one reference does only while the scales lie within 2^-32 and
// 2^32: a weight is then lost from l below 2^-60 of the largest.  From the first
// page on with another scale l is kept relative to 2^Z, Z the running maximum of
// t, and takes (sum P) 2^(M - log2 vp - Z); where that factor passes 2^40, P are
// zeros in f16 anyway, and l takes the sum of 2^(t - Z).  Parts (warps, groups,
// splits) are joined as (M, Z, l), the row is O * 2^(M - Z) / l.
//
// q enters the MMAs as f16: a row is scaled by the power of two that brings
// its largest element into [1, 2) (folded into the score factor), which keeps
// bf16 and f16 rows exact but for elements 2^-14 below the row's largest,
// that lose low bits.  e4m3 codes are exact in f16.  P is rounded to f16: half
// a step, 2^-12 to 2^-11 of the weight, while that is above 2^-29 of the largest
// weight times scale of the row (tcgen05 form: 2^-21), below 2^-25 of a step of
// that, to nothing at 2^-40 (2^-32).  l has the weights before they are rounded.
// Scores, sums and outputs are fp32.
//
// This form: 16 packed rows a tile, mma.sync (a tcgen05 tile would be an
// eighth full at best, and a page's work is its bytes).  A warp takes whole
// pages, so its warps never meet inside an item, and one TMA warp keeps 11
// (head_dim 64: 22) pages in flight, 176 KB of an SM's shared memory.  Bound by
// DRAM at many sequences: 19 of 16384 positions, 8 kv heads of 128, 119 us =
// 5.4 TB/s (0.79 of a measured copy; 32 of 4096 to 16384 159 us, 4.6 TB/s, as
// the last items run alone), by latency at few: one of 1088 10.7 us, of which
// the launch, finding the item, tables, pages and the fold are a chain of
// about eight trips to memory.
//
// Splits, items and the tcgen05 form's cases: kv8_attn_plan below.

#include <mutex>

#include "attention_dev.cuh"
#include "kv8_attn_dev.cuh"
#include "tc_dev.cuh"

namespace dfl {
namespace {

using adev::ldsm_x4_trans;
using namespace kv8;

constexpr float ROOM = 15.f;        // log2 of the largest P: f16 ends at 2^16, and what lies far below should count
constexpr int KT = 16;              // packed rows of a tile (the M side of the MMAs)
constexpr int KW = 8;               // consumer warps; each takes whole pages, every eighth
constexpr int KC = 32 * KW;         // consumer threads
constexpr int KTHREADS = KC + 32;
template <int HD> constexpr int stages() { return HD == 128 ? 11 : 22; }   // pages in flight: 176 KB

template <int HD> constexpr int tile_bytes() { return KV8_PAGE * HD; }
template <int HD> constexpr int red_ld() { return HD + 16; }   // row pitch of the merge buffer (floats)

template <int HD> struct KvSmem {
    static constexpr int ring = 0;
    static constexpr int red = ring + stages<HD>() * 2 * tile_bytes<HD>();
    static constexpr int ml = red + KW / 2 * KT * red_ld<HD>() * 4;    // half of the warps at a time
    static constexpr int scales = ml + KW / 2 * KT * 4 * 4;  // [stages] (k, v)
    static constexpr int bars = scales + stages<HD>() * 8;   // full, empty
    static constexpr int items = bars + stages<HD>() * 16;   // item ring: full, empty
    static constexpr int work = items + 2 * 16;
    static constexpr int flag = work + 2 * sizeof(Work);
    static constexpr size_t bytes = 1024 + flag + 16;
};

// Key of MMA column n (0..7) inside a group of 8: for 128-byte rows columns
// 2j, 2j + 1 are keys j, j + 4, whose swizzled chunks lie in different bank
// halves; 64-byte rows need no reordering.
template <int HD>
__device__ __forceinline__ int key_of(int n) { return HD == 128 ? (n >> 1) + 4 * (n & 1) : n; }

template <typename T>
__device__ __forceinline__ void store_row4(T* p, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void store_row4<__nv_bfloat16>(__nv_bfloat16* p, float a, float b, float c, float d) {
    uint2 v{pack_bf16x2(a, b), pack_bf16x2(c, d)};
    *reinterpret_cast<uint2*>(p) = v;
}
template <>
__device__ __forceinline__ void store_row4<__half>(__half* p, float a, float b, float c, float d) {
    uint2 v{pack_f16x2(a, b), pack_f16x2(c, d)};
    *reinterpret_cast<uint2*>(p) = v;
}

// A warp's rows g and g + 8 of a tile: q, the keys they see, and what its pages
// have left of them.
template <int HD> struct Rows {
    uint32_t qa[HD / 16][4];
    float fr[2];                // score factors
    int klo[2], khi[2];
    float M[2], l[2], Z[2];     // l relative to 2^M, in far_pages to 2^Z
    float o[HD / 8][4];
};

// Page p of item w; false: before its first use (FARS: the form for any scale, the
// other one ends at a page that is not near()), or at the end (flag[1]).
template <int HD, bool FARS>
__device__ __forceinline__ bool take_page(const Kv8AttnArgs& a, const Item& w, uint8_t* sm, unsigned base,
                                          unsigned n_items, int p, Rows<HD>& u) {
    using S_ = KvSmem<HD>;
    constexpr int TB = tile_bytes<HD>(), KSTAGES = stages<HD>();
    const float2* scales = reinterpret_cast<const float2*>(sm + S_::scales);
    uint64_t *full = reinterpret_cast<uint64_t*>(sm + S_::bars), *empty = full + KSTAGES;
    volatile int* flag = reinterpret_cast<volatile int*>(sm + S_::flag);
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const unsigned it = base + (p - w.p0);
    const int st = it % KSTAGES;
    if (flag[1]) return false;
    if (!__all_sync(0xffffffffu, mbar_wait(full + st, (it / KSTAGES) & 1))) {
        report(a.err, DERR_TIMEOUT, SITE_FULL);
        flag[1] = 1;
        return false;
    }
    const float2 sc = scales[st];
    const uint8_t* kt = sm + S_::ring + st * 2 * TB;
    uint8_t* vt = sm + S_::ring + st * 2 * TB + TB;
    const int key0 = p * KV8_PAGE;
    if (sc.x >= 0.f && sc.y > 0.f) {
        if (!FARS && !near(sc.y)) return false;
        float s[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) {
                const uint4 kk = lds128(kt + tile_off<HD>(8 * t + key_of<HD>(g), 4 * h + c));
                const uint32_t kw[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b[2] = {f16_of_codes(kw[j]), f16_of_codes(kw[j] >> 16)};
                    mma_f16_16816(s[t], u.qa[4 * h + j], b);
                }
            }
        const float ev = log2f(sc.y);
        const bool whole = key0 >= w.in_lo && key0 + KV8_PAGE <= w.in_hi;
        const float f0 = u.fr[0] * sc.x, f1 = u.fr[1] * sc.x;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = fmaf(s[t][e], e < 2 ? f0 : f1, ev);
                if (!whole) {
                    const int key = key0 + 8 * t + key_of<HD>(2 * c + (e & 1));
                    if (key < u.klo[e >> 1] || key >= u.khi[e >> 1]) x = -INFINITY;
                }
                s[t][e] = x;
                mx[e >> 1] = fmaxf(mx[e >> 1], x);
            }
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            if (FARS) {
                const float z = fmaxf(u.Z[r], mx[r] - ev);
                if (z != u.Z[r] && u.Z[r] != -INFINITY) u.l[r] *= ex2(u.Z[r] - z);
                u.Z[r] = z;
            }
            mx[r] = fmaxf(mx[r] - ROOM, u.M[r]);
            alpha[r] = mx[r] == u.M[r] ? 1.f : ex2(u.M[r] - mx[r]);   // M = -inf: 0
            u.M[r] = mx[r];
        }
        float m0 = u.M[0] == -INFINITY ? 0.f : u.M[0], m1 = u.M[1] == -INFINITY ? 0.f : u.M[1];
        float k[2];                          // weights on values to the sum's
        bool lost[2] = {false, false};
        if (FARS) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                k[r] = u.M[r] == -INFINITY ? 0.f : ex2(u.M[r] - ev - u.Z[r]);
                if (k[r] > FAR_PAGE) {
                    lost[r] = true;
                    k[r] = 1.f;
                    (r ? m1 : m0) = u.Z[r] + ev;
                }
            }
        }
        float sum[2] = {0.f, 0.f};
        uint32_t pa[4][4];      // P of the four 16-key steps, as A fragments
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float p0 = ex2(s[t][0] - m0), p1 = ex2(s[t][1] - m0);
            const float p2 = ex2(s[t][2] - m1), p3 = ex2(s[t][3] - m1);
            sum[0] += p0 + p1;
            sum[1] += p2 + p3;
            pa[t >> 1][2 * (t & 1)] = pack_f16x2(p0, p1);
            pa[t >> 1][2 * (t & 1) + 1] = pack_f16x2(p2, p3);
        }
        const float iv = 1.f / sc.y;
        u.l[0] = FARS ? fmaf(sum[0], k[0], u.l[0]) : fmaf(sum[0], iv, u.l[0] * alpha[0]);
        u.l[1] = FARS ? fmaf(sum[1], k[1], u.l[1]) : fmaf(sum[1], iv, u.l[1] * alpha[1]);
        if (FARS) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) pa[x][e] = lost[e & 1] ? 0u : pa[x][e];
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int d = 0; d < HD / 8; ++d) {
                u.o[d][0] *= alpha[0];
                u.o[d][1] *= alpha[0];
                u.o[d][2] *= alpha[1];
                u.o[d][3] *= alpha[1];
            }
        }
        // a key's V must not reach a row that does not see it, and 0 * NaN is NaN:
        // where not all rows see all keys, codes that no row sees and NaN ones
        // are taken as zeros, and the rows that see a NaN get it after the merge
        uint32_t seen = 0;
        if (!whole) {
#pragma unroll 1
            for (int x = lane; x < KV8_PAGE * HD / 16; x += 32) {
                const int key = x / (HD / 16);
                uint4* at = reinterpret_cast<uint4*>(vt + tile_off<HD>(key, x % (HD / 16)));
                const uint32_t keep = key0 + key >= w.lo && key0 + key < w.hi ? 0xffffffffu : 0u;
                const uint4 y = *at;
                *at = make_uint4(drop_nan(y.x & keep, &seen), drop_nan(y.y & keep, &seen),
                                 drop_nan(y.z & keep, &seen), drop_nan(y.w & keep, &seen));
            }
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // V: matrices (keys 0-7 | 8-15 of the step) x (16-byte chunks d, d + 1),
            // transposed in units of two codes: a register holds dims 2g, 2g + 1 of
            // keys 2c, 2c + 1; one byte permute pairs the keys of each dim
            const int vrow = 16 * k + 8 * ((lane >> 3) & 1) + key_of<HD>(lane & 7);
#pragma unroll
            for (int d = 0; d < HD / 16; d += 2) {
                uint32_t r[4];
                ldsm_x4_trans(r, vt + tile_off<HD>(vrow, d + (lane >> 4)));
#pragma unroll
                for (int x = 0; x < 4; ++x) r[x] = __byte_perm(r[x], 0, 0x3120);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t be[2] = {f16_of_codes(r[2 * x]), f16_of_codes(r[2 * x + 1])};
                    const uint32_t bo[2] = {f16_of_codes(r[2 * x] >> 16), f16_of_codes(r[2 * x + 1] >> 16)};
                    mma_f16_16816(u.o[2 * (d + x)], pa[k], be);
                    mma_f16_16816(u.o[2 * (d + x) + 1], pa[k], bo);
                }
            }
        }
        if (!whole) {
            if (seen) flag[3] = n_items + 1;
            tc::fence_async_smem();     // the next copy into this page comes after the zeros
        }
    }
    // the page goes back once its codes have arrived: an arrival can
    // overtake loads that are still queued
    __threadfence_block();
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + st);
    return true;
}

// The pages from p on once the V scales of the warp's pages lie far apart (top of
// this file).  A call, so that usual pages keep their registers and their place
// in the instruction cache (inline: one token of one sequence 10.9 us for 10.4).
template <int HD>
__device__ __noinline__ void far_pages(const Kv8AttnArgs& a, const Item& w, uint8_t* sm, unsigned base, unsigned n_items,
                                       int p, Rows<HD>* rows) {
    Rows<HD>& u = *rows;
    u.Z[0] = u.M[0];
    u.Z[1] = u.M[1];
    while (p < w.p1 && take_page<HD, true>(a, w, sm, base, n_items, p, u)) p += KW;
}

template <typename T, int HD>
__global__ void __launch_bounds__(KTHREADS, 1)
kv8_attn_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ Kv8AttnArgs a) {
    using S_ = KvSmem<HD>;
    constexpr int TB = tile_bytes<HD>(), KSTAGES = stages<HD>();
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    float* red = reinterpret_cast<float*>(sm + S_::red);
    float* ml = reinterpret_cast<float*>(sm + S_::ml);
    float2* scales = reinterpret_cast<float2*>(sm + S_::scales);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + S_::bars);
    uint64_t* empty = full + KSTAGES;
    uint64_t* i_full = reinterpret_cast<uint64_t*>(sm + S_::items);   // [2] items on their way to the consumers
    uint64_t* i_empty = i_full + 2;
    Work* ring = reinterpret_cast<Work*>(sm + S_::work);
    // [0] last arriver, [1] a wait ran out, [2] there is a next item, [3] the last item (count) with NaN codes to look up
    volatile int* flag = reinterpret_cast<volatile int*>(sm + S_::flag);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_trigger();
    if (tid == 0) {
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
        for (int i = 0; i < KSTAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(i_full + i, 1);
            mbar_init(i_empty + i, KW);
        }
        fence_mbar_init();
        flag[1] = 0;
        flag[3] = 0;
    }
    pdl_wait();
    Finder f{};
    Work first;
    first.item = -1;
    if (warp == KW) {      // the first item, while the barriers are made ready
        f = make_finder(a, lane);
        if ((int)blockIdx.x < f.total) first = find_item(a, f, (int)blockIdx.x, lane);
    }
    __syncthreads();

    if (warp == KW) {
        // ---- producer: pages of every item of this CTA, in order.  The lanes
        // look up 32 pages and their scales at a time, the next 32 while lane 0
        // issues these.
        unsigned it = 0;
        bool ok = true;
        Work wk = first;
        for (unsigned k = 0; ok; ++k) {
            const int item = wk.item;
            int asked = 0;
            if (lane == 0) {
                if (k >= 2 && !mbar_wait(i_empty + (k & 1), ((k >> 1) - 1) & 1)) {
                    report(a.err, DERR_TIMEOUT, SITE_EMPTY);
                    flag[1] = 1;
                } else {
                    ring[k & 1] = wk;
                    mbar_arrive(i_full + (k & 1));
                }
                if (item >= 0) asked = ask_item(a, f.total);
            }
            if (item < 0) break;
            const Item w = wk.w;
            auto look = [&](int b, int* page, float* ks, float* vs) {
                *page = -1;
                *ks = -1.f;
                *vs = 1.f;
                if (b + lane >= w.p1) return;
                const int pg = a.table[(size_t)w.s * a.max_pages + b + lane];
                if (pg < 0 || pg >= a.n_pages) {
                    report(a.err, DERR_INDEX, SITE_PAGE);   // its keys are left out
                    return;
                }
                *page = pg;
                *ks = a.k_scale[(size_t)pg * a.n_kv + w.kh];
                *vs = a.v_scale[(size_t)pg * a.n_kv + w.kh];
            };
            int page, next_page;
            float ks, vs, next_ks, next_vs;
            look(w.p0, &page, &ks, &vs);
            for (int b = w.p0; b < w.p1 && ok; b += 32) {
                look(b + 32, &next_page, &next_ks, &next_vs);
                if (page >= 0 && !scales_fit(ks, vs)) {      // not in look, which would wait for the scales
                    report(a.err, DERR_INDEX, SITE_SCALE);
                    page = -1;
                    ks = -1.f;
                }
                const int m = w.p1 - b < 32 ? w.p1 - b : 32;
                for (int j = 0; j < m; ++j) {
                    const int pg = __shfl_sync(0xffffffffu, page, j);
                    const float kj = __shfl_sync(0xffffffffu, ks, j), vj = __shfl_sync(0xffffffffu, vs, j);
                    const int st = it % KSTAGES;
                    bool issued = true;
                    if (lane == 0) {
                        if (it >= KSTAGES && !mbar_wait(empty + st, (it / KSTAGES - 1) & 1)) {
                            report(a.err, DERR_TIMEOUT, SITE_EMPTY);
                            flag[1] = 1;
                            issued = false;
                        } else {
                            scales[st] = make_float2(kj, vj);
                            uint8_t* kt = sm + S_::ring + st * 2 * TB;
                            if (pg >= 0) {
                                mbar_arrive_expect_tx(full + st, 2 * TB);
                                const int y = (pg * a.n_kv + w.kh) * KV8_PAGE;
                                tma_load_2d(kt, &k_map, full + st, 0, y);
                                tma_load_2d(kt + TB, &v_map, full + st, 0, y);
                            } else {
                                mbar_arrive(full + st);
                            }
                        }
                    }
                    if (!__shfl_sync(0xffffffffu, (int)issued, 0)) {
                        ok = false;
                        break;
                    }
                    ++it;
                    ok = __shfl_sync(0xffffffffu, flag[1], 0) == 0;
                    if (!ok) break;
                }
                page = next_page;
                ks = next_ks;
                vs = next_vs;
            }
            int next = lane == 0 ? settle_item(a, f.total, asked) : 0;
            next = __shfl_sync(0xffffffffu, next, 0);
            wk.item = -1;
            if (next >= 0) wk = find_item(a, f, next, lane);
        }
        // no copy of this CTA is in flight when it ends
        if (lane == 0) {
            const unsigned n = it < KSTAGES ? it : KSTAGES;
            for (unsigned i = it - n; i < it; ++i) mbar_wait(full + i % KSTAGES, (i / KSTAGES) & 1);
        }
        return;
    }

    // ---- consumers
    const int g = lane >> 2, c = lane & 3;
    unsigned base = 0;   // pages of the items before
    for (unsigned n_items = 0;; ++n_items) {
        // the next item, the same for all warps; a wait that ran out ends the CTA
        // (err says so)
        const int slot_i = n_items & 1;
        if (warp == 0) {
            const bool got = __all_sync(0xffffffffu, !flag[1] && mbar_wait(i_full + slot_i, (n_items >> 1) & 1));
            if (lane == 0) {
                if (!got && !flag[1]) {
                    report(a.err, DERR_TIMEOUT, SITE_FULL);
                    flag[1] = 1;
                }
                flag[2] = got;
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(KC) : "memory");   // the merge buffer is free again, too
        if (!flag[2]) break;
        const Work wk = ring[slot_i];
        __threadfence_block();     // read before the slot goes back
        __syncwarp();
        if (lane == 0) mbar_arrive(i_empty + slot_i);
        if (wk.item < 0) break;
        const Seq& q = wk.q;
        const Item& w = wk.w;
        const int item = wk.item;

        // q of rows g, g + 8 as A fragments: k step (h, j) of 16 covers the
        // dims 64 h + 16 c + 4 j .. + 3 of every lane c of a quad, so a
        // lane's fragments are its own 16 consecutive dims
        Rows<HD> u;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int pr = w.tile * KT + g + 8 * r;
            const int i = pr / a.group, hq = w.kh * a.group + pr % a.group;
            const bool real = i < q.n;
            float v[HD / 4];
            float top = 0.f;
            if (real) {
                const T* src = reinterpret_cast<const T*>(a.q) + (long long)(q.r0 + i) * a.q_row + (long long)hq * a.q_head;
#pragma unroll
                for (int h = 0; h < HD / 64; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 e = *reinterpret_cast<const uint4*>(src + 64 * h + 16 * c + 8 * k);
                        const T* ev = reinterpret_cast<const T*>(&e);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[16 * h + 8 * k + j] = to_f32(ev[j]);
                    }
                row_keys(a, q, i, &u.klo[r], &u.khi[r]);
            } else {
#pragma unroll
                for (int j = 0; j < HD / 4; ++j) v[j] = 0.f;
                u.klo[r] = 0;
                u.khi[r] = 0x7fffffff;   // computed on zeros, never written
            }
#pragma unroll
            for (int j = 0; j < HD / 4; ++j) {
                const float x = fabsf(v[j]);
                top = fmaxf(top, x < INFINITY ? x : 0.f);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float inv, back;
            row_factor(top, &inv, &back);
            u.fr[r] = back * a.scale_log2;
#pragma unroll
            for (int h = 0; h < HD / 64; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u.qa[4 * h + j][r] = pack_f16x2(v[16 * h + 4 * j] * inv, v[16 * h + 4 * j + 1] * inv);
                    u.qa[4 * h + j][2 + r] = pack_f16x2(v[16 * h + 4 * j + 2] * inv, v[16 * h + 4 * j + 3] * inv);
                }
        }

#pragma unroll
        for (int r = 0; r < 2; ++r) {
            u.M[r] = -INFINITY;
            u.l[r] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < HD / 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) u.o[d][e] = 0.f;

        int p = w.p0 + warp;
        while (p < w.p1 && take_page<HD, false>(a, w, sm, base, n_items, p, u)) p += KW;
        if (p < w.p1) {
            const Item far_w = w;      // copies: what a call names lies in memory
            Rows<HD> v = u;
            far_pages<HD>(a, far_w, sm, base, n_items, p, &v);
            u = v;
        } else {
            u.Z[0] = u.M[0];
            u.Z[1] = u.M[1];
        }
        base += w.p1 - w.p0;

        // ---- the warps' pages merged: the upper half into the lower half's
        // registers, then the lower half row by row, in warp order
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            u.l[r] += __shfl_xor_sync(0xffffffffu, u.l[r], 1);
            u.l[r] += __shfl_xor_sync(0xffffffffu, u.l[r], 2);
        }
        constexpr int HW = KW / 2;
        auto put = [&](int slot) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (c == 0) *reinterpret_cast<float4*>(ml + (slot * KT + g + 8 * r) * 4) = make_float4(u.M[r], u.Z[r], u.l[r], 0.f);
                float* dst = red + (slot * KT + g + 8 * r) * red_ld<HD>() + 4 * c;
#pragma unroll
                for (int d = 0; d < HD / 16; ++d)
                    *reinterpret_cast<float4*>(dst + 16 * d) =
                        make_float4(u.o[2 * d][2 * r], u.o[2 * d + 1][2 * r], u.o[2 * d][2 * r + 1], u.o[2 * d + 1][2 * r + 1]);
            }
        };
        if (w.p1 - w.p0 > HW) {
            if (warp >= HW) put(warp - HW);
            asm volatile("bar.sync 1, %0;" ::"n"(KC) : "memory");
            if (warp < HW) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float4 b = *reinterpret_cast<const float4*>(ml + (warp * KT + g + 8 * r) * 4);
                    const float m = fmaxf(u.M[r], b.x), z = fmaxf(u.Z[r], b.y);
                    const float fa = u.M[r] == -INFINITY ? 0.f : ex2(u.M[r] - m), fb = b.x == -INFINITY ? 0.f : ex2(b.x - m);
                    u.l[r] = part_of(u.l[r], u.Z[r], z) + part_of(b.z, b.y, z);
                    u.M[r] = m;
                    u.Z[r] = z;
                    const float* src = red + (warp * KT + g + 8 * r) * red_ld<HD>() + 4 * c;
#pragma unroll
                    for (int d = 0; d < HD / 16; ++d) {
                        const float4 x = *reinterpret_cast<const float4*>(src + 16 * d);
                        u.o[2 * d][2 * r] = fmaf(x.x, fb, u.o[2 * d][2 * r] * fa);
                        u.o[2 * d + 1][2 * r] = fmaf(x.y, fb, u.o[2 * d + 1][2 * r] * fa);
                        u.o[2 * d][2 * r + 1] = fmaf(x.z, fb, u.o[2 * d][2 * r + 1] * fa);
                        u.o[2 * d + 1][2 * r + 1] = fmaf(x.w, fb, u.o[2 * d + 1][2 * r + 1] * fa);
                    }
                }
            }
            asm volatile("bar.sync 1, %0;" ::"n"(KC) : "memory");
        }
        if (warp < HW) put(warp);
        asm volatile("bar.sync 1, %0;" ::"n"(KC) : "memory");
        constexpr int NF = HD / 64;                       // float4s of a thread
        const int row = tid >> 4, col = (tid & 15) * 4;   // columns col + 64 k
        const int pr = w.tile * KT + row;
        const int qi = pr / a.group, hq = w.kh * a.group + pr % a.group;
        const bool real = qi < q.n;
        float fm = -INFINITY, fz = -INFINITY, fl = 0.f;
        float4 fo[NF];
#pragma unroll
        for (int k = 0; k < NF; ++k) fo[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < HW; ++v) {
            const float4 x = *reinterpret_cast<const float4*>(ml + (v * KT + row) * 4);
            fm = fmaxf(fm, x.x);
            fz = fmaxf(fz, x.y);
        }
#pragma unroll
        for (int v = 0; v < HW; ++v) {
            const float4 mzl = *reinterpret_cast<const float4*>(ml + (v * KT + row) * 4);
            const float f = fm == -INFINITY ? 0.f : ex2(mzl.x - fm);
            fl += part_of(mzl.z, mzl.y, fz);
#pragma unroll
            for (int k = 0; k < NF; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(red + (v * KT + row) * red_ld<HD>() + col + 64 * k);
                fo[k].x = fmaf(x.x, f, fo[k].x);
                fo[k].y = fmaf(x.y, f, fo[k].y);
                fo[k].z = fmaf(x.z, f, fo[k].z);
                fo[k].w = fmaf(x.w, f, fo[k].w);
            }
        }
        if (flag[3] == (int)n_items + 1) {
            const int idx = ((q.tiles - 1 - w.tile) * a.n_kv + w.kh) * q.splits + w.split;
#pragma unroll
            for (int k = 0; k < NF; ++k) {
                const uint32_t m = nan_dims<HD>(a, w.s, idx, qi, col + 64 * k, 4);
                const float nan = __int_as_float(0x7fffffff);
                if (m & 1) fo[k].x = nan;
                if (m & 2) fo[k].y = nan;
                if (m & 4) fo[k].z = nan;
                if (m & 8) fo[k].w = nan;
            }
        }
        bool write = true;
        if (q.splits > 1) {
            // partial of this split; the last split to arrive folds them all,
            // in split order
            const long long slot0 = (long long)item - w.split;   // splits of a tile are neighbours
            const long long tk = ((long long)q.r0 * a.group / KT + w.s + w.tile) * a.n_kv + w.kh;
            const bool fits = slot0 + q.splits <= a.part_cap && tk < a.ticket_cap;   // by the plan's bounds
            constexpr int PL = KT * (HD + 4);   // floats of a partial: outputs, then (max, sum) pairs
            if (fits && real) {
                float* dst = a.part + (slot0 + w.split) * PL;
#pragma unroll
                for (int k = 0; k < NF; ++k)
                    *reinterpret_cast<float4*>(dst + row * HD + col + 64 * k) = fo[k];
                if ((tid & 15) == 0) *reinterpret_cast<float4*>(dst + KT * HD + row * 4) = make_float4(fm, fz, fl, 0.f);
            }
            __threadfence();
            asm volatile("bar.sync 1, %0;" ::"n"(KC) : "memory");
            if (tid == 0) flag[0] = fits && atomicAdd(a.tickets + tk, 1) == q.splits - 1;
            asm volatile("bar.sync 1, %0;" ::"n"(KC) : "memory");
            write = flag[0] != 0;
            if (write) {
                __threadfence();
                if (tid == 0) a.tickets[tk] = 0;
                fm = fz = -INFINITY;
                fl = 0.f;
#pragma unroll
                for (int k = 0; k < NF; ++k) fo[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (real) {
                    const float* src = a.part + slot0 * PL;
                    // four splits' loads in flight, the maximum running along: a pass for
                    // it alone would be one more trip to memory
#pragma unroll 1
                    for (int v0 = 0; v0 < q.splits; v0 += 4) {
                        float4 x[4], y[4][NF];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const bool in = v0 + v < q.splits;
                            const float* from = src + (size_t)(v0 + v) * PL;
                            x[v] = in ? __ldcg(reinterpret_cast<const float4*>(from + KT * HD + row * 4))
                                      : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
#pragma unroll
                            for (int k = 0; k < NF; ++k)
                                y[v][k] = in ? __ldcg(reinterpret_cast<const float4*>(from + row * HD + col + 64 * k))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        const float m = fmaxf(fm, fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)));
                        const float z = fmaxf(fz, fmaxf(fmaxf(x[0].y, x[1].y), fmaxf(x[2].y, x[3].y)));
                        const float g = fm == -INFINITY ? 0.f : ex2(fm - m);
                        fl = part_of(fl, fz, z);
#pragma unroll
                        for (int k = 0; k < NF; ++k) fo[k] = make_float4(fo[k].x * g, fo[k].y * g, fo[k].z * g, fo[k].w * g);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const float f = x[v].x == -INFINITY ? 0.f : ex2(x[v].x - m);
                            fl += part_of(x[v].z, x[v].y, z);
#pragma unroll
                            for (int k = 0; k < NF; ++k) {
                                fo[k].x = fmaf(y[v][k].x, f, fo[k].x);
                                fo[k].y = fmaf(y[v][k].y, f, fo[k].y);
                                fo[k].z = fmaf(y[v][k].z, f, fo[k].z);
                                fo[k].w = fmaf(y[v][k].w, f, fo[k].w);
                            }
                        }
                        fm = m;
                        fz = z;
                    }
                }
            }
        }
        if (write && real) {
            const float inv = out_factor(fm, fz, fl);
            T* dst = reinterpret_cast<T*>(a.out) + (long long)(q.r0 + qi) * a.out_row + (long long)hq * a.out_head;
#pragma unroll
            for (int k = 0; k < NF; ++k)
                store_row4<T>(dst + col + 64 * k, fo[k].x * inv, fo[k].y * inv, fo[k].z * inv, fo[k].w * inv);
            if (a.lse && (tid & 15) == 0)
                a.lse[(long long)(q.r0 + qi) * a.n_q + hq] = row_lse(fz, fl);
        }
    }
}

template <typename T, int HD>
int launch_t(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a, int sms, cudaStream_t s) {
    const size_t smem = KvSmem<HD>::bytes;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv8_attn_kernel<T, HD>));
    if (e != cudaSuccess) return (int)e;
    const long long most = a.ticket_cap * a.split_cap;   // items there can be
    const long long grid = most < sms ? most : sms;
    return (int)launch_k(kv8_attn_kernel<T, HD>, dim3((unsigned)grid), dim3(KTHREADS), smem, s, k_map, v_map, a);
}

}  // namespace

// The largest dynamic shared memory, allowed once per kernel and device.
cudaError_t allow_smem(const void* kern) {
    static std::mutex mu;
    constexpr int MAX = 128;
    static const void* kerns[MAX];
    static int devs[MAX], n = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n; ++i)
        if (kerns[i] == kern && devs[i] == dev) return cudaSuccess;
    int most = 0;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)fa.sharedSizeBytes);
    if (e == cudaSuccess && n < MAX) {
        kerns[n] = kern;
        devs[n++] = dev;
    }
    return e;
}

// The form of a call, by its packed rows (rows x q heads of a kv head) per
// sequence: the mma.sync kernel's 16-row tiles up to 16, a tile whose two
// softmax groups take alternate keys up to 128 (64 rows where a block of 16
// rows fits, as sequences differ and a second tile reads the keys again; 128
// else), two 128-row tiles over the same keys above.  While items are few, the
// next smaller tiles are the faster ones though they read the keys again: more
// SMs have work, and a small tile's own chain is shorter.  Microseconds at 8 kv
// heads of 128, by the smaller tile (and its items) and the larger:
//   rows of a call          positions   smaller tile       larger
//   1 x 32 packed                4000   16 (16 items) 14.6  64  20.4
//   1 x 64                       4000   16 (32)       17.8  64  21.5
//   1 x 64                      16384   16 (32)       37.5  64  33.8
//   16 x 32                      4000   16 (256)      70.4  64  42.5
//   1 x 256                      8000   64 (32)       30.9  128 33.9
//   1 x 512                      8000   64 (64)       45.1  128 41.5
//   2 x 1024                     8000   128 (128)     97.0  256 99.0
//   2 x 2048                     8000   128 (256)    184.6  256 159.2
// so 16-row tiles up to a sixth of the SMs, 64-row ones up to a quarter,
// 128-row ones up to all of them.
//
// Both this and the splits of a tile's pages follow from the call's row,
// sequence and head counts and the sequence's own length alone: its results
// do not depend on what the other sequences hold.
Kv8AttnPlan kv8_attn_plan(int rows, int S, int n_q, int n_kv, int head_dim, int max_pages, int sms) {
    Kv8AttnPlan p;
    const int group = n_q / n_kv;
    const long long packed = (long long)rows * group;
    const long long each = (packed + S - 1) / S;
    // items of a split each: were all rows dealt evenly, and at most
    auto even = [&](int tile) { return S * ((each + tile - 1) / tile) * n_kv; };
    auto most = [&](int tile) { return S == 1 ? even(tile) : (packed / tile + S) * n_kv; };
    p.form = KV8_TC_KEYS;
    long long at_once;
    if (each <= KT || most(KT) * 6 <= sms) {
        p.form = KV8_MMA;
        p.tile = KT;
        at_once = each <= KT ? even(KT) : most(KT);
    } else if (each <= 64 && 16 * group <= 64) {
        p.tile = 64;
        at_once = even(64);
    } else if (most(64) * 4 <= sms) {
        p.tile = 64;
        at_once = most(64);
    } else if (each <= 128) {
        p.tile = 128;
        at_once = even(128);
    } else if (most(128) <= sms) {
        p.tile = 128;
        at_once = most(128);
    } else {
        p.form = KV8_TC_ROWS;
        p.tile = 256;
        at_once = even(256);
    }
    if (at_once < 1) at_once = 1;
    const long long tiles = packed / p.tile + S;           // slots: floor(first packed row / tile) + sequence
    // Splits of a sequence with P pages (a value for each power of two): as many
    // as let every item start at once, an SM each, but not below 4 (6) pages an
    // item.  An item behind another one costs far more than its pages: 8
    // sequences of 16384 positions, 8 kv heads: 74, 104, 84 us with 2, 3, 4
    // splits for single tokens, 92, 129, 109 us for 16 rows; one of 6000: 49,
    // 25, 18 us with 1, 4, 16.  Where more items than SMs wait anyway, single tokens
    // of long sequences are halved all the same, so that the last items are short:
    // 32 of 4096 to 16384 positions 180 -> 159 us (equal ones of 10000: 162 -> 180).
    const long long once = at_once < sms ? sms / at_once : 1, least = p.form == KV8_MMA ? 4 : 6;
    long long cap = 1;
    for (int b = 0; b < 32; ++b) {
        long long c = (1LL << b) / least;
        if (c > once) c = once;
        if (c > 64) c = 64;
        if (at_once > sms && p.form == KV8_MMA && b >= 7) c = 2;
        p.caps[b] = (uint8_t)(c < 1 || tiles * n_kv > KV8_TICKETS ? 1 : c);
        if ((1LL << b) <= max_pages && p.caps[b] > cap) cap = p.caps[b];
    }
    p.split_cap = (int)cap;
    p.ticket_cap = tiles * n_kv;
    p.part_cap = cap > 1 ? tiles * n_kv * cap : 0;
    // the tickets' place is the same in every call, so that calls of different
    // shapes can share a workspace: none's partials lie where another counts
    p.ticket_bytes = cap > 1 ? KV8_TICKETS * 4 : 0;
    p.bytes = KV8_QUEUE_BYTES + p.ticket_bytes + (size_t)p.part_cap * p.tile * (head_dim + 4) * 4;
    return p;
}

int launch_kv8_attention(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a,
                         int form, int head_dim, int sms, cudaStream_t s) {
    if (form != KV8_MMA) return launch_kv8_attention_tc(k_map, v_map, a, head_dim, sms, s);
    if (a.dtype == 1)
        return head_dim == 128 ? launch_t<__nv_bfloat16, 128>(k_map, v_map, a, sms, s)
                               : launch_t<__nv_bfloat16, 64>(k_map, v_map, a, sms, s);
    return head_dim == 128 ? launch_t<__half, 128>(k_map, v_map, a, sms, s)
                           : launch_t<__half, 64>(k_map, v_map, a, sms, s);
}

}  // namespace dfl
