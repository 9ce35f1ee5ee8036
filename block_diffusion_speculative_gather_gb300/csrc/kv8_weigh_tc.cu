// Accumulated attention weight for many rows a sequence, on the fifth-generation
// tensor cores (tcgen05).  The mathematics is the one stated in kv8_weigh.cu.
//
// Scores are K q^T tiles in tensor memory: 128 cached keys (two pages) are the
// lanes, up to 128 (row, q head) pairs of one kv head the columns, so a key's sum
// stays within a thread, and neither its scale nor its total ever leaves it.  K's
// codes become the f16 or bf16 operand (exactly: they have four significant bits),
// whichever type the rows have, so these come by TMA as they stand, in boxes of
// whole rows x the kv head's q heads.  NaN or any other numbers in rows that are no
// item's stay in their own columns, whose lse stands as inf: they add nothing.
//
// A CTA per SM takes a run of neighbouring items (128 keys of a sequence, all kv
// heads).  Roles: a thread brings K's codes and the tiles of rows, four warps
// convert K, a thread issues the MMAs, and two groups of four warps take the
// tiles in turn, one thread to a key: 128 columns of tensor memory, an
// exponential each, summed.  Each group has two tiles of tensor memory, so that the
// next one's scores are there when it comes.  Bound by the exponentials (16 a
// cycle and SM: 1024 cycles a tile, whose MMAs take 512) and the instructions around
// them where rows are many: the last 64 rows of four prompts behind up to 8192 positions (32
// heads on 8) take 24.6 us, 144 items on 152 CTAs.  About 11 us pass before the first
// columns (tables, tensor memory, the first keys) and on eight heads' keys, then a tile
// takes 0.8 to 0.9 us where its exponentials need 0.54 (32 rows 16.4 us, 128 38.8, 256 65).
// Few rows: the work on a head's keys, their way in (two places) and conversion.

#include <type_traits>

#include "capi_internal.cuh"
#include "f32x2.cuh"
#include "gemm.cuh"
#include "kv8.cuh"
#include "kv8_attn_dev.cuh"
#include "kv8_weigh_dev.cuh"
#include "tc_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;

constexpr int TILE = 128;                      // keys of an item, columns of a tile at most
constexpr int CONV_WARP = 8, CONV = 4, ISSUE_WARP = 12, TCT = 32 * 14;      // and a warp that loads
constexpr int SITE_WEIGH = 340;                // + role

template <int HD> struct TcWeighSmem {
    static constexpr int QS = HD == 128 ? 3 : 4;               // tiles of rows in flight
    static constexpr int QB = TILE * HD * 2, KB = TILE * HD * 2, RB = TILE * HD;
    static constexpr int q = 0, k = q + QS * QB, raw = k + 2 * KB;       // raw: K's codes of two heads
    static constexpr int col = raw + 2 * RB;                             // [2 groups][2][128] -lse in base 2
    static constexpr int part = col + 4 * TILE * 4;                      // [2][128] the second group's sums
    static constexpr int bars = part + 2 * TILE * 4;
    static constexpr int n_bars = 2 * QS + 4 + 4 + 8 + 1;
    static constexpr int misc = bars + n_bars * 8;                       // tensor-memory base, abort flag
    static constexpr int sums = misc + 16;
    static constexpr int before = sums + 64;
    static constexpr size_t bytes(int S) { return 1024 + before + ((size_t)S + 1) * 4; }
};

// Bounded wait that gives up early once another role has given up.
__device__ __forceinline__ bool wait_or(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int site) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (clock64() - t0 > WAIT_CYCLES) {
            report(err, DERR_TIMEOUT, site);
            *abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// What every role goes through alike: the items of the CTA, and of each its tiles
// of rows [t0, t1) (those that some key of the item can be seen from).
struct Walk {
    int item, last, s;
    Span q;
    int key0, packed, t0, t1;
};

__device__ __forceinline__ void walk_to(const Kv8WeighArgs& a, const int* before, int per_tile, Walk& w) {
    if (w.item >= before[w.s + 1]) {
        do ++w.s;
        while (w.item >= before[w.s + 1]);
        w.q = span_of(a, w.s, false);
    }
    w.key0 = (w.q.lo / TILE + (w.item - before[w.s])) * TILE;
    w.packed = (w.q.i1 - w.q.i0) * a.group;
    w.t0 = 0;
    w.t1 = (w.packed + per_tile - 1) / per_tile;
    if (a.causal && w.packed > 0) {
        // rows from which the item's first key is seen, and with a window its last one
        const long long from = (long long)w.key0 - w.q.first - w.q.i0;
        if (from > 0) w.t0 = (int)min(from * a.group / per_tile, (long long)w.t1);
        if (a.window > 0) {
            const long long to = (from + TILE - 1 + a.window) * a.group;        // behind the last such pair
            w.t1 = to <= 0 ? w.t0 : (int)min((to + per_tile - 1) / per_tile, (long long)w.t1);
            if (w.t1 < w.t0) w.t1 = w.t0;
        }
    }
}

// The item's page e (0, 1) as an index into the pool; -1: no position of it counts.
__device__ __forceinline__ int item_page(const Kv8WeighArgs& a, const Walk& w, int e, bool tell) {
    const int k = w.key0 + e * KV8_PAGE;
    if (!(k < w.q.hi && k + KV8_PAGE > w.q.lo)) return -1;
    const int pg = a.table[(size_t)w.s * a.max_pages + k / KV8_PAGE];
    if (pg >= 0 && pg < a.n_pages) return pg;
    if (tell) report(a.err, DERR_INDEX, SITE_PAGE);
    return -1;
}

template <typename T, int HD>
__global__ void __launch_bounds__(TCT, 1)
kv8_weigh_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ Kv8WeighArgs a) {
    using L = TcWeighSmem<HD>;
    constexpr int QS = L::QS;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint64_t *q_full = bars, *q_empty = bars + QS, *r_full = bars + 2 * QS, *r_empty = r_full + 2, *k_full = r_full + 4,
             *k_empty = r_full + 6, *s_full = r_full + 8, *s_free = r_full + 12, *drain = r_full + 16;
    uint32_t* tmem_base = reinterpret_cast<uint32_t*>(sm + L::misc);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::misc + 4);
    int* before = reinterpret_cast<int*>(sm + L::before);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform, so each role's code is
    const int rows_tile = TILE / a.group, per_tile = rows_tile * a.group;

    pdl_trigger();
    if (tid == 0) {
        tma_prefetch_desc(&q_map);
        for (int i = 0; i < QS; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(r_full + i, 1);
            mbar_init(r_empty + i, CONV);
            mbar_init(k_full + i, CONV);
            mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_free + i, 4);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        *abort = 0;
    }
    if (warp == ISSUE_WARP) tc::tmem_alloc(tmem_base, 512);
    pdl_wait();
    const Run run = my_items<TILE, TCT>(a, before, reinterpret_cast<int*>(sm + L::sums));
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_base, 0);
    Walk w;
    w.s = run.s;
    w.last = run.last;
    w.q = span_of(a, w.s, false);
    auto wait = [&](uint64_t* bar, unsigned parity, int role) { return wait_or(bar, parity & 1, abort, a.err, SITE_WEIGH + role); };

    if (warp < 8) {
        // ---------------------------------------------------------- exponentials
        const int t = warp >> 2, r = tid & 127;      // group, key of the item
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        float* col = reinterpret_cast<float*>(sm + L::col) + t * 2 * TILE;
        float* part = reinterpret_cast<float*>(sm + L::part);
        unsigned n = 0;                              // tiles so far
        bool ok = true;
        // once a wait has run out these warps go on to the end without waiting, so that
        // none stays behind at a barrier
        for (w.item = run.first; w.item < run.last; ++w.item) {
            walk_to(a, before, per_tile, w);
            const int pg = item_page(a, w, r / KV8_PAGE, t == 0 && r % KV8_PAGE == 0), j = w.key0 + r;
            float* wp = a.weights + (size_t)max(pg, 0) * KV8_PAGE + r % KV8_PAGE;
            const bool mine = pg >= 0 && j < w.q.kv;
            float old = 0.f;
            if (t == 0 && mine && !(a.fresh && j >= w.q.first)) old = *wp;
            // pairs that see the key: [from, to)
            int from = 0, to = w.packed;
            if (a.causal) {
                const long long i = (long long)j - w.q.first - w.q.i0;
                from = (int)min(max(i, 0ll) * a.group, (long long)w.packed);
                if (a.window > 0) to = (int)min(max(i + a.window, 0ll) * a.group, (long long)w.packed);
            } else if (a.window > 0 && j < (long long)w.q.first - a.window) {
                to = 0;
            }
            if (!mine || to < from) from = to = 0;
            const int tiles = w.t1 - w.t0, all = tiles * a.n_kv;
            // lse of column r of a tile of head h (-inf: it does not count)
            const int ri = r / a.group, rg = r - ri * a.group;
            auto lse_at = [&](int h, int tile) {
                if (r >= per_tile || tile * per_tile + r >= w.packed) return -INFINITY;
                return a.lse[(long long)(w.q.r0 + w.q.i0 + tile * rows_tile + ri) * a.n_q + h * a.group + rg];
            };
            auto scale_of = [&](int h) { return pg >= 0 && h < a.n_kv ? a.k_scale[(size_t)pg * a.n_kv + h] : 0.f; };
            const int idx0 = (int)((n & 1) != (unsigned)t);        // this group's first tile of the item
            int h = 0, tile = w.t0 + idx0, head = -1;              // the tile at hand
            if (tile >= w.t1) tile -= tiles, ++h;
            float scale = 0.f, next_scale = scale_of(0), lse = idx0 < all ? lse_at(h, tile) : 0.f;
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            for (int idx = idx0; idx < all; idx += 2) {
                const unsigned m = n + idx;                        // the CTA's m-th tile
                float* cl = col + ((m >> 1) & 1) * TILE;
                cl[r] = lse > -INFINITY ? lse * -1.4426950408889634f : -INFINITY;
                // the next one's; what it loads is not used before
                const int c0 = tile * per_tile, now = h;
                tile += 2;
                while (tile >= w.t1) tile -= tiles, ++h;
                if (idx + 2 < all) lse = lse_at(h, tile);
                while (head < now) {
                    scale = next_scale;
                    ++head;
                    next_scale = scale_of(head + 1);
                }
                if (!(scale >= 0.f && scale < INFINITY)) {
                    report(a.err, DERR_INDEX, SITE_SCALE);
                    scale = __int_as_float(0x7fffffff);            // scores that add nothing
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
                if (ok) ok = __all_sync(0xffffffffu, wait(s_full + (m & 3), m >> 2, 0));
                if (!ok) continue;
                tc::fence_after_sync();
                const float f = scale * a.scale_log2;
                const float2 f2 = make_float2(f, f);
                const bool whole = __all_sync(0xffffffffu, from <= c0 && to >= min(c0 + per_tile, w.packed));
                const int cols = (min(per_tile, w.packed - c0) + 31) / 32 * 2;      // by 16
                // 16 columns: their scores, then their weights, side by side
                auto take = [&](int b, uint32_t (&d)[16]) {
                    float2 u[8];
#pragma unroll
                    for (int x = 0; x < 8; x += 2) {
                        const float4 l = *reinterpret_cast<const float4*>(cl + 16 * b + 2 * x);
                        u[x] = fma2(make_float2(__uint_as_float(d[2 * x]), __uint_as_float(d[2 * x + 1])), f2, make_float2(l.x, l.y));
                        u[x + 1] = fma2(make_float2(__uint_as_float(d[2 * x + 2]), __uint_as_float(d[2 * x + 3])), f2, make_float2(l.z, l.w));
                    }
                    if (!whole) {
                        const int at = c0 + 16 * b - from;
                        const unsigned seen = (unsigned)(to - from);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            if ((unsigned)(at + 2 * x) >= seen) u[x].x = -200.f;
                            if ((unsigned)(at + 2 * x + 1) >= seen) u[x].y = -200.f;
                        }
                    }
                    // a NaN score (a NaN code) adds nothing: 2^-200 is 0
#pragma unroll
                    for (int x = 0; x < 8; ++x) u[x] = make_float2(ex2(fmaxf(u[x].x, -200.f)), ex2(fmaxf(u[x].y, -200.f)));
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[x] = add2(acc[x], add2(u[x], u[x + 4]));
                };
                uint32_t d0[16], d1[16];
                const uint32_t sc = tm + (m & 3) * TILE + lanes;
                tc::ld_x16_async(sc, d0);
                for (int b = 0; b < cols; b += 2) {            // 16 columns are on their way while 16 are summed
                    tc::ld_wait16(d0);
                    tc::ld_x16_async(sc + 16 * (b + 1), d1);
                    take(b, d0);
                    tc::ld_wait16(d1);
                    if (b + 2 < cols) {
                        tc::ld_x16_async(sc + 16 * (b + 2), d0);
                    } else {
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free + (m & 3));
                    }
                    take(b + 1, d1);
                }
            }
            n += all;
            // the second group's sums to the first
            const int par = w.item & 1;
            const float2 both = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
            const float sum = both.x + both.y;
            if (t == 1) part[par * TILE + r] = sum;
            asm volatile("bar.sync 3, 256;" ::: "memory");
            if (t == 0 && mine && ok) *wp = old + (sum + part[par * TILE + r]);
        }
    } else if (warp < ISSUE_WARP) {
        // ---------------------------------------------------------- K's codes to operands
        const int cw = warp - CONV_WARP;
        unsigned kn = 0;                             // heads so far
        bool ok = true;
        for (w.item = run.first; ok && w.item < run.last; ++w.item) {
            walk_to(a, before, per_tile, w);
            if (w.t1 <= w.t0) continue;
            for (int h = 0; ok && h < a.n_kv; ++h, ++kn) {
                const int b = kn & 1;
                ok = __all_sync(0xffffffffu, wait(r_full + b, kn >> 1, 1));
                if (ok && kn >= 2) ok = __all_sync(0xffffffffu, wait(k_empty + b, (kn >> 1) - 1, 1));
                if (!ok) break;
                const uint8_t* src = sm + L::raw + b * L::RB;
                uint8_t* dst = sm + L::k + b * L::KB;
                constexpr int CH = HD / 16, ALL = TILE * CH / (32 * CONV), N = 4;    // 16-byte chunks of a key, of a lane
#pragma unroll
                for (int i0 = 0; i0 < ALL; i0 += N) {
                    uint4 x[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) x[i] = lds128(src + (((i0 + i) * CONV + cw) * 32 + lane) * 16);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int at = ((i0 + i) * CONV + cw) * 32 + lane, key = at / CH, ch = at % CH;
                        const uint32_t e[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            o[2 * k] = f16_of_codes(e[k]);
                            o[2 * k + 1] = f16_of_codes(e[k] >> 16);
                        }
                        if constexpr (!std::is_same<T, __half>::value) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
                                o[k] = pack_bf16x2(v.x, v.y);
                            }
                        }
                        uint8_t* d = dst + (ch >> 2) * TILE * 128;
                        *reinterpret_cast<uint4*>(d + swz128(key, 2 * (ch & 3))) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(d + swz128(key, 2 * (ch & 3) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
                tc::fence_async_smem();
                __threadfence_block();               // the codes have been read before their place goes back
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(r_empty + b);
                    mbar_arrive(k_full + b);
                }
            }
        }
    } else if (warp == ISSUE_WARP) {
        // ---------------------------------------------------------- MMAs
        unsigned n = 0, kn = 0;
        bool ok = true;
        for (w.item = run.first; ok && w.item < run.last; ++w.item) {
            walk_to(a, before, per_tile, w);
            if (w.t1 <= w.t0) continue;
            for (int h = 0; ok && h < a.n_kv; ++h, ++kn) {
                ok = __all_sync(0xffffffffu, wait(k_full + (kn & 1), kn >> 1, 2));
                for (int tile = w.t0; ok && tile < w.t1; ++tile, ++n) {
                    const int stage = n % QS;
                    ok = __all_sync(0xffffffffu, wait(q_full + stage, n / QS, 2));
                    if (ok && n >= 4) ok = __all_sync(0xffffffffu, wait(s_free + (n & 3), (n >> 2) - 1, 2));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const int left = min(per_tile, w.packed - tile * per_tile);
                    const int cols = (left + 31) & ~31;
                    const uint32_t idesc = std::is_same<T, __half>::value ? tc::idesc_f16_f32(TILE, cols) : tc::idesc_bf16_f32(TILE, cols);
                    if (tc::elect_one()) {
                        const uint8_t* kp = sm + L::k + (kn & 1) * L::KB;
                        const uint8_t* qp = sm + L::q + stage * L::QB;
#pragma unroll
                        for (int x = 0; x < HD / 16; ++x)
                            tc::mma_f16(tm + (n & 3) * TILE, tc::desc_sw128(kp + (x >> 2) * TILE * 128 + (x & 3) * 32),
                                        tc::desc_sw128(qp + (x >> 2) * TILE * 128 + (x & 3) * 32), idesc, x > 0);
                        tc::commit(q_empty + stage);
                        tc::commit(s_full + (n & 3));
                        if (tile == w.t1 - 1) tc::commit(k_empty + (kn & 1));
                    }
                    __syncwarp();
                }
            }
        }
        // every MMA has finished before tensor memory is given back, those too whose readers gave up
        if (tc::elect_one()) tc::commit(drain);
        __syncwarp();
        mbar_wait(drain, 0);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- loads
        if (lane == 0) {
            unsigned n = 0, kn = 0;
            bool ok = true;
            const uint32_t box = (uint32_t)per_tile * 128;           // bytes of 64 dims
            for (w.item = run.first; ok && w.item < run.last; ++w.item) {
                walk_to(a, before, per_tile, w);
                if (w.t1 <= w.t0) continue;
                const int pg[2] = {item_page(a, w, 0, false), item_page(a, w, 1, false)};
                for (int h = 0; ok && h < a.n_kv; ++h, ++kn) {
                    const int b = kn & 1;
                    if (kn >= 2) ok = wait(r_empty + b, (kn >> 1) - 1, 3);
                    if (!ok) break;
                    const uint32_t there = (pg[0] >= 0) + (pg[1] >= 0);
                    if (there) {
                        mbar_arrive_expect_tx(r_full + b, there * (L::RB / 2));
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (pg[e] >= 0)
                                bulk_load_1d(sm + L::raw + b * L::RB + e * (L::RB / 2),
                                             a.k_codes + ((size_t)pg[e] * a.n_kv + h) * KV8_PAGE * HD, L::RB / 2, r_full + b);
                    } else {
                        mbar_arrive(r_full + b);
                    }
                    for (int tile = w.t0; ok && tile < w.t1; ++tile, ++n) {
                        const int stage = n % QS;
                        if (n >= (unsigned)QS) ok = wait(q_empty + stage, n / QS - 1, 3);
                        if (!ok) break;
                        mbar_arrive_expect_tx(q_full + stage, box * (HD / 64));
#pragma unroll
                        for (int x = 0; x < HD / 64; ++x)
                            tma_load_3d(sm + L::q + stage * L::QB + x * TILE * 128, &q_map, q_full + stage, 64 * x, h * a.group,
                                        w.q.r0 + w.q.i0 + tile * rows_tile);
                    }
                }
            }
            // no copy of this CTA is in flight when it ends
            for (unsigned i = n < (unsigned)QS ? 0 : n - QS; i < n; ++i) mbar_wait(q_full + i % QS, (i / QS) & 1);
            for (unsigned i = kn < 2 ? 0 : kn - 2; i < kn; ++i) mbar_wait(r_full + (i & 1), (i >> 1) & 1);
        }
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == ISSUE_WARP) tc::tmem_dealloc(tm, 512);
}

template <typename T, int HD>
int launch_tc(const CUtensorMap& q_map, const Kv8WeighArgs& a, int sms, cudaStream_t s) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv8_weigh_tc_kernel<T, HD>));
    if (e != cudaSuccess) return (int)e;
    const long long most = (long long)a.S * ((a.max_pages + 1) / 2);   // items
    return (int)launch_k(kv8_weigh_tc_kernel<T, HD>, dim3((unsigned)(most < sms ? most : sms)), dim3(TCT),
                         TcWeighSmem<HD>::bytes(a.S), s, q_map, a);
}

}  // namespace

// From this many (row, q head) pairs of a kv head a sequence on, of the call's rows (its
// padding among them) on average.  32 heads on 8, bf16, caches that are not in L2, in us by
// this form and by kv8_weigh.cu: 32 sequences of 8000 positions, 4 pairs 107, 50; 16 pairs 107,
// 89; 20 pairs 107, 120; 64 pairs 112, 264.  8 of them, 16 pairs 35, 29; 20 pairs 35, 38; one, 12
// pairs 12.7, 13.9.  One of 1088, 8 pairs 10.9, 8.6; 16 pairs 10.9, 11.6; 64 pairs 11.6, 30.  f16:
// 32 of 8000, 20 pairs 102, 102; 32 pairs 103, 124.
constexpr int TC_PAIRS = 20;

bool kv8_weigh_by_tc(const Kv8WeighArgs& a) {
    long long rows = a.rows / a.S;
    if (a.observe > 0 && rows > a.observe) rows = a.observe;
    // a tensor map's strides are above 0 and below 2^40 bytes
    const bool fits = a.q_row > 0 && a.q_head > 0 && a.q_row < (1LL << 39) && a.q_head < (1LL << 39);
    return fits && rows * a.group >= TC_PAIRS;
}

int launch_kv8_weigh_tc(const CUtensorMap& q_map, const Kv8WeighArgs& a, int head_dim, int sms, cudaStream_t s) {
    if (a.dtype == 1)
        return head_dim == 128 ? launch_tc<__nv_bfloat16, 128>(q_map, a, sms, s) : launch_tc<__nv_bfloat16, 64>(q_map, a, sms, s);
    return head_dim == 128 ? launch_tc<__half, 128>(q_map, a, sms, s) : launch_tc<__half, 64>(q_map, a, sms, s);
}

}  // namespace dfl
