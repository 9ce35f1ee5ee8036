// Attention over the 8-bit paged cache for many rows per kv head, on the
// fifth-generation tensor cores (tcgen05).  The mathematics is the one stated
// in kv8_attn.cu.
//
// A CTA per SM takes items (row tile, kv head, split of the pages).  Its two
// softmax groups of four warps, one thread to a row, each own a 128 x 128
// score tile and an output accumulator in tensor memory:
//   ROWS form (more than 128 packed rows a sequence): the groups take two
//     128-row tiles of q over the same keys, which are converted once;
//   KEYS form: both take the same rows and alternate 128-key steps; at the
//     item's end each takes half of the columns of both sums from tensor
//     memory.  Up to 64 packed rows a tile holds each row twice, and a copy's
//     thread takes one of the step's two pages (a third less time a step).
// Roles: two warps bring the pages' K and V codes by TMA and look up pages and
// scales; four warps turn a step's K codes (two pages) into an f16 operand
// tile, four its V codes into a transposed one (keys contiguous; with two warps
// each a verify of 8 sequences took 110 us instead of 75); one issues the MMAs:
// S = Q K^T, then O += P V with P read from tensor memory, where the softmax
// warps wrote it over the scores.  While one group's softmax runs, the
// tensor core works for the other.
//
// Bound: a 128-key step of 128 rows takes about 1900 cycles where its MMAs
// take 1030 (tensor pipe 37 % busy; 41 % with two tiles over the same keys).
// Each group waits in a chain (scores, softmax 1500 cycles, P V, the next
// scores), shared memory moves 224 KB a step (codes in and out, f16 tiles in,
// operands out: 1750 cycles at 128 bytes), and the roles' code together
// exceeds the instruction cache, so what a step rarely needs is kept out of
// its unrolled loops: masks as a pass over tensor memory before it instead of
// selects in it took a tenth off prompt chunks.  19 sequences x 16 rows x 16384
// positions, 32 heads of 128: 140 us (580 TFLOP/s, 4.6 TB/s); 4 ragged prompt
// chunks of up to 2048 rows behind 6000: 496 us (910 TFLOP/s).  An item also costs
// about 10 us beside its steps: found, its first pages brought, its sums
// joined and written.
//
// The reference of a row's weights is set 2^ROOM below its maximum and moves only
// when that rises by more than 2^LAZY (weights stay within f16's range), so
// outputs are rescaled in tensor memory rarely.  When one row of a warp moves,
// all whose maximum has risen do, as the warp's outputs are rewritten anyway, but
// only while all rows have seen the same keys: a row's bits must not follow from
// keys that it does not see.  Room below the largest weight costs rescales; 4
// prompt chunks, verify of 8 sequences, 32 draft blocks, in us, by ROOM and LAZY,
// rows moving together everywhere:
//   3, 12: 484, 75.0, 27.3;  5, 10: 491, 75.1, 27.6;  7, 8: 500, 75.3, 28.0;
//   9, 6: 519, 76.2, 29.5 (rows moving one by one 581, 83.9, 34.2)
// and as it stands 496, 76.8, 28.4.
// (7: keys of 2^-21 of the largest weight keep their 11 bits, 2^-32 is lost.)
//
// Tensor memory: scores at columns 0 and 128, outputs at 256 and 384.  A
// step's P overwrites its scores (32 keys' weights in the first 16 of their
// 32 columns), and the next step's scores overwrite P: the two MMAs are
// issued in that order by one thread.

#include <type_traits>

#include "attention_dev.cuh"
#include "kv8_attn_dev.cuh"
#include "tc_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;
using adev::ldsm_x4_trans;

// Warps: 0-7 softmax, then K's conversion, V's, the MMA issuer and two loaders.
constexpr int KC_WARP = 8, KC = 4, VC_WARP = 12, VC = 4, MMA_WARP = 16, TMA_K = 17, TC_THREADS = 32 * 19;
constexpr int STEP = 2 * KV8_PAGE;         // keys of a step
constexpr int SITE_TC = 310;               // + role
constexpr float ROOM = 7.f, LAZY = 8.f;    // base 2; sum at most 15

template <int HD, bool KEYS, int DUP> struct TcSmem {
    static constexpr int QB = 128 * HD * 2;                    // one q tile, f16
    static constexpr int QR = KEYS ? QB : 2 * QB;
    static constexpr int KB = STEP * HD * 2;                   // one step's K (or V), f16
    static constexpr int PB = KV8_PAGE * HD;                   // one page's K (or V) codes
    static constexpr int RAW = HD == 64 ? 8 : (KEYS ? 4 : 2);  // pages in flight, K and V each
    static constexpr int q = 0, k = q + QR, v = k + 2 * KB, raw = v + 2 * KB;
    static constexpr int ml = raw + RAW * 2 * PB;              // rows' factors; at the item's end the copies' (max, sum)
    static constexpr int steps = ml + 1024;                    // [8] step scales
    static constexpr int rsc = steps + 8 * 32;                 // [RAW] page scales
    static constexpr int rscv = rsc + RAW * 8;
    static constexpr int bars = rscv + RAW * 8;
    static constexpr int n_bars = 4 * RAW + 8 + 2 + 6 + 1 + 1 + 4 + 3 + 2;
    static constexpr int work = bars + n_bars * 8;             // [2] items
    static constexpr int misc = work + 2 * sizeof(Work);       // tensor-memory base, abort flag, last arriver
    static constexpr int nans = misc + 16;                     // [4] items with NaN codes to look up: (count, s, idx, tile)
    static constexpr size_t bytes = 1024 + nans + 64;
};

// Of the two pages of a step: K scale (negative: no keys), log2 and reciprocal of
// V's.  far: V scales of this step or an earlier one of the item are not near();
// then ks are negative and iv are the K scales.
struct StepScale {
    float ks[2], ev[2], iv[2], far, pad_;
};

__device__ __forceinline__ void stsm_x4(void* p, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(smem_u32(p)), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

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

// Steps of an item, and of them those of softmax group t.
template <bool KEYS>
__device__ __forceinline__ int group_steps(const Kv8AttnArgs& a, const Seq& q, const Item& w, int t) {
    const int n = (w.p1 - w.p0 + 1) / 2;
    if (KEYS) return t == 0 ? (n + 1) / 2 : n / 2;
    return t == 0 || (long long)q.n * a.group - (long long)w.tile * 256 > 128 ? n : 0;
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16], float f) {
    // column n of a 16-column block holds dim 2 (n % 8) + n / 8 (the order the
    // transposed V was written in)
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = sizeof(T) == 2 && std::is_same<T, __half>::value ? pack_f16x2(v[i] * f, v[8 + i] * f)
                                                              : pack_bf16x2(v[i] * f, v[8 + i] * f);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// NaN into a thread's outputs (tensor memory at o) where its row sees NaN codes
// of the item that `rec` names.
template <int HD, bool KEYS, int DUP>
__device__ __noinline__ void put_nans(const Kv8AttnArgs& a, const volatile int* rec, int t, int r, uint32_t o) {
    const int s = rec[1], idx = rec[2], qi = (rec[3] * a.tile + (KEYS ? 0 : t * 128) + (DUP == 2 ? r & 63 : r)) / a.group;
    for (int b = KEYS && t == 1 ? HD / 32 : 0; b < (KEYS && t == 0 ? HD / 32 : HD / 16); ++b) {
        const uint32_t m = nan_dims<HD>(a, s, idx, qi, 16 * b, 16);
        __syncwarp();
        uint32_t y[16];
        tc::ld_x16(o + b * 16, y);
#pragma unroll
        for (int n = 0; n < 16; ++n)      // the columns' order: store16
            if ((m >> (2 * (n & 7) + (n >> 3))) & 1) y[n] = 0x7fffffffu;
        tc::st_x16(o + b * 16, y);
    }
    tc::st_wait();
}

template <typename T, int HD, bool KEYS, int DUP>
__global__ void __launch_bounds__(TC_THREADS, 1)
kv8_attn_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                   const __grid_constant__ Kv8AttnArgs a) {
    using L = TcSmem<HD, KEYS, DUP>;
    constexpr int R = L::RAW, PB = L::PB;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    StepScale* steps = reinterpret_cast<StepScale*>(sm + L::steps);
    float2* rsc = reinterpret_cast<float2*>(sm + L::rsc);     // with K's pages and with V's
    float2* rscv = reinterpret_cast<float2*>(sm + L::rscv);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint64_t *rawk_full = bars, *rawk_empty = bars + R, *rawv_full = bars + 2 * R, *rawv_empty = bars + 3 * R,
             *k_full = bars + 4 * R, *k_empty = k_full + 2, *v_full = k_full + 4, *v_empty = k_full + 6,
             *q_full = k_full + 8, *q_free = q_full + 1, *s_full = q_full + 2, *p_full = q_full + 4,
             *o_done = q_full + 6, *handed = q_full + 8, *drain = q_full + 9, *i_full = q_full + 10,
             *i_empty = q_full + 12, *copy_full = q_full + 14, *copy_free = q_full + 15,
             *stored = q_full + 16, *counted = q_full + 17;
    uint32_t* tmem_base = reinterpret_cast<uint32_t*>(sm + L::misc);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::misc + 4);
    volatile int* last = reinterpret_cast<volatile int*>(sm + L::misc + 8);
    volatile int* nan_rec = reinterpret_cast<volatile int*>(sm + L::nans);
    Work* works = reinterpret_cast<Work*>(sm + L::work);
    float* back_of = reinterpret_cast<float*>(sm + L::ml);     // what a row of q was divided by
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform, so each role's code is

    pdl_trigger();
    if (tid == 0) {
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
        for (int i = 0; i < R; ++i) {
            mbar_init(rawk_full + i, 1);
            mbar_init(rawk_empty + i, KC);
            mbar_init(rawv_full + i, 1);
            mbar_init(rawv_empty + i, VC);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + i, KC);
            mbar_init(k_empty + i, 1);
            mbar_init(v_full + i, VC);
            mbar_init(v_empty + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(o_done + i, 1);
        }
        mbar_init(q_full, 8);
        mbar_init(q_free, 1);
        mbar_init(handed, 8);
        mbar_init(drain, 1);
        mbar_init(copy_full, 8);
        mbar_init(copy_free, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(i_full + i, 1);
            mbar_init(i_empty + i, TC_THREADS / 32 - 1);
        }
        mbar_init(stored, 8);
        mbar_init(counted, 1);
        fence_mbar_init();
        *abort = 0;
        for (int i = 0; i < 4; ++i) nan_rec[4 * i] = 0;
    }
    if (warp == MMA_WARP) tc::tmem_alloc(tmem_base, 512);
    pdl_wait();
    Finder f{};
    Work first;
    first.item = -1;
    if (warp == TMA_K) {      // the first item, while the barriers are made ready
        f = make_finder(a, lane);
        if ((int)blockIdx.x < f.total) first = find_item(a, f, (int)blockIdx.x, lane);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_base, 0);

    // This warp's k-th item; false at the end.  The K loader posts them.
    auto take = [&](unsigned k, Work* wk) -> bool {
        if (!__all_sync(0xffffffffu, wait_or(i_full + (k & 1), (k >> 1) & 1, abort, a.err, SITE_TC + 13))) return false;
        *wk = works[k & 1];
        __threadfence_block();     // read before the slot goes back: an arrival can overtake queued loads
        __syncwarp();
        if (lane == 0) mbar_arrive(i_empty + (k & 1));
        return wk->item >= 0;
    };

    if (warp < 8) {
        // ---------------------------------------------------------- softmax
        const int t = warp >> 2, r = tid & 127;      // group, row of its tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_tm = tm + t * 128 + lanes, o_tm = tm + 256 + t * 128 + lanes;
        unsigned cs = 0, base = 0, folds = 0;   // this group's steps, all steps, split items so far
        bool ok = true;
        Work wk;
        for (unsigned items = 0; ok && take(items, &wk); ++items) {
            const Seq& q = wk.q;
            const Item& w = wk.w;
            const int item = wk.item;
            // the issuing thread is done with the item before: Q is free, and no
            // group is further ahead than the next item
            if (items > 0) {
                ok = __all_sync(0xffffffffu, wait_or(q_free, (items - 1) & 1, abort, a.err, SITE_TC));
                // and the copies' sums, which lie over Q, have been read
                if (ok && DUP == 2) ok = __all_sync(0xffffffffu, wait_or(copy_free, (items - 1) & 1, abort, a.err, SITE_TC));
                if (!ok) break;
            }
            const int n = (w.p1 - w.p0 + 1) / 2, nt = group_steps<KEYS>(a, q, w, t);
            const int copy = DUP == 2 ? r >> 6 : 0, row = DUP == 2 ? r & 63 : r;
            const int pr = w.tile * a.tile + (KEYS ? 0 : t * 128) + row;
            const int qi = pr / a.group, hq = w.kh * a.group + pr % a.group;
            const bool real = qi < q.n;
            int klo = 0, khi = 0;
            {
                // q, scaled into f16: a warp takes rows whole, 16 bytes a lane, so that
                // lanes read neighbours (a row a thread, with 16 times the L1 lookups,
                // took 7500 to 10500 cycles an item; this 3500)
                constexpr int LPR = HD / 8, RPI = 32 / LPR;           // lanes of a row, rows at a time
                constexpr int MINE = (KEYS ? 128 / DUP : 256) / 8;     // rows of a warp
                constexpr int N = MINE / RPI < 4 ? MINE / RPI : 4;
                const int at = lane & (LPR - 1);
                const int i0 = w.tile * a.tile / a.group, rest = w.tile * a.tile - i0 * a.group;
                const int by_group = (65536 + a.group - 1) / a.group;  // x / group = x by_group >> 16 below 4096
                const T* q0 = reinterpret_cast<const T*>(a.q) + (long long)(q.r0 + i0) * a.q_row +
                              (long long)w.kh * a.group * a.q_head + 8 * at;
#pragma unroll 1
                for (int x0 = 0; x0 < MINE; x0 += N * RPI) {
                    uint4 e[N];
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        const int p = rest + warp * MINE + x0 + x * RPI + lane / LPR, i = p * by_group >> 16;
                        e[x] = make_uint4(0, 0, 0, 0);
                        if (i0 + i < q.n)
                            e[x] = *reinterpret_cast<const uint4*>(q0 + (long long)i * a.q_row + (long long)(p - i * a.group) * a.q_head);
                    }
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        const T* ev = reinterpret_cast<const T*>(&e[x]);
                        float v[8], top = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            v[j] = to_f32(ev[j]);
                            const float y = fabsf(v[j]);
                            top = fmaxf(top, y < INFINITY ? y : 0.f);
                        }
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        float inv, back;
                        row_factor(top, &inv, &back);
                        uint4 o;
                        uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
                        for (int j = 0; j < 4; ++j) ow[j] = pack_f16x2(v[2 * j] * inv, v[2 * j + 1] * inv);
                        const int lr = warp * MINE + x0 + x * RPI + lane / LPR;      // of the item's rows
                        uint8_t* qs = sm + L::q + (KEYS ? 0 : (lr >> 7) * L::QB) + (at >> 3) * 128 * 128;
                        *reinterpret_cast<uint4*>(qs + swz128(lr & 127, at & 7)) = o;
                        if (DUP == 2) *reinterpret_cast<uint4*>(qs + swz128(lr + 64, at & 7)) = o;
                        if (at == 0) back_of[lr] = back;
                    }
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }

            if (real) row_keys(a, q, qi, &klo, &khi);
            // a warp without rows only takes part: its lanes' weights stay whatever
            // tensor memory holds, and nothing of them is written
            const bool any = __any_sync(0xffffffffu, real);
            // a step that not all rows see whole: masked scores become -inf in
            // tensor memory first (code in the loop below would cost every step)
            auto mask = [&](const float* ks, int k0) {
#pragma unroll 1
                for (int c = 2 * copy; c < 2 * copy + 4 / DUP; ++c) {
                    uint32_t v[32];
                    tc::ld_x32_async(s_tm + c * 32, v);
                    tc::ld_wait(v);
                    const int lo = klo - k0 - c * 32, hi = ks[c >> 1] < 0.f ? 0 : khi - k0 - c * 32;
                    const uint32_t seen = lo < 32 && hi > 0 && lo < hi ? ~0u >> (hi < 32 ? 32 - hi : 0) & ~0u << (lo > 0 ? lo : 0) : 0u;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (!(seen & (1u << x))) v[x] = 0xff800000u;      // -inf
                    tc::st_x16(s_tm + c * 32, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
                    tc::st_x16(s_tm + c * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
                }
                tc::st_wait();
            };
            // all rows have seen the same keys up to steps from here on
            const int same = w.lo == w.in_lo || w.p0 * KV8_PAGE >= w.in_lo ? (w.hi == w.in_hi ? 0x7fffffff : w.in_hi - STEP + 1) : 0;
            float M = -INFINITY, l = 0.f;
            int i = 0;
            for (; i < nt && ok; ++i, ++cs) {
                const int j = KEYS ? 2 * i + t : i;
                ok = __all_sync(0xffffffffu, wait_or(s_full + t, cs & 1, abort, a.err, SITE_TC + 1));
                if (!ok) break;
                if (!any) {
                    if (lane == 0) mbar_arrive(p_full + t);
                    continue;
                }
                tc::fence_after_sync();
                const StepScale& sc = steps[(base + j) & 7];
                const float fr = back_of[KEYS ? row : t * 128 + row] * a.scale_log2;
                const int k0 = (w.p0 + 2 * j) * KV8_PAGE;
                if (k0 < w.in_lo || k0 + STEP > w.in_hi || sc.ks[0] < 0.f || sc.ks[1] < 0.f) {
                    if (sc.far > 0.f) break;
                    mask(sc.ks, k0);
                }
                const float rise = k0 < same ? ROOM : INFINITY;      // that moves a row beside another one
                // 32 keys at a time, the next 32 scores on their way meanwhile
                uint32_t buf[2][32];
                const int c0 = 2 * copy;
                tc::ld_x32_async(s_tm + c0 * 32, buf[0]);
                if (DUP == 2) {      // the other page's weights are the other copy's
                    uint32_t p[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) p[x] = 0;
                    tc::st_x16(s_tm + (2 - c0) * 32, p);
                    tc::st_x16(s_tm + (3 - c0) * 32, p);
                }
#pragma unroll
                for (int cc = 0; cc < 4 / DUP; ++cc) {
                    const int c = c0 + cc;
                    uint32_t (&v)[32] = buf[cc & 1];
                    tc::ld_wait(v);
                    const float ks = sc.ks[c >> 1], ev = sc.ev[c >> 1];
                    const bool there = ks >= 0.f;
                    const float f = there ? fmaxf(fr * ks, 0x1p-126f) : 1.f;   // above 0: a masked score stays -inf
                    float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        m[0] = fmaxf(m[0], fmaxf(__uint_as_float(v[x]), __uint_as_float(v[x + 1])));
                        m[1] = fmaxf(m[1], fmaxf(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])));
                    }
                    const float top = fmaxf(m[0], m[1]);
                    const float mx = top == -INFINITY ? -INFINITY : fmaf(top, f, ev);
                    // move the reference where this row's maximum has risen far: the sums,
                    // the outputs and this step's weights so far follow
                    bool need = mx > M + (ROOM + LAZY) || (M == -INFINITY && mx > -INFINITY);
                    if (__any_sync(0xffffffffu, need)) {
                        const bool first = M == -INFINITY;
                        // the others that have risen: only where all rows have seen the same keys
                        // so far, as a row's bits must not follow from keys that it does not see
                        need = need || (!first && mx > M + rise);
                        const float f0 = need ? (first ? 0.f : ex2(M + ROOM - mx)) : 1.f;
                        if (need) M = mx - ROOM;
                        l *= f0;
                        // the weights and outputs of a row without any so far are zeros; others
                        // follow, by 0 where the maximum has risen by 126 or more
                        if (__any_sync(0xffffffffu, need && !first)) {
                            tc::st_wait();
#pragma unroll 1
                            for (int b = c0; b < c; ++b) {
                                uint32_t p[16];
                                tc::ld_x16(s_tm + b * 32, p);
#pragma unroll
                                for (int x = 0; x < 16; ++x) {
                                    const float2 y = __half22float2(*reinterpret_cast<__half2*>(&p[x]));
                                    p[x] = pack_f16x2(y.x * f0, y.y * f0);
                                }
                                tc::st_x16(s_tm + b * 32, p);
                            }
                            if (i > 0) {
                                ok = __all_sync(0xffffffffu, wait_or(o_done + t, (cs - 1) & 1, abort, a.err, SITE_TC + 2));
                                tc::fence_after_sync();
#pragma unroll 1
                                for (int b = 0; b < HD / 16 && ok; ++b) {
                                    uint32_t o[16];
                                    tc::ld_x16(o_tm + b * 16, o);
#pragma unroll
                                    for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f0);
                                    tc::st_x16(o_tm + b * 16, o);
                                }
                            }
                        }
                    }
                    if (cc < 4 / DUP - 1) tc::ld_x32_async(s_tm + (c + 1) * 32, buf[(cc + 1) & 1]);
                    const float off = ev - (M == -INFINITY ? 0.f : M);
                    const float2 ff = make_float2(f, f), oo = make_float2(off, off);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t p[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        float2 y = fma2(make_float2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), ff, oo);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        sum[x & 1] = add2(sum[x & 1], y);
                        p[x] = pack_f16x2(y.x, y.y);
                    }
                    tc::st_x16(s_tm + c * 32, p);
                    const float2 s2 = add2(sum[0], sum[1]);
                    l = fmaf(s2.x + s2.y, sc.iv[c >> 1], l);
                }
                if (!ok) break;
                tc::st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + t);
            }
            // the steps from the first one on whose V scales lie far apart: two references,
            // M and Z; the same for all of the group (the tensor core has done the first
            // one's scores already: its wait is over at once)
            float Z = M;
#pragma unroll 1
            for (; i < nt && ok; ++i, ++cs) {
                const int j = KEYS ? 2 * i + t : i, c0 = 2 * copy;
                ok = __all_sync(0xffffffffu, wait_or(s_full + t, cs & 1, abort, a.err, SITE_TC + 1));
                if (!ok) break;
                tc::fence_after_sync();
                const StepScale& sc = steps[(base + j) & 7];
                const float fr = back_of[KEYS ? row : t * 128 + row] * a.scale_log2;
                mask(sc.iv, (w.p0 + 2 * j) * KV8_PAGE);
                if (DUP == 2) {
                    uint32_t p[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) p[x] = 0;
                    tc::st_x16(s_tm + (2 - c0) * 32, p);
                    tc::st_x16(s_tm + (3 - c0) * 32, p);
                }
#pragma unroll 1
                for (int c = c0; c < c0 + 4 / DUP && ok; ++c) {
                    uint32_t v[32], p[16];
                    tc::ld_x32_async(s_tm + c * 32, v);
                    tc::ld_wait(v);
                    const float ks = sc.iv[c >> 1], ev = sc.ev[c >> 1];
                    const float f = ks >= 0.f ? fmaxf(fr * ks, 0x1p-126f) : 1.f;
                    float top = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 32; ++x) top = fmaxf(top, __uint_as_float(v[x]));
                    const float mt = top == -INFINITY ? -INFINITY : top * f, mx = mt + ev;
                    const bool first = M == -INFINITY;
                    const float m = mx > M + (ROOM + LAZY) || (first && mx > -INFINITY) ? mx - ROOM : M;
                    const float z = fmaxf(Z, mt);
                    const float f0 = first ? 1.f : ex2(M - m);
                    if (!first) l *= ex2(Z - z);
                    M = m;
                    Z = z;
                    if (__any_sync(0xffffffffu, f0 != 1.f)) {
                        tc::st_wait();
#pragma unroll 1
                        for (int b = c0; b < c; ++b) {
                            tc::ld_x16(s_tm + b * 32, p);
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                const float2 y = __half22float2(*reinterpret_cast<__half2*>(&p[x]));
                                p[x] = pack_f16x2(y.x * f0, y.y * f0);
                            }
                            tc::st_x16(s_tm + b * 32, p);
                        }
                        if (i > 0) {
                            ok = __all_sync(0xffffffffu, wait_or(o_done + t, (cs - 1) & 1, abort, a.err, SITE_TC + 2));
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int b = 0; b < HD / 16 && ok; ++b) {
                                tc::ld_x16(o_tm + b * 16, p);
#pragma unroll
                                for (int x = 0; x < 16; ++x) p[x] = __float_as_uint(__uint_as_float(p[x]) * f0);
                                tc::st_x16(o_tm + b * 16, p);
                            }
                        }
                    }
                    const float k = M == -INFINITY ? 0.f : ex2(M - ev - Z);      // weights on values to the sum's
                    const bool lost = k > FAR_PAGE;
                    const float off = lost ? -Z : ev - (M == -INFINITY ? 0.f : M);
                    float sum = 0.f;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const float y0 = ex2(fmaf(__uint_as_float(v[2 * x]), f, off)), y1 = ex2(fmaf(__uint_as_float(v[2 * x + 1]), f, off));
                        sum += y0 + y1;
                        p[x] = lost ? 0u : pack_f16x2(y0, y1);
                    }
                    tc::st_x16(s_tm + c * 32, p);
                    l = fmaf(sum, lost ? 1.f : k, l);
                }
                if (!ok) break;
                tc::st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + t);
            }
            if (ok && nt > 0) {
                ok = __all_sync(0xffffffffu, wait_or(o_done + t, (cs - 1) & 1, abort, a.err, SITE_TC + 2));
                tc::fence_after_sync();
            }
            base += n;
            if (!ok) break;

            // KEYS: the groups see the same lanes of tensor memory.  Each writes its
            // references and sum over its scores, and takes half of the columns of
            // both outputs.
            float fa = 1.f, fb = 0.f;                      // factors of this group's and the other's sums
            const int nt_other = KEYS ? group_steps<KEYS>(a, q, w, 1 - t) : 0;
            const uint32_t other = t == 0 ? 128u : (uint32_t)-128;
            if (KEYS) {
                tc::st_x2(s_tm, M, l);
                tc::st_x2(s_tm + 2, Z, 0.f);
                tc::st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(handed);
                ok = __all_sync(0xffffffffu, wait_or(handed, items & 1, abort, a.err, SITE_TC + 4));
                if (!ok) break;
                tc::fence_after_sync();
                float bm, bl, bz, none;
                tc::ld_x2(s_tm + other, &bm, &bl);
                tc::ld_x2(s_tm + other + 2, &bz, &none);
                const float m = fmaxf(M, bm);
                fa = M == -INFINITY ? 0.f : ex2(M - m);
                fb = bm == -INFINITY ? 0.f : ex2(bm - m);
                const float z = fmaxf(sum_ref(M, Z), sum_ref(bm, bz));
                l = part_of(l, Z, z) + part_of(bl, bz, z);
                Z = z;
                M = m;
            }
            constexpr int NB = HD / 16 / (KEYS ? 2 : 1);           // 16-column blocks of a group
            const int b_first = KEYS && t == 1 ? NB : 0;
            if ((KEYS || nt > 0) && nan_rec[4 * (items & 3)] == (int)items + 1)     // the same for all of a group's threads
                put_nans<HD, KEYS, DUP>(a, nan_rec + 4 * (items & 3), t, r, nt > 0 ? o_tm : o_tm + other);

            // ---- the row's outputs, or its partial of this split
            const long long slot0 = (long long)item - w.split;    // splits of a tile are neighbours
            const long long tk = (((long long)q.r0 * a.group >> a.tile_log2) + w.s + w.tile) * a.n_kv + w.kh;
            const bool split = q.splits > 1;
            const bool fits = !split || (slot0 + q.splits <= a.part_cap && tk < a.ticket_cap);   // by the plan's bounds
            const int RT = a.tile;
            const long long PL = (long long)RT * (HD + 4);         // floats of a partial
            const int prow = KEYS ? row : t * 128 + row;
            float* part = split ? a.part + (slot0 + w.split) * PL : nullptr;
            T* dst = reinterpret_cast<T*>(a.out) + (long long)(q.r0 + qi) * a.out_row + (long long)hq * a.out_head;
            auto sums = [&](int b, float (&v)[16]) {      // of both groups, block b of 16 columns
                __syncwarp();
                uint32_t y[16];
                if (nt > 0) {
                    tc::ld_x16(o_tm + b * 16, y);
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x] = __uint_as_float(y[x]);
                } else {
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x] = 0.f;
                }
                if (KEYS && nt_other > 0) {
                    tc::ld_x16(o_tm + other + b * 16, y);
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x] = fmaf(__uint_as_float(y[x]), fb, v[x] * fa);
                }
            };
            // DUP: a copy gives the other one half of its group's blocks, and adds
            // the other's half to its own; both write
            constexpr int HALF = NB / DUP;
            float4* xb = reinterpret_cast<float4*>(sm + L::q) + (size_t)t * NB * 4 * 64 + row;    // [copy][HALF][4][64]
            float2* xml = reinterpret_cast<float2*>(sm + L::ml) + row;                            // [copy][64]: (M, log2 of the sum)
            float ga = 1.f, gb = 0.f;      // factors of copy 0's and copy 1's sums
            if (DUP == 2) {
#pragma unroll 1
                for (int x = 0; x < HALF; ++x) {
                    float v[16];
                    sums(b_first + (1 - copy) * HALF + x, v);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        xb[((copy * HALF + x) * 4 + y) * 64] = make_float4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
                }
                if (t == 0) xml[copy * 64] = make_float2(M, l == 0.f ? -INFINITY : Z + log2f(l));      // the same in both groups
                __syncwarp();
                if (lane == 0) mbar_arrive(copy_full);
                ok = __all_sync(0xffffffffu, wait_or(copy_full, items & 1, abort, a.err, SITE_TC + 15));
                if (!ok) break;
                const float2 m0 = xml[0], m1 = xml[64];
                M = fmaxf(m0.x, m1.x);
                ga = m0.x == -INFINITY ? 0.f : ex2(m0.x - M);
                gb = m1.x == -INFINITY ? 0.f : ex2(m1.x - M);
                Z = fmaxf(m0.y, m1.y);
                l = (m0.y == -INFINITY ? 0.f : ex2(m0.y - Z)) + (m1.y == -INFINITY ? 0.f : ex2(m1.y - Z));
            }
            const float inv = out_factor(M, Z, l);
#pragma unroll 1
            for (int x = 0; x < HALF; ++x) {
                const int b = b_first + copy * HALF + x;
                float v[16];
                sums(b, v);
                if (DUP == 2) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float4 z = xb[(((1 - copy) * HALF + x) * 4 + y) * 64];
                        const float u[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[4 * y + k] = copy == 0 ? fmaf(u[k], gb, v[4 * y + k] * ga) : fmaf(v[4 * y + k], gb, u[k] * ga);
                    }
                }
                if (real && split && fits) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        reinterpret_cast<float4*>(part)[(size_t)(b * 4 + y) * RT + prow] =
                            make_float4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
                }
                if (real && !split) store16<T>(dst + b * 16, v, inv);
            }
            __syncwarp();
            tc::fence_before_sync();   // the accumulator has been read
            if (DUP == 2 && lane == 0) mbar_arrive(copy_free);
            if (!split) {
                if (real && copy == 0 && a.lse && b_first == 0)
                    a.lse[(long long)(q.r0 + qi) * a.n_q + hq] = row_lse(Z, l);
                continue;
            }
            if (real && fits && copy == 0 && b_first == 0) reinterpret_cast<float4*>(part + (size_t)RT * HD)[prow] = make_float4(M, sum_ref(M, Z), l, 0.f);
            // the CTA whose split of the tile is the last to arrive folds them all, in
            // split order: a thread takes a row and a share of its columns
            __threadfence();
            __syncwarp();
            if (lane == 0) mbar_arrive(stored);
            if (warp == 0) {
                ok = __all_sync(0xffffffffu, wait_or(stored, folds & 1, abort, a.err, SITE_TC + 15));
                if (!ok) break;
                if (lane == 0) {
                    *last = fits && atomicAdd(a.tickets + tk, 1) == q.splits - 1;
                    if (*last) a.tickets[tk] = 0;
                    mbar_arrive(counted);
                }
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, wait_or(counted, folds & 1, abort, a.err, SITE_TC + 15));
            if (!ok) break;
            ++folds;
            if (!*last) continue;
            __threadfence();
            const int frow = tid % RT, shares = 256 / RT, share = tid / RT;
            const int fr_ = w.tile * RT + frow, fi = fr_ / a.group, fh = w.kh * a.group + fr_ % a.group;
            if (fi < q.n) {
                const float* src = a.part + slot0 * PL;
                const float4* mls = reinterpret_cast<const float4*>(src + (size_t)RT * HD) + frow;    // (M, Z, l)
                const long long PL4 = PL / 4;
                float fm = -INFINITY, fz = -INFINITY, fl = 0.f;
#pragma unroll 4
                for (int v = 0; v < q.splits; ++v) {
                    const float4 x = __ldcg(mls + v * PL4);
                    fm = fmaxf(fm, x.x);
                    fz = fmaxf(fz, x.y);
                }
#pragma unroll 4
                for (int v = 0; v < q.splits; ++v) {
                    const float4 x = __ldcg(mls + v * PL4);
                    fl += part_of(x.z, x.y, fz);
                }
                const float finv = out_factor(fm, fz, fl);
                T* fdst = reinterpret_cast<T*>(a.out) + (long long)(q.r0 + fi) * a.out_row + (long long)fh * a.out_head;
#pragma unroll 1
                for (int b = share * (HD / 16) / shares; b < (share + 1) * (HD / 16) / shares; ++b) {
                    float o[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) o[x] = 0.f;
                    const float4* col = reinterpret_cast<const float4*>(src) + (size_t)b * 4 * RT + frow;
#pragma unroll 2
                    for (int v = 0; v < q.splits; ++v) {
                        float4 y[4];
                        const float m = __ldcg(mls + v * PL4).x;
#pragma unroll
                        for (int x = 0; x < 4; ++x) y[x] = __ldcg(col + v * PL4 + x * RT);
                        const float f = m == -INFINITY ? 0.f : ex2(m - fm);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            o[4 * x] = fmaf(y[x].x, f, o[4 * x]);
                            o[4 * x + 1] = fmaf(y[x].y, f, o[4 * x + 1]);
                            o[4 * x + 2] = fmaf(y[x].z, f, o[4 * x + 2]);
                            o[4 * x + 3] = fmaf(y[x].w, f, o[4 * x + 3]);
                        }
                    }
                    store16<T>(fdst + 16 * b, o, finv);
                }
                if (a.lse && share == 0)
                    a.lse[(long long)(q.r0 + fi) * a.n_q + fh] = row_lse(fz, fl);
            }
            __syncwarp();
        }
    } else if (warp < VC_WARP) {
        // ---------------------------------------------------------- K's conversion
        const int cw = warp - KC_WARP;
        unsigned g = 0;     // steps so far
        bool ok = true;
        Work wk;
        for (unsigned items = 0; ok && take(items, &wk); ++items) {
            const Item& w = wk.w;
            const int n = (w.p1 - w.p0 + 1) / 2;
            bool far = false;
            for (int j = 0; j < n; ++j, ++g) {
                const int st = g & 1;
                const unsigned r0 = (2 * g) % R, par = (2 * g / R) & 1;      // R is even: both pages share a parity
                ok = (g < 2 || wait_or(k_empty + st, ((g >> 1) - 1) & 1, abort, a.err, SITE_TC + 5)) &&
                     wait_or(rawk_full + r0, par, abort, a.err, SITE_TC + 6) &&
                     wait_or(rawk_full + r0 + 1, par, abort, a.err, SITE_TC + 6);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (cw == 0) {
                    const float2 sc = rsc[r0 + (lane & 1)];
                    const bool there = sc.x >= 0.f && sc.y > 0.f;
                    far = far || __any_sync(0xffffffffu, there && !near(sc.y));
                    if (lane < 2) {
                        StepScale* d = steps + (g & 7);
                        const float ks = there ? sc.x : -1.f;
                        d->ks[lane] = far ? -1.f : ks;
                        d->ev[lane] = there ? log2f(sc.y) : 0.f;
                        d->iv[lane] = far ? ks : (there ? 1.f / sc.y : 0.f);
                        d->far = far ? 1.f : 0.f;
                    }
                }
                uint8_t* dst = sm + L::k + st * L::KB;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {                  // the step's pages
                    constexpr int MINE = HD / 8 / KC;          // units of 32 keys x 16 dims
                    uint4 e[MINE];
#pragma unroll
                    for (int y = 0; y < MINE; ++y) {
                        const int u = cw + y * KC;
                        // a page that is not there: its scores are masked whatever the bytes
                        e[y] = lds128(sm + L::raw + (r0 + h) * PB + tile_off<HD>((u & 1) * 32 + lane, u >> 1));
                    }
#pragma unroll
                    for (int y = 0; y < MINE; ++y) {
                        const int u = cw + y * KC, key = (u & 1) * 32 + lane, c = u >> 1;
                        const uint32_t ew[4] = {e[y].x, e[y].y, e[y].z, e[y].w};
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            o[2 * k] = f16_of_codes(ew[k]);
                            o[2 * k + 1] = f16_of_codes(ew[k] >> 16);
                        }
                        uint8_t* d = dst + (c >> 2) * STEP * 128;
                        *reinterpret_cast<uint4*>(d + swz128(h * KV8_PAGE + key, 2 * (c & 3))) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(d + swz128(h * KV8_PAGE + key, 2 * (c & 3) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    // the page goes back once its codes have been used: an arrival can
                    // overtake loads that are still queued
                    __syncwarp();
                    if (lane == 0) mbar_arrive(rawk_empty + r0 + h);
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(k_full + st);
            }
        }
    } else if (warp < MMA_WARP) {
        // ---------------------------------------------------------- V's conversion
        const int cw = warp - VC_WARP;
        unsigned g = 0;
        bool ok = true;
        Work wk;
        for (unsigned items = 0; ok && take(items, &wk); ++items) {
            const Item& w = wk.w;
            const int n = (w.p1 - w.p0 + 1) / 2;
            for (int j = 0; j < n; ++j, ++g) {
                const int st = g & 1;
                const unsigned r0 = (2 * g) % R, par = (2 * g / R) & 1;
                ok = (g < 2 || wait_or(v_empty + st, ((g >> 1) - 1) & 1, abort, a.err, SITE_TC + 7)) &&
                     wait_or(rawv_full + r0, par, abort, a.err, SITE_TC + 6) &&
                     wait_or(rawv_full + r0 + 1, par, abort, a.err, SITE_TC + 6);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const float2 sa = rscv[r0], sb = rscv[r0 + 1];
                const bool there[2] = {sa.x >= 0.f && sa.y > 0.f, sb.x >= 0.f && sb.y > 0.f};
                // a key's V must not reach a row that does not see it, and 0 * NaN is NaN:
                // where not all rows see all keys, codes that no row sees and NaN ones
                // are taken as zeros, and the item is marked: the rows that see a NaN
                // get it with their outputs
                const int kp = (w.p0 + 2 * j) * KV8_PAGE;
                const bool plain = kp >= w.in_lo && kp + STEP <= w.in_hi && there[0] && there[1];
                uint32_t seen = 0;
                uint8_t* dst = sm + L::v + st * L::KB;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    constexpr int MINE = HD / 8 / VC;          // units of 32 keys x 16 dims
                    uint32_t r4[MINE][4];
#pragma unroll
                    for (int y = 0; y < MINE; ++y) {
                        const int x = cw + y * VC;
                        ldsm_x4_trans(r4[y], sm + L::raw + (R + r0 + h) * PB + tile_off<HD>((x & 1) * 32 + lane, x >> 1));
                    }
                    if (!plain) {
                        const bool valid = h ? there[1] : there[0];
                        const bool whole = kp + h * KV8_PAGE >= w.in_lo && kp + (h + 1) * KV8_PAGE <= w.in_hi;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // VC is even, so all of this warp's units have the same 32 keys
                            const int k = kp + h * KV8_PAGE + (cw & 1) * 32 + 8 * i + 2 * (lane & 3);
                            const uint32_t keep = (valid && k >= w.lo && k < w.hi ? 0x0000ffffu : 0u) |
                                                  (valid && k + 1 >= w.lo && k + 1 < w.hi ? 0xffff0000u : 0u);
#pragma unroll
                            for (int y = 0; y < MINE; ++y) {
                                const uint32_t x = r4[y][i] & keep;
                                r4[y][i] = whole ? x : drop_nan(x, &seen);
                            }
                        }
                    }
#pragma unroll
                    for (int y = 0; y < MINE; ++y) {
                        const int x = cw + y * VC, kb = x & 1, d = x >> 1;
                        uint32_t e[4], o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t p = __byte_perm(r4[y][i], 0, 0x3120);
                            e[i] = f16_of_codes(p);
                            o[i] = f16_of_codes(p >> 16);
                        }
                        const int row = 16 * d + (lane & 7), ch = 4 * kb + (lane >> 3);
                        uint8_t* vd = dst + h * HD * 128;
                        stsm_x4(vd + swz128(row, ch), e);
                        stsm_x4(vd + swz128(row + 8, ch), o);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(rawv_empty + r0 + h);   // its codes have been used
                }
                // read at the item's end: no role is four items ahead
                if (!plain && seen) {
                    volatile int* rec = nan_rec + 4 * (items & 3);
                    rec[1] = w.s;
                    rec[2] = ((wk.q.tiles - 1 - w.tile) * a.n_kv + w.kh) * wk.q.splits + w.split;
                    rec[3] = w.tile;
                    rec[0] = items + 1;
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_full + st);
            }
        }
    } else if (warp == MMA_WARP) {
        // ---------------------------------------------------------- MMAs
        // the warp stays converged and one lane issues: what an MMA names is
        // uniform (issuing from a divergent lane took about twice as long)
        constexpr uint32_t IS = tc::idesc_f16_f32(128, STEP), IO = tc::idesc_f16_f32(128, HD);
        unsigned base = 0, done[2] = {0, 0};
        bool ok = true;
        // descriptors of the tiles' first bytes; a k step adds 32 bytes, a
        // 64-element half of K or Q its rows (in 16-byte units)
        const uint64_t qd = tc::desc_sw128(sm + L::q), kd = tc::desc_sw128(sm + L::k), vd = tc::desc_sw128(sm + L::v);
        Work wk;
        for (unsigned items = 0; ok && take(items, &wk); ++items) {
            const Seq& q = wk.q;
            const Item& w = wk.w;
            const int n = (w.p1 - w.p0 + 1) / 2;
            const int nt[2] = {__shfl_sync(0xffffffffu, group_steps<KEYS>(a, q, w, 0), 0),
                               __shfl_sync(0xffffffffu, group_steps<KEYS>(a, q, w, 1), 0)};
            ok = __all_sync(0xffffffffu, wait_or(q_full, items & 1, abort, a.err, SITE_TC + 8));
            auto qk = [&](int t, int i) -> bool {     // S_t = Q_t K^T of the group's step i
                const unsigned g = __shfl_sync(0xffffffffu, base + (KEYS ? 2 * i + t : i), 0);
                const unsigned st = g & 1;
                if (!__all_sync(0xffffffffu, wait_or(k_full + st, (g >> 1) & 1, abort, a.err, SITE_TC + 9))) return false;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint64_t qt = qd + (KEYS ? 0 : t * (L::QB >> 4)), kt = kd + st * (L::KB >> 4);
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        tc::mma_f16(tm + t * 128, qt + ((k >> 2) * (128 * 128 >> 4) + (k & 3) * 2),
                                    kt + ((k >> 2) * (STEP * 128 >> 4) + (k & 3) * 2), IS, k > 0);
                    tc::commit(s_full + t);
                    if (KEYS || t == 1 || nt[1] == 0) tc::commit(k_empty + st);
                }
                __syncwarp();
                return true;
            };
            auto pv = [&](int t, int i) -> bool {     // O_t += P_t V
                const unsigned g = __shfl_sync(0xffffffffu, base + (KEYS ? 2 * i + t : i), 0);
                const unsigned st = g & 1;
                if (!__all_sync(0xffffffffu, wait_or(v_full + st, (g >> 1) & 1, abort, a.err, SITE_TC + 11) &&
                                                 wait_or(p_full + t, (done[t] + i) & 1, abort, a.err, SITE_TC + 10)))
                    return false;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint64_t vt = vd + st * (L::KB >> 4);
                    const uint32_t more = i > 0;
#pragma unroll
                    for (int k = 0; k < STEP / 16; ++k)
                        tc::mma_f16_ta(tm + 256 + t * 128, tm + t * 128 + 32 * (k >> 1) + 8 * (k & 1),
                                       vt + ((k >> 2) * (HD * 128 >> 4) + (k & 3) * 2), IO, k > 0 ? 1u : more);
                    tc::commit(o_done + t);
                    if (KEYS || t == 1 || nt[1] == 0) tc::commit(v_empty + st);
                }
                __syncwarp();
                return true;
            };
            ok = ok && (nt[0] == 0 || qk(0, 0)) && (nt[1] == 0 || qk(1, 0));
            for (int i = 0; i < nt[0] && ok; ++i) {
                ok = pv(0, i) && (i + 1 >= nt[0] || qk(0, i + 1));
                if (ok && i < nt[1]) ok = pv(1, i) && (i + 1 >= nt[1] || qk(1, i + 1));
            }
            done[0] += nt[0];
            done[1] += nt[1];
            base += n;
            if (ok && tc::elect_one()) tc::commit(q_free);
            __syncwarp();
        }
        // every MMA has finished before tensor memory is given back
        if (tc::elect_one()) tc::commit(drain);
        __syncwarp();
        mbar_wait(drain, 0);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- pages
        const bool is_k = warp == TMA_K;
        const CUtensorMap* map = is_k ? &k_map : &v_map;
        uint64_t *rfull = is_k ? rawk_full : rawv_full, *rempty = is_k ? rawk_empty : rawv_empty;
        float2* scales = is_k ? rsc : rscv;
        uint8_t* ring = sm + L::raw + (is_k ? 0 : R * PB);
        unsigned it = 0;   // pages issued
        bool ok = true;
        int asked = 0;
        Work wk = first;
        for (unsigned items = 0; ok; ++items) {
            if (is_k) {
                // posts the item; the next one's number is on its way
                if (lane == 0) {
                    if (items < 2 || wait_or(i_empty + (items & 1), ((items >> 1) - 1) & 1, abort, a.err, SITE_TC + 14)) {
                        works[items & 1] = wk;
                        mbar_arrive(i_full + (items & 1));
                    }
                    if (wk.item >= 0) asked = ask_item(a, f.total);
                }
                if (wk.item < 0) break;
            } else if (!take(items, &wk)) {
                break;
            }
            const Item& w = wk.w;
            const int slots = (w.p1 - w.p0 + 1) / 2 * 2;
            // lane i looks up page b + i and its scales; the next 32 are on their
            // way while these are issued
            auto look = [&](int b, int* page, float* ks, float* vs) {
                *page = -1;
                *ks = -1.f;
                *vs = 1.f;
                if (w.p0 + b + lane >= w.p1) return;
                const int pg = a.table[(size_t)w.s * a.max_pages + w.p0 + b + lane];
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
            look(0, &page, &ks, &vs);
            for (int b = 0; b < slots && ok; b += 32) {
                look(b + 32, &next_page, &next_ks, &next_vs);
                if (page >= 0 && !scales_fit(ks, vs)) {      // not in look, which would wait for the scales
                    report(a.err, DERR_INDEX, SITE_SCALE);
                    page = -1;
                    ks = -1.f;
                }
                const int m = slots - b < 32 ? slots - b : 32;
                for (int j = 0; j < m; ++j) {
                    const int pg = __shfl_sync(0xffffffffu, page, j);
                    const float kj = __shfl_sync(0xffffffffu, ks, j), vj = __shfl_sync(0xffffffffu, vs, j);
                    const int st = it % R;
                    bool issued = true;
                    if (lane == 0) {
                        issued = it < R || wait_or(rempty + st, (it / R - 1) & 1, abort, a.err, SITE_TC + 12);
                        if (issued) {
                            scales[st] = make_float2(kj, vj);
                            if (pg >= 0) {
                                mbar_arrive_expect_tx(rfull + st, PB);
                                tma_load_2d(ring + st * PB, map, rfull + st, 0, (pg * a.n_kv + w.kh) * KV8_PAGE);
                            } else {
                                mbar_arrive(rfull + st);
                            }
                        }
                    }
                    if (!__shfl_sync(0xffffffffu, (int)issued, 0)) {
                        ok = false;
                        break;
                    }
                    ++it;
                }
                page = next_page;
                ks = next_ks;
                vs = next_vs;
            }
            if (is_k) {
                int next = lane == 0 ? settle_item(a, f.total, asked) : 0;
                next = __shfl_sync(0xffffffffu, next, 0);
                wk.item = -1;
                if (next >= 0) wk = find_item(a, f, next, lane);
            }
        }
        // no copy of this CTA is in flight when it ends
        if (lane == 0) {
            const unsigned n = it < R ? it : R;
            for (unsigned i = it - n; i < it; ++i) mbar_wait(rfull + i % R, (i / R) & 1);
        }
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == MMA_WARP) tc::tmem_dealloc(tm, 512);
}

template <typename T, int HD, bool KEYS, int DUP>
int launch_tc(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a, int sms, cudaStream_t s) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv8_attn_tc_kernel<T, HD, KEYS, DUP>));
    if (e != cudaSuccess) return (int)e;
    const long long most = a.ticket_cap * a.split_cap;   // items there can be
    const long long grid = most < sms ? most : sms;
    return (int)launch_k(kv8_attn_tc_kernel<T, HD, KEYS, DUP>, dim3((unsigned)grid), dim3(TC_THREADS),
                         TcSmem<HD, KEYS, DUP>::bytes, s, k_map, v_map, a);
}

template <typename T, int HD>
int launch_tc_t(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a, int sms, cudaStream_t s) {
    if (a.tile == 64) return launch_tc<T, HD, true, 2>(k_map, v_map, a, sms, s);
    if (a.tile == 128) return launch_tc<T, HD, true, 1>(k_map, v_map, a, sms, s);
    return launch_tc<T, HD, false, 1>(k_map, v_map, a, sms, s);
}

}  // namespace

int launch_kv8_attention_tc(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a,
                            int head_dim, int sms, cudaStream_t s) {
    if (a.dtype == 1)
        return head_dim == 128 ? launch_tc_t<__nv_bfloat16, 128>(k_map, v_map, a, sms, s)
                               : launch_tc_t<__nv_bfloat16, 64>(k_map, v_map, a, sms, s);
    return head_dim == 128 ? launch_tc_t<__half, 128>(k_map, v_map, a, sms, s)
                           : launch_tc_t<__half, 64>(k_map, v_map, a, sms, s);
}

}  // namespace dfl
