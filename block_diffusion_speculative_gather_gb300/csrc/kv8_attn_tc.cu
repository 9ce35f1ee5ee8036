// Attention over the 8-bit paged cache for many rows per kv head, on the
// fifth-generation tensor cores (tcgen05).  The mathematics is the one stated
// in kv8_attn.cu.
//
// A CTA per SM takes items (row tile, kv head, split of the pages).  Its two
// softmax groups of four warps, one thread to a row, each own a 128 x 128
// score tile and an output accumulator in tensor memory:
//   ROWS form (more than 128 packed rows a sequence): the groups take two
//     128-row tiles of q over the same keys, which are converted once;
//   KEYS form: both take the same 128 rows and alternate 128-key steps; at
//     the item's end the first reads the second's sums from tensor memory.
// Roles: a warp brings the pages' codes by TMA and looks up pages and scales;
// four warps turn a step's codes (two pages) into f16 operand tiles, K as it
// stands and V transposed (keys contiguous); one thread issues the MMAs:
// S = Q K^T, then O += P V with P read from tensor memory, where the softmax
// warps wrote it over the scores.  While one group's softmax runs, the
// tensor core works for the other.
//
// The running maximum that weights refer to moves only when a row's maximum
// rises by more than 2^8 (weights stay within f16's range), so outputs are
// rescaled in tensor memory rarely.
//
// Tensor memory: scores at columns 0 and 128, outputs at 256 and 384.  A
// step's P overwrites the first half of its scores, and the next step's
// scores overwrite P: the two MMAs are issued in that order by one thread.

#include <type_traits>

#include "attention_dev.cuh"
#include "kv8_attn_dev.cuh"
#include "tc_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;
using adev::ldsm_x4_trans;

constexpr int CONV_WARP = 8, N_CONV = 4, MMA_WARP = 12, TC_THREADS = 32 * 14;   // the last warp loads
constexpr int STEP = 2 * KV8_PAGE;         // keys of a step
constexpr int SITE_TC = 310;               // + role
constexpr float LAZY = 8.f;                // rise of a row's maximum (base 2) that moves the reference

template <int HD, bool KEYS> struct TcSmem {
    static constexpr int QB = 128 * HD * 2;                    // one q tile, f16
    static constexpr int QR = KEYS ? QB : 2 * QB;
    static constexpr int KB = STEP * HD * 2;                   // one step's K (or V), f16
    static constexpr int PB = KV8_PAGE * HD;                   // one page's K (or V) codes
    static constexpr int RAW = HD == 64 ? 8 : (KEYS ? 4 : 2);  // pages in flight, K and V each
    static constexpr int q = 0, k = q + QR, v = k + 2 * KB, raw = v + 2 * KB;
    static constexpr int steps = raw + RAW * 2 * PB;           // [4] step scales
    static constexpr int rsc = steps + 4 * 32;                 // [RAW] page scales
    static constexpr int bars = rsc + RAW * 8;
    static constexpr int n_bars = 4 * RAW + 8 + 2 + 6 + 1 + 1;
    static constexpr int misc = bars + n_bars * 8;             // tensor-memory base, abort flag
    static constexpr int cum = misc + 16;
    static constexpr size_t bytes = 1024 + cum + (MAX_GROUPS + 1) * 4;
};

struct StepScale {      // of the two pages of a step: K scale (negative: no keys), log2 and reciprocal of V's
    float ks[2], ev[2], iv[2], pad[2];
};

__device__ __forceinline__ void stsm_x4(void* p, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(smem_u32(p)), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// Bounded wait that gives up early once another role has given up.
__device__ __forceinline__ bool wait_or(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int site) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > 2000000000ull) {
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

template <typename T, int HD, bool KEYS>
__global__ void __launch_bounds__(TC_THREADS, 1)
kv8_attn_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                   const Kv8AttnArgs a) {
    using L = TcSmem<HD, KEYS>;
    constexpr int R = L::RAW, PB = L::PB;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    StepScale* steps = reinterpret_cast<StepScale*>(sm + L::steps);
    float2* rsc = reinterpret_cast<float2*>(sm + L::rsc);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint64_t *rawk_full = bars, *rawk_empty = bars + R, *rawv_full = bars + 2 * R, *rawv_empty = bars + 3 * R,
             *k_full = bars + 4 * R, *k_empty = k_full + 2, *v_full = k_full + 4, *v_empty = k_full + 6,
             *q_full = k_full + 8, *q_free = q_full + 1, *s_full = q_full + 2, *p_full = q_full + 4,
             *o_done = q_full + 6, *handed = q_full + 8, *drain = q_full + 9;
    uint32_t* tmem_base = reinterpret_cast<uint32_t*>(sm + L::misc);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::misc + 4);
    int* cum = reinterpret_cast<int*>(sm + L::cum);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_trigger();
    if (tid == 0) {
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
        for (int i = 0; i < R; ++i) {
            mbar_init(rawk_full + i, 1);
            mbar_init(rawk_empty + i, N_CONV);
            mbar_init(rawv_full + i, 1);
            mbar_init(rawv_empty + i, N_CONV);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + i, N_CONV);
            mbar_init(k_empty + i, 1);
            mbar_init(v_full + i, N_CONV);
            mbar_init(v_empty + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(o_done + i, 1);
        }
        mbar_init(q_full, KEYS ? 4 : 8);
        mbar_init(q_free, 1);
        mbar_init(handed, 4);
        mbar_init(drain, 1);
        fence_mbar_init();
        *abort = 0;
    }
    pdl_wait();
    if (warp == MMA_WARP) tc::tmem_alloc(tmem_base, 512);
    tc::fence_before_sync();
    count_items<TC_THREADS>(a, cum);   // ends with a barrier
    tc::fence_after_sync();
    const int total = total_items(a, cum);
    const uint32_t tm = *tmem_base;

    if (warp < 8) {
        // ---------------------------------------------------------- softmax
        const int t = warp >> 2, r = tid & 127;      // group, row of its tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_tm = tm + t * 128 + lanes, o_tm = tm + 256 + t * 128 + lanes;
        unsigned cs = 0, xs = 0, base = 0, items = 0;   // this group's steps, hand-overs, all steps, items so far
        bool ok = true;
        for (int item = blockIdx.x; item < total && ok; item += gridDim.x, ++items) {
            Seq q;
            const Item w = find_item(a, cum, item, &q);
            // the issuing thread is done with the item before: Q is free, and no
            // group is further ahead than the next item
            if (items > 0) {
                ok = __all_sync(0xffffffffu, wait_or(q_free, (items - 1) & 1, abort, a.err, SITE_TC));
                if (!ok) break;
            }
            const int n = (w.p1 - w.p0 + 1) / 2, nt = group_steps<KEYS>(a, q, w, t);
            const int pr = w.tile * a.tile + (KEYS ? 0 : t * 128) + r;
            const int qi = pr / a.group, hq = w.kh * a.group + pr % a.group;
            const bool real = qi < q.n;
            int klo = 0, khi = 0;
            float fr;
            {
                // q: this thread's row, scaled into f16
                uint4 e[HD / 8];
                float top = 0.f;
                if (real) {
                    const T* src = reinterpret_cast<const T*>(a.q) + (long long)(q.r0 + qi) * a.q_row + (long long)hq * a.q_head;
#pragma unroll
                    for (int k = 0; k < HD / 8; ++k) e[k] = reinterpret_cast<const uint4*>(src)[k];
                    row_keys(a, q, qi, &klo, &khi);
                } else {
#pragma unroll
                    for (int k = 0; k < HD / 8; ++k) e[k] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < HD / 8; ++k) {
                    const T* ev = reinterpret_cast<const T*>(&e[k]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float x = fabsf(to_f32(ev[j]));
                        top = fmaxf(top, x < INFINITY ? x : 0.f);
                    }
                }
                float inv, back;
                row_factor(top, &inv, &back);
                fr = back * a.scale_log2;
                if (!KEYS || t == 0) {
                    uint8_t* qs = sm + L::q + (KEYS ? 0 : t * L::QB);
#pragma unroll
                    for (int k = 0; k < HD / 8; ++k) {
                        const T* ev = reinterpret_cast<const T*>(&e[k]);
                        uint4 h;
                        uint32_t* hw = reinterpret_cast<uint32_t*>(&h);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            hw[j] = pack_f16x2(to_f32(ev[2 * j]) * inv, to_f32(ev[2 * j + 1]) * inv);
                        *reinterpret_cast<uint4*>(qs + (k >> 3) * 128 * 128 + swz128(r, k & 7)) = h;
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full);
                }
            }

            float M = -INFINITY, l = 0.f;
            for (int i = 0; i < nt && ok; ++i, ++cs) {
                const int j = KEYS ? 2 * i + t : i;
                ok = __all_sync(0xffffffffu, wait_or(s_full + t, cs & 1, abort, a.err, SITE_TC + 1));
                if (!ok) break;
                tc::fence_after_sync();
                const StepScale sc = steps[(base + j) & 3];
                const int k0 = (w.p0 + 2 * j) * KV8_PAGE;
                bool whole[2];
                float f[2];
                float mx = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f[h] = fr * sc.ks[h];
                    const int kp = k0 + h * KV8_PAGE;
                    whole[h] = kp >= w.in_lo && kp + KV8_PAGE <= w.in_hi;
                    if (sc.ks[h] < 0.f) continue;
                    float m = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v[32];
                        tc::ld_x32(s_tm + h * 64 + c * 32, v);
                        if (whole[h]) {
#pragma unroll
                            for (int x = 0; x < 32; ++x) m = fmaxf(m, v[x]);
                        } else {
                            const int lo = klo - (kp + c * 32), hi = khi - (kp + c * 32);
#pragma unroll
                            for (int x = 0; x < 32; ++x) m = fmaxf(m, x >= lo && x < hi ? v[x] : -INFINITY);
                        }
                    }
                    mx = fmaxf(mx, fmaf(m, f[h], sc.ev[h]));
                }
                // move the reference where this row's maximum has risen far
                const bool need = mx > M + LAZY || (M == -INFINITY && mx > -INFINITY);
                if (__any_sync(0xffffffffu, need)) {
                    const float f0 = need ? (M == -INFINITY ? 0.f : ex2(M - mx)) : 1.f;
                    if (need) M = mx;
                    l *= f0;
                    if (i > 0) {
                        ok = __all_sync(0xffffffffu, wait_or(o_done + t, (cs - 1) & 1, abort, a.err, SITE_TC + 2));
                        if (!ok) break;
                        tc::fence_after_sync();
                        for (int c = 0; c < HD / 32; ++c) {
                            float v[32];
                            tc::ld_x32(o_tm + c * 32, v);
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] *= f0;
                            tc::st_x32(o_tm + c * 32, v);
                        }
                    }
                }
                const float m0 = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int kp = k0 + h * KV8_PAGE;
                    const float off = sc.ev[h] - m0;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t p[16];
                        if (sc.ks[h] < 0.f) {
#pragma unroll
                            for (int x = 0; x < 16; ++x) p[x] = 0;
                        } else {
                            float v[32];
                            tc::ld_x32(s_tm + h * 64 + c * 32, v);
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] = fmaf(v[x], f[h], off);
                            if (!whole[h]) {
                                const int lo = klo - (kp + c * 32), hi = khi - (kp + c * 32);
#pragma unroll
                                for (int x = 0; x < 32; ++x) v[x] = x >= lo && x < hi ? v[x] : -INFINITY;
                            }
#pragma unroll
                            for (int x = 0; x < 32; ++x) {
                                v[x] = ex2(v[x]);
                                sum[x & 3] += v[x];
                            }
#pragma unroll
                            for (int x = 0; x < 16; ++x) p[x] = pack_f16x2(v[2 * x], v[2 * x + 1]);
                        }
                        tc::st_x16(s_tm + h * 32 + c * 16, p);
                    }
                    l = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), sc.iv[h], l);
                }
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

            if (KEYS && t == 1) {
                // (max, sum) go over the scores; the first group's warps read them
                // and the outputs, as they see the same lanes
                if (nt > 0) {
                    tc::st_x2(s_tm, M, l);
                    tc::st_wait();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(handed);
                }
                continue;
            }
            float fa = 1.f, fb = 0.f;
            const bool two = KEYS && group_steps<KEYS>(a, q, w, 1) > 0;
            if (two) {
                ok = __all_sync(0xffffffffu, wait_or(handed, xs & 1, abort, a.err, SITE_TC + 4));
                if (!ok) break;
                ++xs;
                tc::fence_after_sync();
                float bm, bl;
                tc::ld_x2(s_tm + 128, &bm, &bl);
                const float m = fmaxf(M, bm);
                fa = M == -INFINITY ? 0.f : ex2(M - m);
                fb = bm == -INFINITY ? 0.f : ex2(bm - m);
                l = (l != 0.f ? l * fa : 0.f) + (bl != 0.f ? bl * fb : 0.f);   // a NaN sum stays one
                M = m;
            }

            // ---- the row's outputs, or its partial of this split
            const int wi = KEYS ? warp : t * 4 + (warp & 3);
            const long long slot0 = (long long)item - w.split;    // splits of a tile are neighbours
            const long long tk = (((long long)q.r0 * a.group / a.tile + w.s + w.tile) * a.n_kv + w.kh) * 8 + wi;
            const bool split = q.splits > 1;
            const bool fits = !split || (slot0 + q.splits <= a.part_cap && tk < a.ticket_cap);   // by the plan's bounds
            const int RT = a.tile;
            const long long PL = (long long)RT * (HD + 4);         // floats of a partial
            const int prow = KEYS ? r : t * 128 + r;
            float* part = split ? a.part + (slot0 + w.split) * PL : nullptr;
            T* dst = reinterpret_cast<T*>(a.out) + (long long)(q.r0 + qi) * a.out_row + (long long)hq * a.out_head;
            const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that sees no key: zeros
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                float v[32];
                __syncwarp();
                if (nt > 0) {
                    tc::ld_x32(o_tm + c * 32, v);
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = 0.f;
                }
                if (two) {
                    float u[32];
                    tc::ld_x32(o_tm + 128 + c * 32, u);
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = fmaf(u[x], fb, v[x] * fa);
                }
                if (real && split && fits) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        reinterpret_cast<float4*>(part)[(size_t)(c * 8 + x) * RT + prow] =
                            make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                }
                if (real && !split) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float o[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) o[x] = v[16 * b + x];
                        store16<T>(dst + c * 32 + 16 * b, o, inv);
                    }
                }
            }
            __syncwarp();
            tc::fence_before_sync();   // the accumulator has been read
            if (!split) {
                if (real && a.lse)
                    a.lse[(long long)(q.r0 + qi) * a.n_q + hq] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
                continue;
            }
            if (real && fits) reinterpret_cast<float2*>(part + (size_t)RT * HD)[prow] = make_float2(M, l);
            __threadfence();
            __syncwarp();
            int last = 0;
            if (lane == 0) last = fits && atomicAdd(a.tickets + tk, 1) == q.splits - 1;
            last = __shfl_sync(0xffffffffu, last, 0);
            if (!last) continue;
            __threadfence();
            if (lane == 0) a.tickets[tk] = 0;
            if (!real) continue;
            // the last split's warp folds its rows of all splits, in split order
            const float* src = a.part + slot0 * PL;
            float fm = -INFINITY, fl = 0.f;
            for (int v = 0; v < q.splits; ++v)
                fm = fmaxf(fm, __ldcg(&reinterpret_cast<const float2*>(src + v * PL + (size_t)RT * HD)[prow]).x);
            for (int v = 0; v < q.splits; ++v) {
                const float2 x = __ldcg(&reinterpret_cast<const float2*>(src + v * PL + (size_t)RT * HD)[prow]);
                fl = fmaf(x.y, x.x == -INFINITY ? 0.f : ex2(x.x - fm), fl);
            }
            const float finv = fl == 0.f ? 0.f : 1.f / fl;
            for (int b = 0; b < HD / 16; ++b) {
                float o[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] = 0.f;
                for (int v = 0; v < q.splits; ++v) {
                    const float m = __ldcg(&reinterpret_cast<const float2*>(src + v * PL + (size_t)RT * HD)[prow]).x;
                    const float f = m == -INFINITY ? 0.f : ex2(m - fm);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float4 y = __ldcg(&reinterpret_cast<const float4*>(src + v * PL)[(size_t)(b * 4 + x) * RT + prow]);
                        o[4 * x] = fmaf(y.x, f, o[4 * x]);
                        o[4 * x + 1] = fmaf(y.y, f, o[4 * x + 1]);
                        o[4 * x + 2] = fmaf(y.z, f, o[4 * x + 2]);
                        o[4 * x + 3] = fmaf(y.w, f, o[4 * x + 3]);
                    }
                }
                store16<T>(dst + 16 * b, o, finv);
            }
            if (a.lse) a.lse[(long long)(q.r0 + qi) * a.n_q + hq] = fl == 0.f ? -INFINITY : (fm + log2f(fl)) * 0.6931471805599453f;
        }
    } else if (warp < MMA_WARP) {
        // ---------------------------------------------------------- conversion
        const int cw = warp - CONV_WARP;
        unsigned g = 0;     // steps so far
        bool ok = true;
        for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
            Seq q;
            const Item w = find_item(a, cum, item, &q);
            const int n = (w.p1 - w.p0 + 1) / 2;
            for (int j = 0; j < n && ok; ++j, ++g) {
                const int st = g & 1;
                if (g >= 2) ok = __all_sync(0xffffffffu, wait_or(k_empty + st, ((g >> 1) - 1) & 1, abort, a.err, SITE_TC + 5));
                if (!ok) break;
                float2 sc[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const unsigned rs = 2 * g + h;
                    ok = __all_sync(0xffffffffu, wait_or(rawk_full + rs % R, (rs / R) & 1, abort, a.err, SITE_TC + 6));
                    if (!ok) break;
                    sc[h] = rsc[rs % R];
                    if (sc[h].x < 0.f) continue;
                    const uint8_t* src = sm + L::raw + (rs % R) * PB;
                    uint8_t* dst = sm + L::k + st * L::KB;
#pragma unroll
                    for (int x = cw; x < HD / 8; x += N_CONV) {
                        const int key = (x & 1) * 32 + lane, c = x >> 1;     // 16 dims of a key
                        const uint4 e = lds128(src + tile_off<HD>(key, c));
                        const uint32_t ew[4] = {e.x, e.y, e.z, e.w};
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
                }
                if (!ok) break;
                if (cw == 0 && lane < 2) {
                    const float2 s = lane ? sc[1] : sc[0];
                    StepScale* d = steps + (g & 3);
                    d->ks[lane] = s.y > 0.f ? s.x : -1.f;
                    d->ev[lane] = s.y > 0.f ? log2f(s.y) : 0.f;
                    d->iv[lane] = s.y > 0.f ? 1.f / s.y : 0.f;
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(k_full + st);
                    mbar_arrive(rawk_empty + (2 * g) % R);
                    mbar_arrive(rawk_empty + (2 * g + 1) % R);
                }
                if (g >= 2) ok = __all_sync(0xffffffffu, wait_or(v_empty + st, ((g >> 1) - 1) & 1, abort, a.err, SITE_TC + 7));
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const unsigned rs = 2 * g + h;
                    ok = __all_sync(0xffffffffu, wait_or(rawv_full + rs % R, (rs / R) & 1, abort, a.err, SITE_TC + 6));
                    if (!ok) break;
                    const uint8_t* src = sm + L::raw + (R + rs % R) * PB;
                    uint8_t* dst = sm + L::v + st * L::KB + h * HD * 128;
                    const bool valid = sc[h].x >= 0.f && sc[h].y > 0.f;
                    const int kp = (w.p0 + 2 * j + h) * KV8_PAGE;
                    // codes of keys that no row sees may be anything, NaN included: as zeros
                    const bool edge = kp < w.lo || kp + KV8_PAGE > w.hi;
#pragma unroll
                    for (int x = cw; x < HD / 8; x += N_CONV) {
                        const int kb = x & 1, d = x >> 1;        // 32 keys, 16 dims
                        uint32_t r4[4] = {0, 0, 0, 0};
                        if (valid) {
                            ldsm_x4_trans(r4, src + tile_off<HD>(kb * 32 + lane, d));
                            if (edge) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int k = kp + kb * 32 + 8 * i + 2 * (lane & 3);
                                    r4[i] &= (k >= w.lo && k < w.hi ? 0x0000ffffu : 0u) |
                                             (k + 1 >= w.lo && k + 1 < w.hi ? 0xffff0000u : 0u);
                                }
                            }
                        }
                        uint32_t e[4], o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t p = __byte_perm(r4[i], 0, 0x3120);
                            e[i] = f16_of_codes(p);
                            o[i] = f16_of_codes(p >> 16);
                        }
                        const int row = 16 * d + (lane & 7), ch = 4 * kb + (lane >> 3);
                        stsm_x4(dst + swz128(row, ch), e);
                        stsm_x4(dst + swz128(row + 8, ch), o);
                    }
                }
                if (!ok) break;
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(v_full + st);
                    mbar_arrive(rawv_empty + (2 * g) % R);
                    mbar_arrive(rawv_empty + (2 * g + 1) % R);
                }
            }
        }
    } else if (warp == MMA_WARP) {
        // ---------------------------------------------------------- MMAs
        if (lane == 0) {
            constexpr uint32_t IS = tc::idesc_f16_f32(128, STEP), IO = tc::idesc_f16_f32(128, HD);
            unsigned base = 0, items = 0, done[2] = {0, 0};
            bool ok = true;
            for (int item = blockIdx.x; item < total && ok; item += gridDim.x, ++items) {
                Seq q;
                const Item w = find_item(a, cum, item, &q);
                const int n = (w.p1 - w.p0 + 1) / 2;
                const int nt[2] = {group_steps<KEYS>(a, q, w, 0), group_steps<KEYS>(a, q, w, 1)};
                ok = wait_or(q_full, items & 1, abort, a.err, SITE_TC + 8);
                auto qk = [&](int t, int i) -> bool {
                    const unsigned g = base + (KEYS ? 2 * i + t : i);
                    const int st = g & 1;
                    if (!wait_or(k_full + st, (g >> 1) & 1, abort, a.err, SITE_TC + 9)) return false;
                    tc::fence_after_sync();
                    const uint8_t* qs = sm + L::q + (KEYS ? 0 : t * L::QB);
                    const uint8_t* ks = sm + L::k + st * L::KB;
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        tc::mma_f16(tm + t * 128, tc::desc_sw128(qs + (k >> 2) * 128 * 128 + (k & 3) * 32),
                                    tc::desc_sw128(ks + (k >> 2) * STEP * 128 + (k & 3) * 32), IS, k > 0);
                    tc::commit(s_full + t);
                    if (KEYS || t == 1 || nt[1] == 0) tc::commit(k_empty + st);
                    return true;
                };
                for (int t = 0; t < 2 && ok; ++t)
                    if (nt[t] > 0) ok = qk(t, 0);
                for (int i = 0; i < nt[0] && ok; ++i)
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (i >= nt[t]) continue;
                        const unsigned g = base + (KEYS ? 2 * i + t : i);
                        const int st = g & 1;
                        ok = wait_or(p_full + t, (done[t] + i) & 1, abort, a.err, SITE_TC + 10) &&
                             wait_or(v_full + st, (g >> 1) & 1, abort, a.err, SITE_TC + 11);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const uint8_t* vs = sm + L::v + st * L::KB;
#pragma unroll
                        for (int k = 0; k < STEP / 16; ++k)
                            tc::mma_f16_ta(tm + 256 + t * 128, tm + t * 128 + 8 * k,
                                           tc::desc_sw128(vs + (k >> 2) * HD * 128 + (k & 3) * 32), IO, i > 0 || k > 0);
                        tc::commit(o_done + t);
                        if (KEYS || t == 1 || nt[1] == 0) tc::commit(v_empty + st);
                        if (i + 1 < nt[t]) ok = qk(t, i + 1);
                    }
                done[0] += nt[0];
                done[1] += nt[1];
                base += n;
                if (ok) tc::commit(q_free);
            }
            // every MMA has finished before tensor memory is given back
            tc::commit(drain);
            mbar_wait_bounded(drain, 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- pages
        unsigned it = 0, ik = 0;   // pages issued: both tensors', K's
        bool ok = true;
        for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
            Seq q;
            const Item w = find_item(a, cum, item, &q);
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
                const int m = slots - b < 32 ? slots - b : 32;
                for (int j = 0; j < m; ++j) {
                    const int pg = __shfl_sync(0xffffffffu, page, j);
                    const float kj = __shfl_sync(0xffffffffu, ks, j), vj = __shfl_sync(0xffffffffu, vs, j);
                    const int st = it % R;
                    bool issued = true;
                    if (lane == 0) {
                        const int y = (pg * a.n_kv + w.kh) * KV8_PAGE;
                        const uint32_t par = (it / R - 1) & 1;
                        issued = it < R || wait_or(rawk_empty + st, par, abort, a.err, SITE_TC + 12);
                        if (issued) {
                            rsc[st] = make_float2(kj, vj);
                            if (pg >= 0) {
                                mbar_arrive_expect_tx(rawk_full + st, PB);
                                tma_load_2d(sm + L::raw + st * PB, &k_map, rawk_full + st, 0, y);
                            } else {
                                mbar_arrive(rawk_full + st);
                            }
                            ++ik;
                            issued = it < R || wait_or(rawv_empty + st, par, abort, a.err, SITE_TC + 12);
                        }
                        if (issued) {
                            if (pg >= 0) {
                                mbar_arrive_expect_tx(rawv_full + st, PB);
                                tma_load_2d(sm + L::raw + (R + st) * PB, &v_map, rawv_full + st, 0, y);
                            } else {
                                mbar_arrive(rawv_full + st);
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
        }
        // no copy of this CTA is in flight when it ends
        if (lane == 0) {
            const unsigned nk = ik < R ? ik : R, nv = it < R ? it : R;
            for (unsigned i = ik - nk; i < ik; ++i) mbar_wait_bounded(rawk_full + i % R, (i / R) & 1);
            for (unsigned i = it - nv; i < it; ++i) mbar_wait_bounded(rawv_full + i % R, (i / R) & 1);
        }
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == MMA_WARP) tc::tmem_dealloc(tm, 512);
}

template <typename T, int HD, bool KEYS>
int launch_tc(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a, int sms, cudaStream_t s) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv8_attn_tc_kernel<T, HD, KEYS>));
    if (e != cudaSuccess) return (int)e;
    const long long most = a.ticket_cap / 8 * a.split_cap;   // items there can be
    const long long grid = most < sms ? most : sms;
    return (int)launch_k(kv8_attn_tc_kernel<T, HD, KEYS>, dim3((unsigned)grid), dim3(TC_THREADS),
                         TcSmem<HD, KEYS>::bytes, s, k_map, v_map, a);
}

template <typename T>
int launch_tc_t(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a, int form, int hd,
                int sms, cudaStream_t s) {
    if (form == KV8_TC_KEYS)
        return hd == 128 ? launch_tc<T, 128, true>(k_map, v_map, a, sms, s) : launch_tc<T, 64, true>(k_map, v_map, a, sms, s);
    return hd == 128 ? launch_tc<T, 128, false>(k_map, v_map, a, sms, s) : launch_tc<T, 64, false>(k_map, v_map, a, sms, s);
}

}  // namespace

int launch_kv8_attention_tc(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a,
                            int form, int head_dim, int sms, cudaStream_t s) {
    return a.dtype == 1 ? launch_tc_t<__nv_bfloat16>(k_map, v_map, a, form, head_dim, sms, s)
                        : launch_tc_t<__half>(k_map, v_map, a, form, head_dim, sms, s);
}

}  // namespace dfl
