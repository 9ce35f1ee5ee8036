// Appends rows of K and V to the 8-bit paged cache.
//
// A run is a maximal stretch of rows with consecutive slots inside one page.
// Per run, kv head and tensor: the scale is the smallest power of two 2^e
// with amax <= 448 * 2^e (e clamped to [-100, 119]), never below the page's
// old scale unless the run starts the page; a raised scale re-rounds the
// page's earlier codes (exact except where they fall below the format's
// normal range, as powers of two only move the exponent); the rows become
// code = e4m3(x / scale), round to nearest even, saturating.  NaN stays NaN;
// an infinity saturates and does not enter the scale.
//
// Runs of one page that follow one another in the call (skipped rows between
// them, slots repeated or out of order) are a chain and are done in row order
// by the same threads, so a repeated slot keeps its last row.
//
// Work: rows are read once into registers (largest magnitude, then codes) and
// written once at 8 bits.  A CTA takes a window of rows and finds the chains
// that begin in it: a few long ones (prompts) are done by the whole CTA one
// after another, many short ones (single tokens) a warp each.
//
// Bound: at many rows by the chain of each CTA (slots, rows, maximum, codes:
// three dependent trips to memory), which four CTAs an SM do not hide: four
// ragged prompts of 10000 f16 rows x 8 kv heads of 128 take 24 us where their
// bytes take 9 (2.6 TB/s); at few by latency: 32 rows 3.4 us.

#include "gemm.cuh"
#include "kv8.cuh"

namespace dfl {
namespace {

constexpr int AT = 128;          // threads
constexpr int AW = AT / 32;
constexpr int WIN_MAX = 64;      // rows of a window

// Smallest power of two that brings amax within the format's 448.
__device__ __forceinline__ float scale_of(float amax) {
    if (!(amax > 0.f)) return 0x1p-100f;
    int e;
    const float m = frexpf(amax, &e);          // amax = m 2^e, m in [0.5, 1)
    e = m <= 0.875f ? e - 9 : e - 8;           // 448 = 0.875 * 2^9
    e = e < -100 ? -100 : (e > 119 ? 119 : e);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four values to four codes (the first in the lowest byte).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ float2 decode2(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(two));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.f;   // NaN compares false
}

// Eight elements of a row, as they stand and as fp32.
template <typename T> struct alignas(16) Unit {
    T e[8];
};

template <typename T, bool WIDE>
__device__ __forceinline__ void load8(const T* p, Unit<T>& u) {
    if (WIDE) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 8 / V; ++i)
            reinterpret_cast<uint4*>(u.e)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) u.e[i] = p[i];
    }
}

// One run: n rows from row r0 into page `page` at offset `off`, by `nt`
// threads of which this is `t` (a warp or the CTA).  A unit is 8 elements of
// a row; a thread keeps up to KEEP units in registers (a whole page's run of
// the CTA, or 16 rows of a warp at head_dim 128), so that they are read once.
// (10000 rows of ragged prompts: 256 threads keeping 4 units 4 % slower.)
constexpr int KEEP = 8;

template <typename T, int HD, bool WIDE, bool CTA>
__device__ __forceinline__ void run_append(const Kv8AppendArgs& a, int which, int head, int r0, int n, int page,
                                           int off, int t, float* red) {
    constexpr int PER_ROW = HD / 8, NT = CTA ? AT : 32;
    const long long ld = which ? a.row[1] : a.row[0];
    const T* x = reinterpret_cast<const T*>(which ? a.x[1] : a.x[0]) + (long long)r0 * ld +
                 (long long)head * (which ? a.head[1] : a.head[0]);
    float* sp = (which ? a.scale[1] : a.scale[0]) + (long long)page * a.n_kv + head;
    uint8_t* codes = (which ? a.codes[1] : a.codes[0]) + ((long long)page * a.n_kv + head) * KV8_PAGE * HD;
    const float old = off > 0 ? *sp : 0.f;
    const int total = n * PER_ROW;
    Unit<T> v[KEEP];
    float top = 0.f;
    for (int base = 0; base < total; base += KEEP * NT) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const int i = base + k * NT + t;
            if (i < total) load8<T, WIDE>(x + (long long)(i / PER_ROW) * ld + (i % PER_ROW) * 8, v[k]);
        }
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (base + k * NT + t < total) {
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(to_f32(v[k].e[j])));
            }
    }
    top = warp_max(top);
    if (CTA) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < AW; ++i) top = fmaxf(top, red[i]);
        __syncthreads();
    }
    float sc = scale_of(top);
    if (off > 0) {
        if (old >= sc) {
            sc = old;
        } else {
            const float f = old * (1.f / sc);   // a power of two below 1
            for (int i = t; i < off * PER_ROW; i += NT) {
                uint2* p = reinterpret_cast<uint2*>(codes) + i;
                uint2 c = *p;
                uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 lo = decode2(w[j] & 0xffffu), hi = decode2(w[j] >> 16);
                    w[j] = codes4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
                }
                *p = c;
            }
        }
    }
    if (CTA) __syncthreads();   // everyone has read the old scale
    else __syncwarp();
    if (t == 0) *sp = sc;
    const float inv = 1.f / sc;   // exact: scales are powers of two
    for (int base = 0; base < total; base += KEEP * NT) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const int i = base + k * NT + t;
            if (i >= total) continue;
            if (total > KEEP * NT) load8<T, WIDE>(x + (long long)(i / PER_ROW) * ld + (i % PER_ROW) * 8, v[k]);
            uint2 c;
            const T* e = v[k].e;
            c.x = codes4(to_f32(e[0]) * inv, to_f32(e[1]) * inv, to_f32(e[2]) * inv, to_f32(e[3]) * inv);
            c.y = codes4(to_f32(e[4]) * inv, to_f32(e[5]) * inv, to_f32(e[6]) * inv, to_f32(e[7]) * inv);
            reinterpret_cast<uint2*>(codes + (long long)off * HD)[i] = c;
        }
    }
    if (CTA) __syncthreads();   // the next run of the chain reads this one's codes and scale
    else __syncwarp();
}

template <typename T, int HD, bool WIDE>
__global__ void __launch_bounds__(AT) kv8_append_kernel(Kv8AppendArgs a, int win) {
    __shared__ int s_slot[2 * WIN_MAX + 1];   // slots of the window, the row before and the longest run behind
    __shared__ int s_run[WIN_MAX], s_n;
    __shared__ float red[AW];
    pdl_trigger();
    pdl_wait();
    const int w0 = blockIdx.x * win, head = blockIdx.y, which = blockIdx.z;
    const int rows = a.rows - w0 < win ? a.rows - w0 : win;   // rows of this window
    const int tid = threadIdx.x;
    const long long cap = (long long)a.n_pages * KV8_PAGE;
    for (int i = tid; i < 1 + rows + KV8_PAGE; i += AT) {
        const int r = w0 + i - 1;
        int sl = r >= 0 && r < a.rows ? a.slots[r] : -1;
        if (sl >= cap) {     // a slot outside the pool: reported, the row is skipped
            if (a.err && atomicCAS(a.err, 0, DERR_INDEX) == 0) a.err[1] = r;
            sl = -1;
        }
        s_slot[i] = sl;
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
    const int n_seen = 1 + rows + KV8_PAGE;
    auto slot_at = [&](int r) -> int {   // of any row: -1 for skipped ones
        const int i = r - w0 + 1;
        if (i >= 0 && i < n_seen) return s_slot[i];
        const int sl = a.slots[r];
        return sl >= cap ? -1 : sl;
    };
    // the first row from r on (step 1) or back (step -1) that is not skipped, for
    // a whole warp; -1 if there is none.  512 rows at a time, all loads in
    // flight: a padded call has many behind its last (32 of 4096 rows in use:
    // row by row 455 us, so 21 us).
    auto next_row = [&](int r, int step) -> int {
        if (r >= 0 && r < a.rows && slot_at(r) >= 0) return r;
        for (long long b = r; b >= 0 && b < a.rows; b += 512 * step) {
            unsigned first = ~0u;
#pragma unroll
            for (int k = 15; k >= 0; --k) {
                const int d = 32 * k + (tid & 31);
                const long long x = b + (long long)step * d;
                if (x >= 0 && x < a.rows) {
                    const int sl = a.slots[x];
                    if (sl >= 0 && sl < cap) first = d;
                }
            }
            first = __reduce_min_sync(0xffffffffu, first);
            if (first != ~0u) return (int)(b + (long long)step * (int)first);
        }
        return -1;
    };
    // chains that begin in the window, in row order (a warp's ballots): rows on
    // another page than the last row before them that is not skipped
    if (tid < 32) {
        int n = 0, last = -2;      // page of the last row so far; -2: not looked up
        for (int b = 0; b < rows; b += 32) {
            const int i = b + tid, sl = i < rows ? s_slot[i + 1] : -1, page = sl >= 0 ? sl / KV8_PAGE : -1;
            const unsigned valid = __ballot_sync(0xffffffffu, sl >= 0);
            if (!valid) continue;
            if (last == -2) {
                const int r = next_row(w0 - 1, -1);
                last = r < 0 ? -1 : slot_at(r) / KV8_PAGE;
            }
            const unsigned below = valid & ((1u << tid) - 1);
            const int from = __shfl_sync(0xffffffffu, page, below ? 31 - __clz(below) : 0);
            const bool begins = sl >= 0 && (below ? from : last) != page;
            const unsigned m = __ballot_sync(0xffffffffu, begins);
            if (begins) s_run[n + __popc(m & ((1u << tid) - 1))] = i;
            n += __popc(m);
            last = __shfl_sync(0xffffffffu, page, 31 - __clz(valid));
        }
        if (tid == 0) s_n = n;
    }
    __syncthreads();
    const int n_runs = s_n;
    // up to two chains: the whole CTA on each; more: a warp each
    const bool by_cta = n_runs <= 2;
    for (int k = by_cta ? 0 : tid >> 5; k < n_runs; k += by_cta ? 1 : AW) {
        int r = w0 + s_run[k], sl = slot_at(r);
        const int page = sl / KV8_PAGE;
        while (true) {
            const int off = sl % KV8_PAGE;
            // rows that follow on, 64 tested at once by each warp
            unsigned on[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int d = 32 * h + (tid & 31);
                on[h] = __ballot_sync(0xffffffffu, off + d < KV8_PAGE && r + d < a.rows && slot_at(r + d) == sl + d);
            }
            const int n = ~on[0] ? __ffs(~on[0]) - 1 : 32 + (~on[1] ? __ffs(~on[1]) - 1 : 32);
            if (by_cta) run_append<T, HD, WIDE, true>(a, which, head, r, n, page, off, tid, red);
            else run_append<T, HD, WIDE, false>(a, which, head, r, n, page, off, tid & 31, red);
            r = next_row(r + n, 1);
            if (r < 0) break;
            sl = slot_at(r);
            if (sl / KV8_PAGE != page) break;
        }
    }
}

template <typename T>
int launch_append_t(const Kv8AppendArgs& a, cudaStream_t s) {
    // Window: one row while the grid stays small (a decode step's rows are
    // runs of their own and each gets a CTA), 64 rows (about a page's run)
    // for prompts.
    const int win = a.rows <= 256 ? 1 : WIN_MAX;
    const dim3 grid((unsigned)((a.rows + win - 1) / win), (unsigned)a.n_kv, 2);
    if (a.head_dim == 128)
        return (int)(a.wide ? launch_k(kv8_append_kernel<T, 128, true>, grid, dim3(AT), 0, s, a, win)
                            : launch_k(kv8_append_kernel<T, 128, false>, grid, dim3(AT), 0, s, a, win));
    return (int)(a.wide ? launch_k(kv8_append_kernel<T, 64, true>, grid, dim3(AT), 0, s, a, win)
                        : launch_k(kv8_append_kernel<T, 64, false>, grid, dim3(AT), 0, s, a, win));
}

}  // namespace

int launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t s) {
    if (a.dtype == 0) return launch_append_t<float>(a, s);
    if (a.dtype == 1) return launch_append_t<__nv_bfloat16>(a, s);
    return launch_append_t<__half>(a, s);
}

}  // namespace dfl
