// Eviction from the 8-bit paged cache.
//
// A sequence of n positions with a budget b < n keeps its first f, its last l
// and, of those between, the b - f - l heaviest (equal weights: the lower
// positions).  What stays moves down in order, so that positions 0 .. b - 1
// hold it, in every layer's pools.  A page's new scale is the largest of the
// pages its positions came from; codes from a page with a smaller one are
// rounded to it (powers of two: exact but where values fall below the format's
// normal range).
//
// The choice: one CTA a sequence, a radix selection over the weights' bits (8 at
// a time), then one pass in order.  The move: a position only ever moves to a
// lower or its own place, so a page may be written once the positions that go
// into it and into lower pages have been read: a CTA has one kv head's K or V of
// a sequence and layer and does its pages in order.

#include "gemm.cuh"
#include "kv8.cuh"
#include "kv8_attn_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;

constexpr int ST = 1024;

// Larger weights have larger keys; NaN is below all.
__device__ __forceinline__ uint32_t key_of_weight(float w) { return w == w ? float_orderable(w + 0.f) : 0u; }

// Exclusive sum over the CTA, and the total.
__device__ __forceinline__ int block_exclusive(int v, int* total, int* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = sm[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += x;
        }
        sm[lane] = w;
    }
    __syncthreads();
    const int before = warp ? sm[warp - 1] : 0;
    *total = sm[31];
    __syncthreads();
    return before + inc - v;
}

__global__ void __launch_bounds__(ST) kv8_choose_kernel(Kv8EvictArgs a) {
    __shared__ int hist[256], sm[32], s_bin, s_left, s_bad;
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x, tid = threadIdx.x;
    const long long cap = (long long)a.max_pages * KV8_PAGE;
    const int* table = a.table + (size_t)s * a.max_pages;
    const int n = a.kv_len[s];
    if (tid == 0) s_bad = 0;
    __syncthreads();
    bool bad = n < 0 || n > cap;
    if (!bad)
        for (int p = tid; p < (n + KV8_PAGE - 1) / KV8_PAGE; p += ST) {
            const int pg = table[p];
            if (pg < 0 || pg >= a.n_pages) s_bad = 1;
        }
    __syncthreads();
    bad = bad || s_bad;
    const int b = a.budget[s];
    const bool goes = !bad && b > 0 && n > b;
    const int kept = goes ? b : n;
    if (tid == 0) {
        if (bad) report(a.err, DERR_INDEX, n < 0 || n > cap ? SITE_LEN : SITE_PAGE);
        a.new_len[s] = kept;
        if (a.dropped && goes) a.dropped[s] += n - b;
        a.first_moved[s] = kept;
    }
    if (bad) return;
    int* source = a.source + (size_t)s * cap;
    int* from = a.from + (size_t)s * cap;
    auto weight = [&](int j) { return a.weights[(size_t)table[j / KV8_PAGE] * KV8_PAGE + j % KV8_PAGE]; };
    const int last = goes ? min(a.keep_last, b) : 0, first = goes ? min(a.keep_first, b - last) : n;
    const int want = kept - last - first;             // of positions first .. n - last - 1
    uint32_t prefix = 0;
    int left = want;                                  // of those with this prefix
    if (want > 0)
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += ST) hist[i] = 0;
            __syncthreads();
            for (int j = first + tid; j < n - last; j += ST) {
                const uint32_t k = key_of_weight(weight(j));
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(hist + ((k >> shift) & 255), 1);
            }
            __syncthreads();
            if (tid == 0) {
                int bin = 255, rest = left;
                while (rest > hist[bin]) rest -= hist[bin--];
                s_bin = bin;
                s_left = rest;
            }
            __syncthreads();
            prefix |= (uint32_t)s_bin << shift;
            left = s_left;
            __syncthreads();
        }
    // in order: positions with larger keys, and the first `left` with this one
    int ties = 0, out = 0;
    for (int base = 0; base < n; base += ST) {
        const int j = base + tid;
        bool tie = false, stays = false;
        float w = 0.f;
        if (j < n) {
            w = weight(j);
            stays = j < first || j >= n - last;
            if (!stays && want > 0) {
                const uint32_t k = key_of_weight(w);
                stays = k > prefix;
                tie = k == prefix;
            }
        }
        int total;
        const int rank = block_exclusive(tie, &total, sm);
        stays = stays || (tie && ties + rank < left);
        ties += total;
        const int at = out + block_exclusive(stays, &total, sm);
        out += total;
        // every weight of these positions has been read
        if (stays) {
            source[at] = j;
            from[at] = table[j / KV8_PAGE] * KV8_PAGE + j % KV8_PAGE;
            if (at != j) atomicMin(a.first_moved + s, at);
            a.weights_out[(size_t)table[at / KV8_PAGE] * KV8_PAGE + at % KV8_PAGE] = w;
        }
    }
}

// 16 codes times a factor.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    const uint32_t lo2 = f16_of_codes(w), hi2 = f16_of_codes(w >> 16);
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r) : "f"(lo.x * f), "f"(lo.y * f), "f"(hi.x * f), "f"(hi.y * f));
    return r;
}

constexpr int MT = 128;

template <int HD>
__global__ void __launch_bounds__(MT) kv8_move_kernel(Kv8EvictArgs a, Kv8MoveLayers l) {
    constexpr int PER_ROW = HD / 16, N = KV8_PAGE * PER_ROW / MT;     // uint4s of a row, of a thread
    __shared__ float s_scale[KV8_PAGE];
    __shared__ float s_top[2];
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x / a.n_kv, head = blockIdx.x % a.n_kv, layer = blockIdx.y, which = blockIdx.z, tid = threadIdx.x;
    const int kept = a.new_len[s], begin = a.first_moved[s];
    if (begin >= kept) return;
    const long long cap = (long long)a.max_pages * KV8_PAGE;
    const int* from = a.from + (size_t)s * cap;
    uint8_t* codes = which ? l.v_codes[layer] : l.k_codes[layer];
    float* scale = which ? l.v_scale[layer] : l.k_scale[layer];
    for (int d = begin / KV8_PAGE; d * KV8_PAGE < kept; ++d) {
        const int rows = min(KV8_PAGE, kept - d * KV8_PAGE);
        uint4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = (i * MT + tid) / PER_ROW, c = (i * MT + tid) % PER_ROW;
            if (row < rows) {
                const int slot = from[d * KV8_PAGE + row];
                const size_t at = ((size_t)(slot / KV8_PAGE) * a.n_kv + head) * KV8_PAGE + slot % KV8_PAGE;
                x[i] = reinterpret_cast<const uint4*>(codes + at * HD)[c];
            }
        }
        if (tid < KV8_PAGE) {
            float v = 0.f;
            if (tid < rows) v = scale[(size_t)(from[d * KV8_PAGE + tid] / KV8_PAGE) * a.n_kv + head];
            s_scale[tid] = v;
            const float top = warp_max(v);
            if ((tid & 31) == 0) s_top[tid >> 5] = top;
        }
        __syncthreads();
        const float top = fmaxf(s_top[0], s_top[1]);
        const int pg = a.table[(size_t)s * a.max_pages + d];
        uint8_t* dst = codes + ((size_t)pg * a.n_kv + head) * KV8_PAGE * HD;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = (i * MT + tid) / PER_ROW;
            if (row < rows) {
                if (s_scale[row] != top) {
                    const float f = s_scale[row] / top;
                    x[i] = make_uint4(rescale4(x[i].x, f), rescale4(x[i].y, f), rescale4(x[i].z, f), rescale4(x[i].w, f));
                }
                reinterpret_cast<uint4*>(dst)[i * MT + tid] = x[i];
            }
        }
        if (tid == 0) scale[(size_t)pg * a.n_kv + head] = top;
        __syncthreads();
    }
}

// True positions of a step's rows: the cache's, and those the sequence has lost.
__global__ void pages_shift_kernel(PagesShiftArgs a) {
    pdl_trigger();
    pdl_wait();
    const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (t < a.S) {
        const int r0 = a.row_start[t], r1 = a.row_start[t + 1];
        if (r0 >= 0 && r0 < r1 && r1 <= a.rows && a.positions[r0] == 0) a.dropped[t] = 0;   // begins anew
    }
    if (t >= a.rows) return;
    const int r = (int)t, pos = a.positions[r];
    int out = -1;
    if (pos >= 0) {
        int lo = 0, hi = a.S - 1;      // the last s with row_start[s] <= r
        while (lo < hi) {
            const int mid = (int)(((long long)lo + hi + 1) >> 1);
            if (a.row_start[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        const int r0 = a.row_start[lo];
        out = pos;
        if (r0 >= 0 && r0 <= r && r < a.row_start[lo + 1] && a.positions[r0] != 0) out += a.dropped[lo];
    }
    a.out[r] = out;
}

}  // namespace

int launch_kv8_evict(const Kv8EvictArgs& a, const Kv8MoveLayers& l, bool choose, int head_dim, cudaStream_t s) {
    if (choose) {
        const cudaError_t e = launch_k(kv8_choose_kernel, dim3((unsigned)a.S), dim3(ST), 0, s, a);
        if (e != cudaSuccess) return (int)e;
    }
    const dim3 grid((unsigned)(a.S * a.n_kv), (unsigned)l.n, 2), block(MT);
    return (int)(head_dim == 128 ? launch_k(kv8_move_kernel<128>, grid, block, 0, s, a, l)
                                 : launch_k(kv8_move_kernel<64>, grid, block, 0, s, a, l));
}

int launch_pages_shift(const PagesShiftArgs& a, cudaStream_t s) {
    const long long n = a.rows > a.S ? a.rows : a.S;
    return (int)launch_k(pages_shift_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
}

}  // namespace dfl
