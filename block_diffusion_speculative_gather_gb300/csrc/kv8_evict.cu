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
// The choice: one CTA a sequence, a radix selection over the weights' bits (11, 11
// and 10 of them), then one pass in order.  The keys lie in shared memory, up to
// 49152 positions; those of longer sequences are looked up again in every pass.
//
// The move: a position only ever moves to a lower or its own place, so a page may
// be written once the positions that go into it and into lower pages have been
// read.  A CTA has one kv head's K or V of a sequence and layer and does its pages
// in order, four at a time: the next four are on their way while four are
// written, which none of them reads.

#include "gemm.cuh"
#include "kv8.cuh"
#include "kv8_attn_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;

constexpr int ST = 1024, SW = ST / 32;
constexpr int BINS = 2048;
constexpr int KEYS = 49152;           // held in shared memory

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
    __syncthreads();       // the sums before have been read
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    int w = sm[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    return (warp ? before : 0) + inc - v;
}

__global__ void __launch_bounds__(ST) kv8_choose_kernel(const __grid_constant__ Kv8EvictArgs a) {
    extern __shared__ uint32_t keys[];      // [min(n, KEYS)]
    __shared__ int hist[BINS], sm[32], s_bin, s_left, s_bad, s_moved;
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x, tid = threadIdx.x;
    const long long cap = (long long)a.max_pages * KV8_PAGE;
    const int* table = a.table + (size_t)s * a.max_pages;
    const int n = a.kv_len[s], b = a.budget[s];
    bool bad = n < 0 || n > cap;
    const int pages = bad ? 0 : (n + KV8_PAGE - 1) / KV8_PAGE;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    for (int p = tid; p < pages; p += ST) {
        const int pg = table[p];
        if (pg < 0 || pg >= a.n_pages) s_bad = 1;
    }
    __syncthreads();
    const int site = bad ? SITE_LEN : SITE_PAGE;
    bad = bad || s_bad;
    const bool goes = !bad && b > 0 && n > b;
    const int kept = goes ? b : n;
    if (tid == 0) {
        if (bad) report(a.err, DERR_INDEX, site);
        a.new_len[s] = kept;
        if (a.dropped && goes) a.dropped[s] += n - b;
        if (bad) a.first_moved[s] = kept;
        s_moved = kept;
    }
    if (bad) return;
    int* source = a.source + (size_t)s * cap;
    int* from = a.from + (size_t)s * cap;
    auto place = [&](int j) { return (size_t)table[j / KV8_PAGE] * KV8_PAGE + j % KV8_PAGE; };
    const int last = goes ? min(a.keep_last, b) : 0, first = goes ? min(a.keep_first, b - last) : n;
    const int want = kept - last - first;             // of positions first .. n - last - 1
    uint32_t prefix = 0;
    int left = want;                                  // of those with this prefix
    if (want > 0) {
        const int from_j = first, to_j = n - last;
        const bool held = to_j - from_j <= a.keys;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < BINS; i += ST) hist[i] = 0;
            __syncthreads();
            for (int j0 = from_j; j0 < to_j; j0 += 4 * ST) {
                uint32_t k[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j = j0 + u * ST + tid;
                    if (j >= to_j) continue;
                    if (held && pass) k[u] = keys[j - from_j];
                    else k[u] = key_of_weight(a.weights[place(j)]);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j = j0 + u * ST + tid;
                    if (j >= to_j) continue;
                    if (held && !pass) keys[j - from_j] = k[u];
                    if (pass == 0 || (k[u] ^ prefix) >> (shift + bits) == 0) atomicAdd(hist + ((k[u] >> shift) & ((1 << bits) - 1)), 1);
                }
            }
            __syncthreads();
            // bins from the top: a thread has two
            const int hi = hist[BINS - 1 - 2 * tid], lo = hist[BINS - 2 - 2 * tid];
            int total;
            const int above = block_exclusive(hi + lo, &total, sm);
            if (above < left && above + hi + lo >= left) {
                const bool top = above + hi >= left;
                s_bin = BINS - (top ? 1 : 2) - 2 * tid;
                s_left = left - above - (top ? 0 : hi);
            }
            __syncthreads();
            prefix |= (uint32_t)s_bin << shift;
            left = s_left;
        }
    }
    // in order: positions with larger keys, and the first `left` with this one.
    // A thread has four in a row at a time.
    int ties = 0, out = 0, moved = kept;
    for (int base = 0; base < n; base += 4 * ST) {
        float w[4];
        bool tie[4], stays[4];
        size_t at_slot[4];
        int my_ties = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = base + 4 * tid + u;
            tie[u] = stays[u] = false;
            if (j >= n) continue;
            at_slot[u] = place(j);
            w[u] = a.weights[at_slot[u]];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = base + 4 * tid + u;
            if (j >= n) continue;
            stays[u] = j < first || j >= n - last;
            if (!stays[u] && want > 0) {
                const uint32_t k = key_of_weight(w[u]);
                stays[u] = k > prefix;
                tie[u] = k == prefix;
                my_ties += tie[u];
            }
        }
        int total;
        int rank = ties + block_exclusive(my_ties, &total, sm), mine = 0;
        ties += total;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (tie[u]) stays[u] = rank++ < left;
            mine += stays[u];
        }
        int at = out + block_exclusive(mine, &total, sm);
        out += total;
        // every weight of these positions has been read, here and by the others
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (!stays[u]) continue;
            const int j = base + 4 * tid + u;
            source[at] = j;
            from[at] = (int)at_slot[u];
            if (at != j) moved = min(moved, at);
            if (at != j || a.weights_out != a.weights) a.weights_out[place(at)] = w[u];
            ++at;
        }
    }
    moved = (int)__reduce_min_sync(0xffffffffu, (unsigned)moved);
    if ((tid & 31) == 0) atomicMin(&s_moved, moved);
    __syncthreads();
    if (tid == 0) a.first_moved[s] = s_moved;
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

constexpr int MT = 512;               // threads of the move
constexpr int MP = 4;                 // pages at a time
constexpr int MROWS = MP * KV8_PAGE;

template <int HD>
__global__ void __launch_bounds__(MT, 2) kv8_move_kernel(const __grid_constant__ Kv8EvictArgs a,
                                                         const __grid_constant__ Kv8MoveLayers l) {
    constexpr int PER_ROW = HD / 16, N = MROWS * PER_ROW / MT;      // uint4s of a row, of a thread
    __shared__ float s_scale[2][MROWS];
    __shared__ float s_top[2][MROWS / 32];
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x / a.n_kv, head = blockIdx.x % a.n_kv, layer = blockIdx.y, which = blockIdx.z, tid = threadIdx.x;
    const int kept = a.new_len[s], begin = a.first_moved[s];
    if (begin >= kept) return;
    const long long cap = (long long)a.max_pages * KV8_PAGE;
    const int* from = a.from + (size_t)s * cap;
    const int* table = a.table + (size_t)s * a.max_pages;
    uint8_t* codes = which ? l.v_codes[layer] : l.k_codes[layer];
    float* scale = which ? l.v_scale[layer] : l.k_scale[layer];
    uint4 x[N], y[N];
    int slot[N], scale_slot = 0;
    float sc = 0.f;
    // slots of the positions d0 .. that this thread reads
    auto look = [&](int d0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int d = d0 + (i * MT + tid) / PER_ROW;
            slot[i] = d < kept ? from[d] : -1;
        }
        if (tid < MROWS) scale_slot = d0 + tid < kept ? from[d0 + tid] : -1;
    };
    auto fetch = [&](uint4 (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (slot[i] >= 0) {
                const size_t at = ((size_t)(slot[i] / KV8_PAGE) * a.n_kv + head) * KV8_PAGE + slot[i] % KV8_PAGE;
                v[i] = reinterpret_cast<const uint4*>(codes + at * HD)[(i * MT + tid) % PER_ROW];
            }
        if (tid < MROWS) sc = scale_slot >= 0 ? scale[(size_t)(scale_slot / KV8_PAGE) * a.n_kv + head] : 0.f;
    };
    int d0 = begin / KV8_PAGE * KV8_PAGE;
    look(d0);
    fetch(x);
    look(d0 + MROWS);
    for (int turn = 0; d0 < kept; d0 += MROWS, turn ^= 1) {
        if (tid < MROWS) {
            s_scale[turn][tid] = sc;
            const float top = warp_max(sc);
            if ((tid & 31) == 0) s_top[turn][tid >> 5] = top;
        }
        // these pages have been read, by every thread
        __syncthreads();
        fetch(y);
        look(d0 + 2 * MROWS);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = (i * MT + tid) / PER_ROW, d = d0 + row;
            if (d >= kept) continue;
            const float top = fmaxf(s_top[turn][row / KV8_PAGE * 2], s_top[turn][row / KV8_PAGE * 2 + 1]);
            if (s_scale[turn][row] != top) {
                const float f = s_scale[turn][row] / top;
                x[i] = make_uint4(rescale4(x[i].x, f), rescale4(x[i].y, f), rescale4(x[i].z, f), rescale4(x[i].w, f));
            }
            const size_t at = ((size_t)table[d / KV8_PAGE] * a.n_kv + head) * KV8_PAGE + d % KV8_PAGE;
            reinterpret_cast<uint4*>(codes + at * HD)[(i * MT + tid) % PER_ROW] = x[i];
        }
        if (tid < MP && d0 + tid * KV8_PAGE < kept)
            scale[(size_t)table[d0 / KV8_PAGE + tid] * a.n_kv + head] = fmaxf(s_top[turn][2 * tid], s_top[turn][2 * tid + 1]);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = y[i];
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

int launch_kv8_evict(const Kv8EvictArgs& args, const Kv8MoveLayers& l, bool choose, int head_dim, cudaStream_t s) {
    Kv8EvictArgs a = args;
    const long long cap = (long long)a.max_pages * KV8_PAGE;
    a.keys = (int)(cap < KEYS ? cap : KEYS);
    if (choose) {
        cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv8_choose_kernel));
        if (e == cudaSuccess)
            e = launch_k(kv8_choose_kernel, dim3((unsigned)a.S), dim3(ST), (size_t)a.keys * 4, s, a);
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
