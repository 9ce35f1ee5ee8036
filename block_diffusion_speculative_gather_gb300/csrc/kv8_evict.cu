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
// The choice: one CTA a sequence.  Up to 8192 positions their weights stay in
// registers, eight a thread, and the budget's smallest weight is found bit by bit,
// two bits a round; longer ones take a radix selection (11, 11 and 10 bits), the
// keys in shared memory up to 49152 positions, looked up again above.  Then one
// pass in order.
//
// The move: a position only ever moves to a lower or its own place, so a page may
// be written once the positions that go into it and into lower pages have been
// read.  A CTA has one kv head's K or V of a sequence and layer (or a part of its
// dims, where they are few) and goes through the pages in order, 32 KB at a time:
// the next ones are on their way while these are written, which none of them
// reads.

#include "cluster_dev.cuh"
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

// The smallest key that stays of `want` (above 0) among the keys of positions
// first .. to - 1, and how many of those that have it.
struct Border {
    uint32_t key;
    int ties;
};

constexpr int HELD = 8;               // keys of a thread
constexpr int SHORT = ST * HELD;      // positions whose keys the threads hold

// key[u] is position u * ST + tid's; 0 .. 2^32 - 1 are searched two bits at a time,
// as counts of keys at or above three borders (at most SHORT, 14 bits: two in a
// word's halves would not do, so three words).
__device__ __forceinline__ Border border_of_held(const uint32_t (&key)[HELD], const bool (&in)[HELD], int want, int* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t low = 0;                 // at least `want` keys are at or above it
    int above = 0;                    // keys above the searched range
    for (int shift = 30; shift >= 0; shift -= 2) {
        int c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const uint32_t d = in[u] && key[u] >= low ? (key[u] - low) >> shift : 0;   // 3 and more: above the range, too
            c1 += d >= 1;
            c2 += d >= 2;
            c3 += d >= 3;
        }
        c1 = __reduce_add_sync(0xffffffffu, c1);
        c2 = __reduce_add_sync(0xffffffffu, c2);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        int* at = sm + (shift & 2) * (3 * SW / 2);      // in turn: one barrier a round
        if (lane == 0) at[warp] = c1, at[SW + warp] = c2, at[2 * SW + warp] = c3;
        __syncthreads();
        c1 = __reduce_add_sync(0xffffffffu, at[lane]);
        c2 = __reduce_add_sync(0xffffffffu, at[SW + lane]);
        c3 = __reduce_add_sync(0xffffffffu, at[2 * SW + lane]);
        // the highest quarter that still leaves `want`
        if (c3 >= want) low += 3u << shift;
        else if (c2 >= want) low += 2u << shift, above = c3;
        else if (c1 >= want) low += 1u << shift, above = c2;
        else above = c1;
    }
    return {low, want - above};
}

__global__ void __launch_bounds__(ST) kv8_choose_kernel(const __grid_constant__ Kv8EvictArgs a) {
    extern __shared__ uint32_t keys[];      // [a.keys]
    __shared__ int hist[BINS], sm[2 * 3 * SW], s_bin, s_left, s_bad, s_moved;
    __shared__ int s_table[SHORT / KV8_PAGE];
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
        if (p < SHORT / KV8_PAGE) s_table[p] = pg;
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
    const int last = goes ? min(a.keep_last, b) : 0, first = goes ? min(a.keep_first, b - last) : n;
    const int want = kept - last - first;             // of positions first .. n - last - 1
    int moved = kept;
    if (n <= SHORT) {
        auto place = [&](int j) { return s_table[j / KV8_PAGE] * KV8_PAGE + j % KV8_PAGE; };
        float w[HELD];
        uint32_t key[HELD];
        bool in[HELD], stays[HELD];
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const int j = u * ST + tid;
            w[u] = j < n ? a.weights[place(j)] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const int j = u * ST + tid;
            key[u] = key_of_weight(w[u]);
            in[u] = j >= first && j < n - last;
            stays[u] = j < n && !in[u];
        }
        if (want > 0) {
            const Border r = border_of_held(key, in, want, sm);
            // the first `ties` of those on the border, in order of u, then of threads
            __syncthreads();
            int mine[HELD];
#pragma unroll
            for (int u = 0; u < HELD; ++u) {
                const unsigned m = __ballot_sync(0xffffffffu, in[u] && key[u] == r.key);
                mine[u] = __popc(m & ((1u << lane) - 1));
                if (lane == 0) hist[u * SW + warp] = __popc(m);
            }
            __syncthreads();
            if (warp == 0) {                          // HELD * SW counts, HELD a lane
                int run[HELD], sum = 0;
#pragma unroll
                for (int u = 0; u < HELD; ++u) run[u] = hist[lane * HELD + u], sum += run[u];
                int before = warp_inclusive(sum, lane) - sum;
#pragma unroll
                for (int u = 0; u < HELD; ++u) hist[lane * HELD + u] = before, before += run[u];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < HELD; ++u) {
                if (!in[u]) continue;
                stays[u] = key[u] > r.key || (key[u] == r.key && hist[u * SW + warp] + mine[u] < r.ties);
            }
            __syncthreads();
        }
        int mine[HELD];
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const unsigned m = __ballot_sync(0xffffffffu, stays[u]);
            mine[u] = __popc(m & ((1u << lane) - 1));
            if (lane == 0) hist[u * SW + warp] = __popc(m);
        }
        __syncthreads();
        if (warp == 0) {
            int run[HELD], sum = 0;
#pragma unroll
            for (int u = 0; u < HELD; ++u) run[u] = hist[lane * HELD + u], sum += run[u];
            int before = warp_inclusive(sum, lane) - sum;
#pragma unroll
            for (int u = 0; u < HELD; ++u) hist[lane * HELD + u] = before, before += run[u];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            if (!stays[u]) continue;
            const int j = u * ST + tid, at = hist[u * SW + warp] + mine[u];
            source[at] = j;
            from[at] = place(j);
            if (at != j) moved = min(moved, at);
            if (at != j || a.weights_out != a.weights) a.weights_out[place(at)] = w[u];
        }
    } else {
        auto place = [&](int j) { return (size_t)table[j / KV8_PAGE] * KV8_PAGE + j % KV8_PAGE; };
        uint32_t prefix = 0;
        int left = want;                              // of those with this prefix
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
                        if (pass == 0 || (k[u] ^ prefix) >> (shift + bits) == 0)
                            atomicAdd(hist + ((k[u] >> shift) & ((1 << bits) - 1)), 1);
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
        int ties = 0, out = 0;
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
    }
    moved = (int)__reduce_min_sync(0xffffffffu, (unsigned)moved);
    if (lane == 0) atomicMin(&s_moved, moved);
    __syncthreads();
    if (tid == 0) a.first_moved[s] = s_moved;
}

// Four codes times a factor.
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

// The same by a power of two of at most 1, in f16: a code times 2^-15 is exact
// there, what is below lies far under half of the format's smallest step.
__device__ __forceinline__ uint32_t rescale4_f16(uint32_t w, __half2 f) {
    const uint32_t lo = f16_of_codes(w), hi = f16_of_codes(w >> 16);
    const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&lo), f), b = __hmul2(*reinterpret_cast<const __half2*>(&hi), f);
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r) : "r"(*reinterpret_cast<const uint32_t*>(&a)), "r"(*reinterpret_cast<const uint32_t*>(&b)));
    return r;
}

constexpr int MT = 512;               // threads of the move
constexpr int MN = 4;                 // 16-byte pieces of a thread at a time

// PB: bytes of a row that the CTA moves (a row, or 32 of it: the parts' CTAs are a
// cluster, since they read the scales that the first one writes).
template <int HD, int PB>
__global__ void __launch_bounds__(MT, 2) kv8_move_kernel(const __grid_constant__ Kv8EvictArgs a,
                                                         const __grid_constant__ Kv8MoveLayers l) {
    constexpr int PER_ROW = PB / 16, ROWS = MT * MN / PER_ROW, PARTS = HD / PB, PAGES = ROWS / KV8_PAGE;
    constexpr int EACH = (ROWS + MT - 1) / MT;                      // rows whose scales a thread looks up
    __shared__ float s_ratio[2][ROWS];
    __shared__ float s_top[2][ROWS / 32];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const int part = blockIdx.x % PARTS, chain = blockIdx.x / PARTS, s = chain / a.n_kv, head = chain - s * a.n_kv;
    const int layer = blockIdx.y, which = blockIdx.z;
    const int kept = a.new_len[s], begin = a.first_moved[s];
    if (begin >= kept) return;
    const int* from = a.from + (size_t)s * ((long long)a.max_pages * KV8_PAGE);
    const int* table = a.table + (size_t)s * a.max_pages;
    const int c = tid % PER_ROW, r0 = tid / PER_ROW;                // this thread's piece of rows r0, r0 + MT / PER_ROW, ..
    uint8_t* codes = (which ? l.v_codes[layer] : l.k_codes[layer]) + (size_t)head * KV8_PAGE * HD + part * PB + c * 16;
    float* scale = (which ? l.v_scale[layer] : l.k_scale[layer]) + head;
    const int page_rows = a.n_kv * KV8_PAGE;                        // rows of a page, all heads (slots x heads fit int32)
    auto row_of = [&](int slot) { return (size_t)(unsigned)((slot / KV8_PAGE) * page_rows + slot % KV8_PAGE) * HD; };
    uint4 x[MN], y[MN];
    int slot[MN], scale_slot[EACH];
    float sc[EACH];
    // slots of the positions d0 .. that this thread reads
    auto look = [&](int d0) {
#pragma unroll
        for (int i = 0; i < MN; ++i) {
            const int d = d0 + r0 + i * (MT / PER_ROW);
            slot[i] = d < kept ? from[d] : -1;
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int d = d0 + e * MT + tid;
            scale_slot[e] = e * MT + tid < ROWS && d < kept ? from[d] : -1;
        }
    };
    auto fetch = [&](uint4 (&v)[MN]) {
#pragma unroll
        for (int i = 0; i < MN; ++i)
            if (slot[i] >= 0) v[i] = *reinterpret_cast<const uint4*>(codes + row_of(slot[i]));
#pragma unroll
        for (int e = 0; e < EACH; ++e) sc[e] = scale_slot[e] >= 0 ? scale[(size_t)(scale_slot[e] / KV8_PAGE) * a.n_kv] : 0.f;
    };
    int d0 = begin / KV8_PAGE * KV8_PAGE;
    look(d0);
    fetch(x);
    look(d0 + ROWS);
    for (int turn = 0; d0 < kept; d0 += ROWS, turn ^= 1) {
        float own[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            own[e] = sc[e];
            const float top = warp_max(sc[e]);
            if (lane == 0 && e * MT + tid < ROWS) s_top[turn][(e * MT + tid) >> 5] = top;
        }
        // these pages have been read, by every thread (of the row's other parts, too)
        if (PARTS > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        fetch(y);
        look(d0 + 2 * ROWS);
        // a row's factor; -1: as it is
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int row = e * MT + tid;
            if (row >= ROWS) continue;
            const float top = fmaxf(s_top[turn][row / KV8_PAGE * 2], s_top[turn][row / KV8_PAGE * 2 + 1]);
            s_ratio[turn][row] = own[e] == top ? -1.f : own[e] / top;
            const int d = d0 + row;
            if (part == 0 && row % KV8_PAGE == 0 && d < kept) scale[(size_t)table[d / KV8_PAGE] * a.n_kv] = top;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MN; ++i) {
            const int row = r0 + i * (MT / PER_ROW), d = d0 + row;
            if (d >= kept) continue;
            const float f = s_ratio[turn][row];
            if (f != -1.f) {
                if ((__float_as_uint(f) & 0x807fffffu) == 0) {      // a power of two (or 0)
                    const __half2 h = __float2half2_rn(f);
                    x[i] = make_uint4(rescale4_f16(x[i].x, h), rescale4_f16(x[i].y, h), rescale4_f16(x[i].z, h),
                                      rescale4_f16(x[i].w, h));
                } else {
                    x[i] = make_uint4(rescale4(x[i].x, f), rescale4(x[i].y, f), rescale4(x[i].z, f), rescale4(x[i].w, f));
                }
            }
            *reinterpret_cast<uint4*>(codes + row_of(table[d / KV8_PAGE] * KV8_PAGE + d % KV8_PAGE)) = x[i];
        }
#pragma unroll
        for (int i = 0; i < MN; ++i) x[i] = y[i];
    }
    static_assert(PAGES >= 1 && ROWS % KV8_PAGE == 0, "whole pages at a time");
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

int launch_kv8_evict(const Kv8EvictArgs& args, const Kv8MoveLayers& l, bool choose, int head_dim, int sms, cudaStream_t s) {
    Kv8EvictArgs a = args;
    const long long cap = (long long)a.max_pages * KV8_PAGE;
    a.keys = (int)(cap < KEYS ? cap : KEYS);
    if (choose) {
        cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv8_choose_kernel));
        if (e == cudaSuccess)
            e = launch_k(kv8_choose_kernel, dim3((unsigned)a.S), dim3(ST), (size_t)a.keys * 4, s, a);
        if (e != cudaSuccess) return (int)e;
    }
    // parts of 32 bytes a row while whole rows leave SMs without work: a CTA then has
    // that many more pages at a time
    const bool parts = 2LL * a.S * a.n_kv * l.n < sms;
    const int each = parts ? head_dim / 32 : 1;
    const dim3 grid((unsigned)(a.S * a.n_kv * each), (unsigned)l.n, 2), block(MT);
    if (head_dim == 128)
        return (int)(parts ? launch_cluster_k(kv8_move_kernel<128, 32>, grid, block, each, s, a, l)
                           : launch_k(kv8_move_kernel<128, 128>, grid, block, 0, s, a, l));
    return (int)(parts ? launch_cluster_k(kv8_move_kernel<64, 32>, grid, block, each, s, a, l)
                       : launch_k(kv8_move_kernel<64, 64>, grid, block, 0, s, a, l));
}

int launch_pages_shift(const PagesShiftArgs& a, cudaStream_t s) {
    const long long n = a.rows > a.S ? a.rows : a.S;
    return (int)launch_k(pages_shift_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
}

}  // namespace dfl
