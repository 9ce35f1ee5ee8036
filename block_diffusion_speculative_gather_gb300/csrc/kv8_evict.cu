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
// and 10 of them), then one pass in order.  Up to 8192 positions the weights stay
// in registers, eight a thread; the keys of longer sequences lie in shared memory
// up to 49152 positions and are looked up again in every pass above.  It is a chain
// of three trips to memory and about 20 barriers, 8 us of a call whatever the number of
// sequences.
//
// The move: a position only ever moves to a lower or its own place, so a page may
// be written once the positions that go into it and into lower pages have been
// read.  A CTA has one kv head's K or V of a sequence and layer and goes through
// its pages in order, 16 KB at a time, by a ring in shared memory: the copies of
// the next three turns are on their way while one is written, which none of them
// reads.  Where CTAs are few, a cluster shares the pages of a turn; its barrier stands
// between a turn's reads and its writes.  Bound by DRAM where
// sequences and layers are many: 8 of up to 6000 positions to 2500, 10 layers of 8 heads of
// 128, move 818 MB in 139 us with the choice, 5.9 TB/s (three turns in the ring 152 us).
// One of 4095 to 2048, 5 layers: 22.3 us (18.6 with the pools in L2), the choice and a
// chain of turns; of 8192 to 4096 33.7, of 8193 44.1, where the choice looks its weights up.

#include "cluster_dev.cuh"
#include "copy_dev.cuh"
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

constexpr int HELD = 8;               // keys of a thread
constexpr int SHORT = ST * HELD;      // positions whose keys the threads hold

// One digit of the selection, once the bins are counted: the bin that the
// `left`-th largest key falls into and what is left of it there, two bins a thread.
__device__ __forceinline__ void pick_bin(const int* hist, int* sm, int* s_bin, int* s_left, int left) {
    const int tid = threadIdx.x, hi = hist[BINS - 1 - 2 * tid], lo = hist[BINS - 2 - 2 * tid];
    int total;
    const int above = block_exclusive(hi + lo, &total, sm);
    if (above < left && above + hi + lo >= left) {
        const bool top = above + hi >= left;
        *s_bin = BINS - (top ? 1 : 2) - 2 * tid;
        *s_left = left - above - (top ? 0 : hi);
    }
    __syncthreads();
}

// Counts of (u, warp) in hist to the counts before each, by warp 0.
__device__ __forceinline__ void counts_before(int* hist) {
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int run[HELD], sum = 0;
#pragma unroll
        for (int u = 0; u < HELD; ++u) run[u] = hist[lane * HELD + u], sum += run[u];
        int before = warp_inclusive(sum, lane) - sum;
#pragma unroll
        for (int u = 0; u < HELD; ++u) hist[lane * HELD + u] = before, before += run[u];
    }
    __syncthreads();
}

__global__ void __launch_bounds__(ST) kv8_choose_kernel(const __grid_constant__ Kv8EvictArgs a) {
    extern __shared__ uint32_t keys[];      // [a.keys]
    __shared__ int hist[BINS], sm[SW], s_bin, s_left, s_bad, s_moved;
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
            uint32_t prefix = 0;
            int left = want;                          // of those with this prefix
            for (int pass = 0; pass < 3; ++pass) {
                const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
                hist[tid] = hist[tid + ST] = 0;
                __syncthreads();
#pragma unroll
                for (int u = 0; u < HELD; ++u)
                    if (in[u] && (pass == 0 || (key[u] ^ prefix) >> (shift + bits) == 0))
                        atomicAdd(hist + ((key[u] >> shift) & ((1 << bits) - 1)), 1);
                __syncthreads();
                pick_bin(hist, sm, &s_bin, &s_left, left);
                prefix |= (uint32_t)s_bin << shift;
                left = s_left;
            }
            // the first `left` of those with this key, in order of u, then of threads
            int mine[HELD];
#pragma unroll
            for (int u = 0; u < HELD; ++u) {
                const unsigned m = __ballot_sync(0xffffffffu, in[u] && key[u] == prefix);
                mine[u] = __popc(m & ((1u << lane) - 1));
                if (lane == 0) hist[u * SW + warp] = __popc(m);
            }
            counts_before(hist);
#pragma unroll
            for (int u = 0; u < HELD; ++u)
                if (in[u]) stays[u] = key[u] > prefix || (key[u] == prefix && hist[u * SW + warp] + mine[u] < left);
            __syncthreads();
        }
        int mine[HELD];
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const unsigned m = __ballot_sync(0xffffffffu, stays[u]);
            mine[u] = __popc(m & ((1u << lane) - 1));
            if (lane == 0) hist[u * SW + warp] = __popc(m);
        }
        counts_before(hist);
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
                pick_bin(hist, sm, &s_bin, &s_left, left);
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

constexpr int MT = 256;               // threads of the move
constexpr int MN = 4;                 // 16-byte pieces of a thread a turn
constexpr int MS = 4;                 // turns in the ring
constexpr int MRANKS = 8;             // CTAs of a cluster at most

template <int HD> struct MoveSmem {
    static constexpr int rows = MT * MN * 16 / HD;                  // of a CTA and turn: whole pages
    uint4 codes[MS][MT * MN];
    float scale[MS][rows];                                          // the rows' old scales
};

template <int HD>
__global__ void __launch_bounds__(MT, 3) kv8_move_kernel(const __grid_constant__ Kv8EvictArgs a,
                                                         const __grid_constant__ Kv8MoveLayers l, int ranks) {
    using S_ = MoveSmem<HD>;
    constexpr int PER_ROW = HD / 16, ROWS = S_::rows, PAGES = ROWS / KV8_PAGE, STEP = MT / PER_ROW;
    static_assert(ROWS % KV8_PAGE == 0 && ROWS <= MT && KV8_PAGE % STEP == 0, "whole pages at a time");
    extern __shared__ __align__(16) uint8_t raw[];
    S_& sm = *reinterpret_cast<S_*>(raw);
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const int chain = blockIdx.x / ranks, rank = blockIdx.x - chain * ranks, s = chain / a.n_kv, head = chain - s * a.n_kv;
    const int layer = blockIdx.y, which = blockIdx.z;
    const int kept = a.new_len[s], begin = a.first_moved[s];
    if (begin >= kept) return;                                      // all of a cluster
    const int* from = a.from + (size_t)s * ((long long)a.max_pages * KV8_PAGE);
    const int* table = a.table + (size_t)s * a.max_pages;
    const int c = tid % PER_ROW, r0 = tid / PER_ROW;                // this thread's piece of rows r0, r0 + STEP, ..
    uint8_t* codes = (which ? l.v_codes[layer] : l.k_codes[layer]) + (size_t)head * KV8_PAGE * HD + c * 16;
    float* scale = (which ? l.v_scale[layer] : l.k_scale[layer]) + head;
    const int page_rows = a.n_kv * KV8_PAGE;                        // rows of a page, all heads (rows fit int32)
    auto row_of = [&](int slot) { return (size_t)(unsigned)((slot / KV8_PAGE) * page_rows + slot % KV8_PAGE) * HD; };
    const int base = begin / KV8_PAGE * KV8_PAGE + rank * ROWS, turn_rows = ranks * ROWS;
    const int turns = (kept - begin / KV8_PAGE * KV8_PAGE + turn_rows - 1) / turn_rows;
    int slot[MN], scale_slot = -1;
    auto look = [&](int t) {            // where the positions of turn t come from
        const int d0 = base + t * turn_rows;
#pragma unroll
        for (int i = 0; i < MN; ++i) {
            const int d = d0 + r0 + i * STEP;
            slot[i] = t < turns && d < kept ? from[d] : -1;
        }
        scale_slot = t < turns && tid < ROWS && d0 + tid < kept ? from[d0 + tid] : -1;
    };
    auto fetch = [&](int t) {           // the copies of turn t (an empty group behind the last)
#pragma unroll
        for (int i = 0; i < MN; ++i)
            if (slot[i] >= 0) copy_async16(&sm.codes[t % MS][i * MT + tid], codes + row_of(slot[i]));
        if (scale_slot >= 0) copy_async4(&sm.scale[t % MS][tid], scale + (size_t)(scale_slot / KV8_PAGE) * a.n_kv);
        copy_commit();
    };
    look(0);
#pragma unroll
    for (int t = 0; t < MS - 1; ++t) {
        fetch(t);
        look(t + 1);
    }
    int page[PAGES];                    // of the turn at hand
    auto pages_at = [&](int t) {
#pragma unroll
        for (int i = 0; i < PAGES; ++i) {
            const int d = base + t * turn_rows + i * KV8_PAGE;
            page[i] = t < turns && d < kept ? table[d / KV8_PAGE] : 0;
        }
    };
    pages_at(0);
    for (int t = 0; t < turns; ++t) {
        copy_wait<MS - 2>();
        // This thread's copies of the turn are complete.  The barrier makes them the CTA's (a
        // row's scale comes by one thread and is read by all), and the ring's place of turn
        // t - 1 has been read.
        __syncthreads();
        // The other CTAs write where this one has read: one thread's fence stands for the CTA's
        // reads, which the barrier above has put before it.
        if (ranks > 1) {
            if (tid == 0) fence_cluster();
            cluster_arrive_relaxed();
        }
        fetch(t + MS - 1);              // into the ring's place of turn t - 1
        look(t + MS);
        const int d0 = base + t * turn_rows;
        float top[PAGES];
#pragma unroll
        for (int i = 0; i < PAGES; ++i) {
            const int d = d0 + i * KV8_PAGE;
            const float* sc = sm.scale[t % MS] + i * KV8_PAGE;
            top[i] = warp_max(fmaxf(d + lane < kept ? sc[lane] : 0.f, d + 32 + lane < kept ? sc[32 + lane] : 0.f));
        }
        if (ranks > 1) cluster_wait();  // the turn's positions have been read, by all who read any of them
#pragma unroll
        for (int i = 0; i < PAGES; ++i)
            if (tid == 0 && d0 + i * KV8_PAGE < kept) scale[(size_t)page[i] * a.n_kv] = top[i];
#pragma unroll
        for (int i = 0; i < MN; ++i) {
            const int row = r0 + i * STEP, d = d0 + row;
            if (d >= kept) continue;
            const int pi = i * STEP / KV8_PAGE;                     // the same for all of the thread's i-th rows
            uint4 x = sm.codes[t % MS][i * MT + tid];
            const float own = sm.scale[t % MS][row];
            if (own != top[pi]) {
                const float f = own * (1.f / top[pi]);              // exact: powers of two
                if ((__float_as_uint(f) & 0x807fffffu) == 0) {
                    const __half2 h = __float2half2_rn(f);
                    x = make_uint4(rescale4_f16(x.x, h), rescale4_f16(x.y, h), rescale4_f16(x.z, h), rescale4_f16(x.w, h));
                } else {
                    x = make_uint4(rescale4(x.x, f), rescale4(x.y, f), rescale4(x.z, f), rescale4(x.w, f));
                }
            }
            *reinterpret_cast<uint4*>(codes + row_of(page[pi] * KV8_PAGE + d % KV8_PAGE)) = x;
        }
        pages_at(t + 1);
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
    const int chains = a.S * a.n_kv;
    // Three CTAs of the move run on an SM.  Few chains: as many CTAs each as run at once (one
    // sequence of 4095 positions to 2048, 5 layers, pools in L2: 18.6 us, by one CTA each 28.3).  More
    // than run at once: two each where that takes at least an eighth less rounds (of 6000
    // positions to 2500: 576 chains 91 us, by one CTA each 113; 960 chains 117 and 124; where
    // it does not, 1280 chains 147 and 139).
    const long long all = 2LL * chains * l.n, room = 3LL * sms;
    int ranks = 1;
    while (ranks < MRANKS && all * ranks * 2 <= room) ranks *= 2;
    if (ranks == 1 && 8 * ((all * 2 + room - 1) / room) <= 14 * ((all + room - 1) / room)) ranks = 2;
    const dim3 grid((unsigned)(chains * ranks), (unsigned)l.n, 2), block(MT);
    auto go = [&](auto kern, size_t smem) {
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern));
        return (int)(e == cudaSuccess ? launch_cluster_k(kern, grid, block, ranks, s, smem, a, l, ranks) : e);
    };
    return head_dim == 128 ? go(kv8_move_kernel<128>, sizeof(MoveSmem<128>)) : go(kv8_move_kernel<64>, sizeof(MoveSmem<64>));
}

int launch_pages_shift(const PagesShiftArgs& a, cudaStream_t s) {
    const long long n = a.rows > a.S ? a.rows : a.S;
    return (int)launch_k(pages_shift_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
}

}  // namespace dfl
