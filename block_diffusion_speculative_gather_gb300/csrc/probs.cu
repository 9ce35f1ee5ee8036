// Probabilities of rows of logits.
//
//   p_v = w_v / sum w,  w_v = exp((x_v - m) / T) where x_v >= m + T ln(min_p), else 0
// with m the row's maximum; T = 0: 1 at the first maximum.  NaN logits count as
// -inf; where the maximum is +inf its holders share the row.
//
// The border m + T ln(min_p) is taken as a pair of fp32 numbers (48 bits) and
// rounded up to the next fp32 value, so that comparing fp32 logits with it is exact.  log2(e) / T is
// held as two fp32 numbers, so that a weight's exponent is off by the
// difference's and the product's rounding alone; weights, sums (of up to 40 terms a
// thread) and quotients are fp32.
//
// A row's maximum is needed before its sum and its sum before its first output:
// the row stays on the SMs between.  A cluster of up to 16 CTAs holds it in
// registers (up to 40 logits a thread), trades maxima and sums through distributed
// shared memory, and writes what it read once.  Rows that all run at once are
// read straight into registers; more of them go through clusters that stay, whose
// next row comes by a bulk copy to shared memory while one is worked on.  Larger
// rows (above 327680 logits) are read three times, by one CTA.
//
// One row of 151936 fp32 logits takes 5.0 us, launch, load, two exchanges and store one
// after the other (6.1 with min_p, for its logarithm in 64 bits).  512 of them move 622 MB in 137 us, 4.5 TB/s: what holds them up is
// each row's two exchanges, in which an SM has no other row to work on, and that clusters
// of 8 with an SM a CTA find room on 120 of the 152 SMs.

#include <mutex>

#include "cluster_dev.cuh"
#include "f32x2.cuh"
#include "gemm.cuh"
#include "kv8.cuh"
#include "sampling.cuh"

namespace dfl {
namespace {

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float no_nan(float x) { return x == x ? x : -INFINITY; }

// A row without one is left as it was.
__device__ __forceinline__ bool has_temperature(float t) { return t >= 0.f && t < INFINITY; }

// What a row's temperature and min_p come to, by one thread.
struct RowSetup {
    float c, c_lo;        // log2(e) / T
    float cut, cut_lo;    // T ln(min_p)
};

__device__ __forceinline__ RowSetup setup_of(float t, float min_p) {
    RowSetup r;
    r.c = fminf(1.44269502f / t, 1e38f);          // no 0 * inf at the smallest T
    // what the quotient and log2(e)'s fp32 value leave over
    r.c_lo = r.c < 1e38f ? (fmaf(-r.c, t, 1.44269502f) + 1.92596303e-8f) / t : 0.f;
    r.cut = -INFINITY;
    r.cut_lo = 0.f;
    if (min_p > 0.f) {
        const double cut = (double)t * log((double)fminf(min_p, 1.f));
        r.cut = (float)cut;
        if (r.cut > -INFINITY) r.cut_lo = (float)(cut - (double)r.cut);
    }
    return r;
}

struct RowRule {
    float m, border;      // maximum (finite), smallest logit that counts (finite)
    float c, c_lo;
};

__device__ __forceinline__ RowRule rule_of(float m, const RowSetup& u) {
    RowRule r{m, -3.402823466e38f, u.c, u.c_lo};
    // m + cut as s + e, exactly, then rounded up
    const float s = __fadd_rn(m, u.cut), b = __fsub_rn(s, m);
    const float e = __fadd_rn(__fsub_rn(m, __fsub_rn(s, b)), __fsub_rn(u.cut, b));
    if (s > -INFINITY) r.border = __fadd_ru(s, __fadd_rn(e, u.cut_lo));
    return r;
}

// NaN and -inf are below any border; a NaN exponent (of a difference beyond fp32)
// is one of nothing.
__device__ __forceinline__ float weight(const RowRule& r, float x) {
    const float d = x - r.m;
    const float y = fmaxf(fmaf(d, r.c, d * r.c_lo), -256.f);
    return x >= r.border ? ex2(y) : 0.f;
}

__device__ __forceinline__ float2 weight2(const RowRule& r, float2 x) {
    const float2 d = add2(x, make_float2(-r.m, -r.m));
    const float2 y = fma2(d, make_float2(r.c, r.c), mul2(d, make_float2(r.c_lo, r.c_lo)));
    return make_float2(x.x >= r.border ? ex2(fmaxf(y.x, -256.f)) : 0.f, x.y >= r.border ? ex2(fmaxf(y.y, -256.f)) : 0.f);
}

__device__ __forceinline__ float row_min_p(const ProbsArgs& a, long long row) { return a.min_p ? a.min_p[row] : 0.f; }

// ---- rows held by a cluster

constexpr int CT = 512;                // threads of a CTA

template <typename T> constexpr int per_vec() { return 16 / (int)sizeof(T); }

// One exchange between the CTAs of a cluster: each sends its word to all, and waits
// for all words by an mbarrier that counts their bytes (a barrier of the cluster
// that orders memory took 3 us in its place).  A CTA's words of the next row cannot
// come before it has this row's: nobody passes the second exchange without it.
struct Trade {
    uint32_t all[16];
    uint64_t bar;
};

// What the threads at work on a row share.
struct RowShared {
    Trade max, sum;
    float warps[2][32];
    int best[2];
    unsigned stop;         // the cluster's row (by its own count) from which on this CTA works on none
    // Behind 16 more bytes a RowSetup stays at an odd multiple of 8, and its fields are loaded one
    // by one as they are needed; by fours they held registers (512 rows of 151936 bf16 logits 155 us).
    unsigned pad[3];
};

// By one thread, then the cluster's opening barrier.
__device__ __forceinline__ void open_row(RowShared& sh) {
    mbar_init(&sh.max.bar, 1);
    mbar_init(&sh.sum.bar, 1);
    fence_mbar_init();
    sh.best[0] = sh.best[1] = 0x7fffffff;
    sh.stop = 0xffffffffu;
}

// A barrier of the NT threads at work.
template <int NT> __device__ __forceinline__ void work_sync() {
    if (NT == CT) __syncthreads();
    else asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
}

// A wait that runs out (the others of a cluster did not come within two seconds) leaves a
// warp without a word; the others of its CTA may have got it.  So no warp changes its
// way: it carries NaN (a greedy row's token: -1) through the same barriers and sends it
// on, and what it writes is NaN.  A row is right, or NaN wherever it might not be.
//
// SELFTEST: the last CTA of a cluster keeps its word `a.quiet` (0: the maximum's, 1: the
// sum's) of row a.quiet_row to itself, and waits end after a.limit_ns.
constexpr unsigned long long LIMIT_NS = 2000000000ull;

template <bool SELFTEST> __device__ __forceinline__ unsigned long long limit_of(const ProbsArgs& a) {
    return SELFTEST ? a.limit_ns : LIMIT_NS;
}

// v the same in all of the CTA, the turn-th exchange by t, of the cluster's n-th row; false,
// in all of a warp: the others' words did not come.
template <bool SELFTEST>
__device__ __forceinline__ bool trade(const ProbsArgs& a, RowShared& sh, bool sum, uint32_t v, int ranks, uint32_t rank, unsigned n,
                                      unsigned turn) {
    Trade& t = sum ? sh.sum : sh.max;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&t.bar, 4 * ranks);
    const bool quiet = SELFTEST && (int)rank == ranks - 1 && sum == (a.quiet == 1) && n == (unsigned)a.quiet_row;
    if ((int)threadIdx.x < ranks && !quiet) send_word(&t.all[rank], &t.bar, threadIdx.x, v);
    const bool came = __all_sync(0xffffffffu, mbar_wait_bounded(&t.bar, turn & 1, limit_of<SELFTEST>(a)));
    if (!came) atomicMin(&sh.stop, n + 1);
    return came;
}

// At the end of a CTA one of whose waits has run out: its shared memory stays until the
// cluster's other warps have ended or wait here too, and their words are in.
template <bool SELFTEST> __device__ __noinline__ void linger(const ProbsArgs& a, RowShared& sh, unsigned turn) {
    cluster_arrive_relaxed();
    cluster_wait();
    mbar_wait_bounded(&sh.max.bar, turn & 1, limit_of<SELFTEST>(a));
    mbar_wait_bounded(&sh.sum.bar, turn & 1, limit_of<SELFTEST>(a));
}

__device__ __forceinline__ float warp_all(float v, bool sum) { return sum ? warp_sum(v) : warp_max(v); }

// The sum (or the largest) of a warp value over the CTA, the same in all of it.
// A lane takes a warp's (below, a CTA's) value and the warp joins them: every thread
// reading all of them cost as many instructions as 20 logits.
template <int NT> __device__ __forceinline__ float over_cta(float* warps, float v, bool sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) warps[warp] = v;
    work_sync<NT>();
    return warp_all(lane < NT / 32 ? warps[lane] : (sum ? 0.f : -INFINITY), sum);
}

// The same of a CTA's value over the cluster; NaN if the other CTAs' did not come.
// `first`: the opening barrier is still to be waited for.
template <bool SELFTEST>
__device__ __forceinline__ float over_cluster(const ProbsArgs& a, RowShared& sh, float v, bool sum, int ranks, uint32_t rank, unsigned n,
                                              unsigned turn, bool first) {
    if (ranks == 1) return v;
    if (first) cluster_wait();
    if (!trade<SELFTEST>(a, sh, sum, __float_as_uint(v), ranks, rank, n, turn)) return NAN;
    const int lane = threadIdx.x & 31;
    const Trade& t = sum ? sh.sum : sh.max;
    return warp_all(lane < ranks ? __uint_as_float(t.all[lane]) : (sum ? 0.f : -INFINITY), sum);
}

// Where a CTA's part of a row lies: vectors of 16 bytes that begin at 16-byte
// boundaries of the logits; the few tokens before the first and behind the last
// are one more a thread of the first CTA.
struct Part {
    int head, v0, n;          // tokens before the vectors; this CTA's n (may be negative) from the v0-th on
    int tail, tail_at;        // tokens behind the vectors, the first of them
};

// RAGGED false: rows of whole vectors.
template <typename T, bool RAGGED>
__device__ __forceinline__ Part part_of_row(const T* x, int vocab, int ranks, uint32_t rank) {
    constexpr int VE = per_vec<T>();
    const int off = RAGGED ? (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)) : 0;
    Part p;
    p.head = min(off ? VE - off : 0, vocab);
    const int vecs = (vocab - p.head) / VE, per = (vecs + ranks - 1) / ranks;
    p.v0 = (int)rank * per;
    p.n = min(per, vecs - p.v0);
    p.tail_at = p.head + vecs * VE;
    p.tail = RAGGED ? vocab - p.tail_at : 0;
    return p;
}

// The extra token of this thread; -1: none.
template <bool RAGGED>
__device__ __forceinline__ int extra_of(const Part& p, uint32_t rank) {
    const int tid = threadIdx.x;
    if (!RAGGED || rank) return -1;
    if (tid < p.head) return tid;
    return tid >= 16 && tid < 16 + p.tail ? p.tail_at + tid - 16 : -1;
}

// The vectors of a thread: at + k * step where below limit, k from 0 on.
struct Mine {
    int at, step, limit;
    __device__ __forceinline__ int operator()(int k) const { return at + k * step; }
    __device__ __forceinline__ bool has(int k) const { return at + k * step < limit; }
};

// A row's logits in registers (w: -inf where there is none) to its probabilities, by
// the NT threads at work of each of the cluster's CTAs; the cluster's n-th row, and the
// turn-th that it works on.  greedy: T is 0.  False, in all of the CTA: it has stopped
// before this row.
template <typename T, int K, int NT, bool SELFTEST>
__device__ __forceinline__ bool finish_row(const ProbsArgs& a, const Part& part, const Mine& mine, float (&w)[K * per_vec<T>()],
                                           float& extra, int e, bool greedy, const RowSetup& setup, RowShared& sh, int ranks,
                                           uint32_t rank, unsigned n, unsigned turn, bool first) {
    constexpr int VE = per_vec<T>();
    const int tid = threadIdx.x;
    float m = no_nan(extra);                       // fmaxf leaves NaN out
#pragma unroll
    for (int i = 0; i < K * VE; ++i) m = fmaxf(m, w[i]);
    m = over_cta<NT>(sh.warps[0], warp_max(m), false);
    if (NT != CT && sh.stop <= n) return false;
    m = over_cluster<SELFTEST>(a, sh, m, false, ranks, rank, n, turn, first);
    if (tid == 0) sh.best[(turn & 1) ^ 1] = 0x7fffffff;      // the next row's: the last one's has been read
    if (greedy) {
        int best = m == m ? 0x7fffffff : -1;
        if (m > -INFINITY) {
#pragma unroll
            for (int k = K - 1; k >= 0; --k)
#pragma unroll
                for (int i = VE - 1; i >= 0; --i)
                    if (w[k * VE + i] == m) best = part.head + (part.v0 + mine(k)) * VE + i;
            if (extra == m) best = min(best, e);
        }
        best = __reduce_min_sync(0xffffffffu, best);
        if ((tid & 31) == 0) atomicMin(&sh.best[turn & 1], best);
        work_sync<NT>();
        best = sh.best[turn & 1];
        if (ranks > 1) {
            const bool came = trade<SELFTEST>(a, sh, true, (uint32_t)best, ranks, rank, n, turn);
            for (int i = 0; i < ranks; ++i) best = came ? min(best, (int)sh.sum.all[i]) : -1;
        }
        const float other = best < 0 ? NAN : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i) w[k * VE + i] = part.head + (part.v0 + mine(k)) * VE + i == best ? 1.f : other;
        extra = best >= 0 && e == best ? 1.f : other;
    } else {
        float sum;
        if (m != INFINITY) {                       // (-inf: no logit above it, all weights are 0)
            const RowRule r = rule_of(m, setup);
            extra = weight(r, extra);
            float2 sums = make_float2(extra, m == m ? 0.f : NAN);
#pragma unroll
            for (int i = 0; i < K * VE; i += 2) {
                const float2 y = weight2(r, make_float2(w[i], w[i + 1]));
                w[i] = y.x, w[i + 1] = y.y;
                sums = add2(sums, y);
            }
            sum = sums.x + sums.y;
        } else {
            sum = extra = extra == INFINITY ? 1.f : 0.f;
#pragma unroll
            for (int i = 0; i < K * VE; ++i) {
                w[i] = w[i] == INFINITY ? 1.f : 0.f;
                sum += w[i];
            }
        }
        sum = over_cluster<SELFTEST>(a, sh, over_cta<NT>(sh.warps[1], warp_sum(sum), true), true, ranks, rank, n, turn, false);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        extra *= inv;
#pragma unroll
        for (int i = 0; i < K * VE; i += 2) {
            const float2 y = mul2(make_float2(w[i], w[i + 1]), make_float2(inv, inv));
            w[i] = y.x, w[i + 1] = y.y;
        }
    }
    return true;
}

// They to memory.
template <typename T, int K>
__device__ __forceinline__ void store_row(float* p, const Part& part, const Mine& mine, const float (&w)[K * per_vec<T>()], float extra, int e) {
    constexpr int VE = per_vec<T>();
    if (e >= 0) p[e] = extra;
    float* pv = p + part.head + (long long)part.v0 * VE;
    if ((reinterpret_cast<uintptr_t>(pv) & 15) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (mine.has(k))
#pragma unroll
                for (int i = 0; i < VE; i += 4)
                    reinterpret_cast<float4*>(pv)[mine(k) * (VE / 4) + i / 4] =
                        make_float4(w[k * VE + i], w[k * VE + i + 1], w[k * VE + i + 2], w[k * VE + i + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (mine.has(k))
#pragma unroll
                for (int i = 0; i < VE; ++i) pv[mine(k) * VE + i] = w[k * VE + i];
    }
}

// K vectors of a thread to numbers.
template <typename T, int K>
__device__ __forceinline__ void to_numbers(const uint4 (&raw)[K], const Mine& mine, float (&w)[K * per_vec<T>()]) {
    constexpr int VE = per_vec<T>();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const T* r = reinterpret_cast<const T*>(&raw[k]);
#pragma unroll
        for (int i = 0; i < VE; ++i) w[k * VE + i] = mine.has(k) ? to_f32(r[i]) : -INFINITY;
    }
}

// A cluster a row.
template <typename T, int K, bool SELFTEST = false>
__global__ void __launch_bounds__(CT, K * per_vec<T>() > 12 ? 2 : 3)
probs_cluster_kernel(const __grid_constant__ ProbsArgs a, int ranks) {
    __shared__ RowShared sh;
    __shared__ RowSetup s_setup;
    pdl_trigger();
    const int tid = threadIdx.x;
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    const long long row = blockIdx.x / (unsigned)ranks;
    if (tid == 0) open_row(sh);
    if (ranks > 1) cluster_arrive_relaxed();
    pdl_wait();
    const float t = a.temperature[row];
    const bool fine = has_temperature(t);          // else the row is left as it was, by all of the cluster
    if (!fine) {
        if (ranks > 1) cluster_wait();
        return;
    }
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_row;
    const Part part = part_of_row<T, true>(x, a.vocab, ranks, rank);
    const Mine mine{tid, CT, part.n};
    const uint4* xv = reinterpret_cast<const uint4*>(x + part.head) + part.v0;
    float w[K * per_vec<T>()], extra = -INFINITY;
    const int e = extra_of<true>(part, rank);
    uint4 raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (mine.has(k)) raw[k] = xv[mine(k)];
    if (e >= 0) extra = to_f32(x[e]);
    if (tid == CT - 1) s_setup = setup_of(t, row_min_p(a, row));      // while they are on their way
    to_numbers<T, K>(raw, mine, w);
    finish_row<T, K, CT, SELFTEST>(a, part, mine, w, extra, e, t == 0.f, s_setup, sh, ranks, rank, 0, 0, true);
    store_row<T, K>(a.p + row * a.p_row, part, mine, w, extra, e);
    if (sh.stop != 0xffffffffu) linger<SELFTEST>(a, sh, 0);
}

__device__ __forceinline__ void bulk_store_1d(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;"
                 ::"l"((uint64_t)dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
template <int N> __device__ __forceinline__ void bulk_store_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Clusters that stay: threads of a CTA, CTAs an SM, threads at work on a row; vectors of a
// lane in a piece of its warp's outputs, and the places for pieces.
// Of 16-bit logits the next row takes half as much shared memory as its outputs would: two
// CTAs fit an SM, one works while the other waits for its cluster, and outputs leave by
// 1 KB pieces (512 rows of 151936: 135 us; by one CTA of 1024 threads an SM 150), though a
// thread's 40 weights do not all fit its 64 registers (it spills 108 bytes a row).  fp32
// rows have one CTA and a place for all of a warp's outputs (137 us; in 1 KB pieces 153; two
// CTAs in clusters of 16 150; two without a place for the next row 187).
template <typename T> struct Stream {
    static constexpr bool wide = sizeof(T) == 4;
    static constexpr int threads = wide ? 1024 : 512, per_sm = wide ? 1 : 2, work = threads - 32;
    static constexpr int most = 5;         // vectors of a thread
    static constexpr int piece = wide ? most : 1, places = wide ? 1 : 2;
    // of parts of cap vectors
    static size_t smem(int cap) {
        return (size_t)2 * cap * 16 + (wide ? (size_t)cap * 16 : (size_t)work * places * piece * per_vec<T>() * 4);
    }
};

// Clusters that take every gridDim.x / ranks-th row.  The last warp brings a CTA's part of
// the next row to shared memory while one is worked on, and the rows' setups.  A warp's
// vectors lie in a row, k_row a lane, so that its outputs leave by bulk copies of its own
// (stores of the threads held up what they read behind them: 512 rows of 151936 fp32
// logits 177 us).  Rows of whole vectors, 16-byte aligned in the output.
// Once a wait has run out the CTA works on no further row: its part of them becomes NaN,
// and the others of the cluster wait for its words in vain and do the same.
template <typename T, bool SELFTEST = false>
__global__ void __launch_bounds__(Stream<T>::threads, Stream<T>::per_sm)
probs_stream_kernel(const __grid_constant__ ProbsArgs a, int ranks, int cap, int k_row) {
    using S_ = Stream<T>;
    constexpr int NT = S_::work, K = S_::most, VE = per_vec<T>(), P = S_::piece;
    extern __shared__ uint4 in[];                  // [2][cap], cap the vectors of a part; then the pieces
    __shared__ RowShared sh;
    __shared__ RowSetup s_setup[3];                // a row's stays until that of the third one behind it comes
    __shared__ float s_t[3];
    __shared__ uint64_t full[2], empty[2];
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    const int first_row = blockIdx.x / (unsigned)ranks, step = gridDim.x / (unsigned)ranks;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, NT / 32);
        }
        open_row(sh);
    }
    __syncthreads();
    if (ranks > 1) {
        cluster_arrive_relaxed();
        cluster_wait();
    }
    pdl_wait();
    const T* x0 = reinterpret_cast<const T*>(a.x);
    if (tid >= NT) {
        if (lane == 0) {
            unsigned n = 0;
            for (long long row = first_row; row < a.rows; row += step, ++n) {
                const float t = a.temperature[row];
                const RowSetup setup = setup_of(t, row_min_p(a, row));
                const T* x = x0 + row * a.x_row;
                const Part part = part_of_row<T, false>(x, a.vocab, ranks, rank);
                const int b = n & 1;
                if (n >= 2 && !mbar_wait_bounded(empty + b, (n / 2 - 1) & 1, limit_of<SELFTEST>(a))) break;
                s_t[n % 3] = t;
                s_setup[n % 3] = setup;
                if (part.n > 0 && has_temperature(t)) {
                    mbar_arrive_expect_tx(full + b, part.n * 16);
                    bulk_load_1d(in + b * cap, reinterpret_cast<const uint4*>(x + part.head) + part.v0, part.n * 16, full + b);
                } else {
                    mbar_arrive(full + b);
                }
            }
            // no copy is in flight when this warp ends
            for (unsigned i = n < 2 ? 0 : n - 2; i < n; ++i) mbar_wait_bounded(full + (i & 1), (i / 2) & 1, limit_of<SELFTEST>(a));
        }
        __syncwarp();
        return;
    }
    uint4* const pieces = in + 2 * cap + warp * (S_::wide ? k_row * 32 : S_::places * P * 32 * VE / 4);
    unsigned n = 0, turn = 0, at_piece = 0;
    long long row = first_row;
    for (; row < a.rows; row += step, ++n) {
        const Part part = part_of_row<T, false>(x0, a.vocab, ranks, rank);
        const Mine mine{warp * k_row * 32 + lane, 32, min(part.n, (warp + 1) * k_row * 32)};
        const int b = n & 1;
        float extra = -INFINITY;
        const bool came = __all_sync(0xffffffffu, mbar_wait_bounded(full + b, (n / 2) & 1, limit_of<SELFTEST>(a)));
        if (!came) {
            // the others of the CTA may have it: they stop behind their next barrier
            atomicMin(&sh.stop, n);
            while (row < a.rows && !has_temperature(a.temperature[row])) row += step;
            if (row < a.rows) work_sync<NT>();
            break;
        }
        const float& t = s_t[n % 3];
        const bool fine = has_temperature(t);            // else the row is left as it was, by all of the cluster
        uint4 raw[K];
        if (fine)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (mine.has(k)) raw[k] = in[b * cap + mine(k)];
        float w[K * VE];
        to_numbers<T, K>(raw, fine ? mine : Mine{0, 0, 0}, w);
        // what was read is in registers before its place goes back (a fence would wait
        // for stores as well)
#pragma unroll
        for (int i = 0; i < K * VE; ++i) asm volatile("" ::"f"(w[i]) : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + b);
        if (!fine) continue;
        if (!finish_row<T, K, NT, SELFTEST>(a, part, mine, w, extra, -1, t == 0.f, s_setup[n % 3], sh, ranks, rank, n, turn, false)) break;
        ++turn;
        float* const warp_p = a.p + row * a.p_row + ((long long)part.v0 + warp * k_row * 32) * VE;
#pragma unroll
        for (int k0 = 0; k0 < K; k0 += P) {
            const int left = mine.limit - warp * k_row * 32 - k0 * 32;      // of the warp's vectors
            if (left <= 0) break;
            float4* out = reinterpret_cast<float4*>(pieces + (S_::wide ? 0 : at_piece++ % S_::places * (P * 32 * VE / 4)));
            if (lane == 0) bulk_store_read<S_::places - 1>();               // the place's last piece has left it
            __syncwarp();
#pragma unroll
            for (int k = 0; k < P; ++k)
                if (!S_::wide || mine.has(k0 + k))
#pragma unroll
                    for (int i = 0; i < VE; i += 4) {
                        const float* v = w + (k0 + k) * VE + i;
                        out[(k * 32 + lane) * (VE / 4) + i / 4] = make_float4(v[0], v[1], v[2], v[3]);
                    }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) bulk_store_1d(warp_p + k0 * 32 * VE, out, min(left, P * 32) * VE * 4);
        }
    }
    if (lane == 0) bulk_store_done();
    for (; row < a.rows; row += step) {                  // of a CTA that has stopped
        if (!has_temperature(a.temperature[row])) continue;
        const Part part = part_of_row<T, false>(x0, a.vocab, ranks, rank);
        float* const p = a.p + row * a.p_row + (long long)part.v0 * VE;
        for (int i = warp * k_row * 32 * VE + lane; i < min(part.n, (warp + 1) * k_row * 32) * VE; i += 32) p[i] = NAN;
    }
    if (ranks > 1 && sh.stop != 0xffffffffu) linger<SELFTEST>(a, sh, turn);
}

// ---- rows of any length

constexpr int PT = 1024;

// A thread sums TERMS weights in fp32, and those sums in 64 bits: in one fp32 number the
// terms of 2^24 logits, 16384 a thread, came out by 10^-4 wrong where they are alike.
constexpr int TERMS = 32;

template <typename T>
__global__ void __launch_bounds__(PT) probs_rows_kernel(const __grid_constant__ ProbsArgs a) {
    __shared__ double red[32];
    __shared__ unsigned long long red_key;
    __shared__ RowSetup s_setup;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const float t = a.temperature[row];
    if (!has_temperature(t)) return;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_row;
    float* p = a.p + row * a.p_row;
    if (tid == 0) {
        red_key = 0;
        s_setup = setup_of(t, row_min_p(a, row));
    }
    __syncthreads();
    unsigned long long key = 0;
    for (int i = tid; i < a.vocab; i += PT) {
        const unsigned long long k = argmax_key(no_nan(to_f32(x[i])) + 0.f, i);
        key = k > key ? k : key;
    }
    atomicMax(&red_key, key);
    __syncthreads();
    const int best = argmax_key_index(red_key);
    const float m = no_nan(to_f32(x[best]));
    __syncthreads();
    if (m == -INFINITY || t == 0.f) {
        for (int i = tid; i < a.vocab; i += PT) p[i] = i == best && m != -INFINITY ? 1.f : 0.f;
        return;
    }
    const RowRule r = rule_of(m, s_setup);
    auto weigh = [&](float v) { return m < INFINITY ? weight(r, v) : (v == INFINITY ? 1.f : 0.f); };
    double sum = 0.0;
    for (int i0 = tid; i0 < a.vocab; i0 += TERMS * PT) {
        const int end = min(i0 + TERMS * PT, a.vocab);
        float part = 0.f;
        for (int i = i0; i < end; i += PT) part += weigh(to_f32(x[i]));
        sum += part;
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = red[lane];
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = (float)(1.0 / sum);
    for (int i = tid; i < a.vocab; i += PT) p[i] = weigh(to_f32(x[i])) * inv;
}

// Clusters of 16 are allowed once per kernel and device.
cudaError_t allow_cluster(const void* kern) {
    static std::mutex mu;
    constexpr int MAX = 256;
    static const void* kerns[MAX];
    static int devs[MAX], n = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n; ++i)
        if (kerns[i] == kern && devs[i] == dev) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && n < MAX) {
        kerns[n] = kern;
        devs[n++] = dev;
    }
    return e;
}

// Clusters of a kernel that run at once on the current device, asked for once (how long
// the rows are, and so how much shared memory a CTA takes, does not change how many fit).
cudaError_t clusters_at_once(const void* kern, int ranks, int threads, size_t smem, int* most) {
    static std::mutex mu;
    constexpr int MAX = 256;
    struct Known {
        const void* kern;
        int dev, ranks, most;
    };
    static Known known[MAX];
    static int n = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n; ++i)
        if (known[i].kern == kern && known[i].dev == dev && known[i].ranks == ranks) {
            *most = known[i].most;
            return cudaSuccess;
        }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ranks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(most, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (*most < 1) *most = 1;
    if (n < MAX) known[n++] = Known{kern, dev, ranks, *most};
    return cudaSuccess;
}

template <typename T, int K>
int launch_cluster(const ProbsArgs& a, int ranks, cudaStream_t s) {
    const void* kern = reinterpret_cast<const void*>(probs_cluster_kernel<T, K>);
    if (ranks > 8) {
        const cudaError_t e = allow_cluster(kern);
        if (e != cudaSuccess) return (int)e;
    }
    return (int)launch_cluster_k(probs_cluster_kernel<T, K>, dim3((unsigned)(a.rows * ranks)), dim3(CT), ranks, s, 0, a, ranks);
}

template <typename T>
int launch_stream(const ProbsArgs& a, int ranks, int cap, cudaStream_t s) {
    const void* kern = reinterpret_cast<const void*>(probs_stream_kernel<T>);
    const size_t smem = Stream<T>::smem(cap);
    int most = 0;
    cudaError_t e = allow_smem(kern);
    if (e == cudaSuccess && ranks > 8) e = allow_cluster(kern);
    if (e == cudaSuccess) e = clusters_at_once(kern, ranks, Stream<T>::threads, smem, &most);
    if (e != cudaSuccess) return (int)e;
    // the rounds that the clusters need, and no more clusters than fill them
    const int rounds = (a.rows + most - 1) / most, clusters = (a.rows + rounds - 1) / rounds;
    return (int)launch_cluster_k(probs_stream_kernel<T>, dim3((unsigned)(clusters * ranks)), dim3(Stream<T>::threads), ranks, s, smem,
                                 a, ranks, cap, (cap + Stream<T>::work - 1) / Stream<T>::work);
}

template <typename T>
int launch_t(const ProbsArgs& a, int sms, cudaStream_t s) {
    constexpr int VE = per_vec<T>(), MOST = 40 / VE;      // vectors of a thread
    const long long vecs = ((long long)a.vocab + VE - 1) / VE;
    auto of_thread = [&](int ranks, int threads) { return (int)(((vecs + ranks - 1) / ranks + threads - 1) / threads); };
    int ranks = 1;
    while (ranks < 16 && of_thread(ranks, CT) > MOST) ranks *= 2;
    const bool held = of_thread(ranks, CT) <= MOST;
    if (!held || (long long)a.rows * ranks > 0x7fffffffll)
        return (int)launch_k(probs_rows_kernel<T>, dim3((unsigned)a.rows), dim3(PT), 0, s, a);
    // Clusters that stay where rows are more than twice what run at once by a cluster a row, and
    // the registers mostly filled, or the clusters of 16 CTAs (in us, by them and by a cluster a
    // row: 151936 logits, fp32 320 rows 89, 101; 160 rows 48, 53; 80 rows 29.6, 29.5; bf16 320
    // rows 91, 102; 100 rows 33, 36; of 262144 logits, in clusters of 16, fp32 320 rows 171, 203;
    // bf16 320 rows of 100000 73, 80; where they fill less, fp32 320 rows of 100000 80, 74, bf16 of
    // 48000 39, 36; of fewer rows, bf16 160 rows of 64000, 640 CTAs, 27.5, 26.1).  Rows that are
    // not of whole aligned vectors would have to be stored by their threads: bf16 512 rows of
    // 32003 41, 36; 320 of 151935 112, 103; fp32 99, 102.
    const int cap = (int)((vecs + ranks - 1) / ranks), k_stream = of_thread(ranks, Stream<T>::work);
    const bool whole = a.vocab % VE == 0 && !(reinterpret_cast<uintptr_t>(a.x) & 15) && a.x_row % VE == 0 &&
                       !(reinterpret_cast<uintptr_t>(a.p) & 15) && a.p_row % 4 == 0;
    const bool filled = VE == 4 ? 4 * cap >= 3 * Stream<T>::most * Stream<T>::work : 8 * cap > 5 * Stream<T>::most * Stream<T>::work;
    const bool many = (long long)a.rows * ranks > (VE == 4 || ranks > 8 ? 4 : 5) * sms;
    if (whole && many && (filled || ranks > 8) && k_stream <= Stream<T>::most &&
        Stream<T>::smem(cap) <= 226 * 1024 / Stream<T>::per_sm)
        return launch_stream<T>(a, ranks, cap, s);
    // few rows: more CTAs each, up to two an SM (50 rows of 32003 bf16 logits 8.3 -> 7.2 us;
    // three: 77 rows 9.7 -> 10.7)
    while (ranks < 8 && (long long)a.rows * ranks * 2 <= 2 * sms && of_thread(ranks, CT) > 1) ranks *= 2;
    const int k = of_thread(ranks, CT);
    if (k <= 1) return launch_cluster<T, 1>(a, ranks, s);
    if (k <= 2) return launch_cluster<T, 2>(a, ranks, s);
    if (k <= 3) return launch_cluster<T, 3>(a, ranks, s);
    if (k <= 5) return launch_cluster<T, 5>(a, ranks, s);
    if (VE == 4 && k <= 7) return launch_cluster<T, VE == 4 ? 7 : 5>(a, ranks, s);
    return launch_cluster<T, MOST>(a, ranks, s);
}

}  // namespace

int launch_probs_selftest(const ProbsArgs& a, bool stays, cudaStream_t s) {
    constexpr int ranks = 2;
    if (!stays)
        return (int)launch_cluster_k(probs_cluster_kernel<float, 1, true>, dim3((unsigned)(a.rows * ranks)), dim3(CT), ranks, s, 0, a, ranks);
    using S_ = Stream<float>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(probs_stream_kernel<float, true>));
    const int cap = (a.vocab / 4 + ranks - 1) / ranks;
    return (int)(e == cudaSuccess ? launch_cluster_k(probs_stream_kernel<float, true>, dim3(ranks), dim3(S_::threads), ranks, s,
                                                     S_::smem(cap), a, ranks, cap, (cap + S_::work - 1) / S_::work)
                                  : e);
}

int launch_probs(const ProbsArgs& a, int sms, cudaStream_t s) {
    if (a.dtype == 0) return launch_t<float>(a, sms, s);
    if (a.dtype == 1) return launch_t<__nv_bfloat16>(a, sms, s);
    return launch_t<__half>(a, sms, s);
}

}  // namespace dfl
