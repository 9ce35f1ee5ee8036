// Probabilities of rows of logits.
//
//   p_v = w_v / sum w,  w_v = exp((x_v - m) / T) where x_v >= m + T ln(min_p), else 0
// with m the row's maximum; T = 0: 1 at the first maximum.  NaN logits count as
// -inf; where the maximum is +inf its holders share the row.
//
// The border m + T ln(min_p) is taken as a pair of fp32 numbers (48 bits) and
// rounded up to the next fp32 value, so that comparing fp32 logits with it is exact.  log2(e) / T is
// held as two fp32 numbers, so that a weight's exponent is off by the
// difference's and the product's rounding alone; weights, sums and quotients are
// fp32.
//
// A row's maximum is needed before its sum and its sum before its first output:
// the row stays on the SMs between.  A cluster of up to 16 CTAs holds it in
// registers (up to 40 logits a thread, 512 threads a CTA), trades maxima and sums
// through distributed shared memory, and writes what it read once.  Larger rows
// (above 327680 logits) are read three times, by one CTA.

#include <mutex>

#include "cluster_dev.cuh"
#include "gemm.cuh"
#include "sampling.cuh"

namespace dfl {
namespace {

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float no_nan(float x) { return x == x ? x : -INFINITY; }

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

__device__ __forceinline__ float row_min_p(const ProbsArgs& a, long long row) { return a.min_p ? a.min_p[row] : 0.f; }

// ---- rows held by a cluster

constexpr int CT = 512, CW = CT / 32;

template <typename T> constexpr int per_vec() { return 16 / (int)sizeof(T); }

// One exchange between the CTAs of a cluster: each sends its word to all, and waits
// for all words by an mbarrier that counts their bytes (a barrier of the cluster
// that orders memory took 3 us in its place).
struct Trade {
    uint32_t all[16];
    uint64_t bar;
};

// By one thread, then the cluster's opening barrier.
__device__ __forceinline__ void open_trade(Trade& t, int ranks) {
    mbar_init(&t.bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&t.bar, 4 * ranks);
}

// By all threads, v the same in all of the CTA; false: the others' did not come.
__device__ __forceinline__ bool trade(Trade& t, uint32_t v, int ranks, uint32_t rank) {
    if ((int)threadIdx.x < ranks) send_word(&t.all[rank], &t.bar, threadIdx.x, v);
    return mbar_wait_bounded(&t.bar, 0);
}

// The largest / the sum of a warp value over the cluster, the same everywhere; NaN
// if the other CTAs' did not come.  `first`: the opening barrier is still to be waited for.
template <typename F>
__device__ __forceinline__ float over_cluster(Trade& t, float* warps, float v, int ranks, uint32_t rank, bool first, F op) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) warps[warp] = v;
    __syncthreads();
    float r = warps[0];
#pragma unroll
    for (int i = 1; i < CW; ++i) r = op(r, warps[i]);
    if (ranks == 1) return r;
    if (first) cluster_wait();
    if (!trade(t, __float_as_uint(r), ranks, rank)) return __int_as_float(0x7fffffff);
    r = __uint_as_float(t.all[0]);
    for (int i = 1; i < ranks; ++i) r = op(r, __uint_as_float(t.all[i]));
    return r;
}

// K vectors of 16 bytes a thread.  The vectors begin at 16-byte boundaries of the
// logits; the few before the first and behind the last are one more a thread.
template <typename T, int K>
__global__ void __launch_bounds__(CT, K * per_vec<T>() > 12 ? 2 : 3)
probs_cluster_kernel(const __grid_constant__ ProbsArgs a, int ranks) {
    constexpr int VE = per_vec<T>();
    __shared__ Trade s_max, s_sum;
    __shared__ float s_warps[2][CW];
    __shared__ RowSetup s_setup;
    __shared__ int s_best;
    pdl_trigger();
    const int tid = threadIdx.x;
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    const long long row = blockIdx.x / (unsigned)ranks;
    pdl_wait();
    const float t = a.temperature[row];
    if (!(t >= 0.f) || t == INFINITY) return;      // such a row is left as it was, by all of the cluster
    if (ranks > 1) {
        if (tid == 0) {
            open_trade(s_max, ranks);
            open_trade(s_sum, ranks);
        }
        cluster_arrive_relaxed();
    }
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_row;
    float* p = a.p + row * a.p_row;
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int head = min(off ? VE - off : 0, a.vocab);
    const int vecs = (a.vocab - head) / VE, per = (vecs + ranks - 1) / ranks;
    const int v0 = (int)rank * per, n = min(per, vecs - v0);      // this CTA's vectors (n may be negative)
    const T* xv = x + head + (long long)v0 * VE;
    float w[K * VE], extra = -INFINITY;
    int e = -1;                                                   // the extra one's index
    {
        uint4 raw[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = k * CT + tid;
            if (v < n) raw[k] = reinterpret_cast<const uint4*>(xv)[v];
        }
        if (rank == 0) {
            const int tail = a.vocab - head - vecs * VE;
            if (tid < head) e = tid;
            else if (tid >= 16 && tid < 16 + tail) e = a.vocab - tail + tid - 16;
            if (e >= 0) extra = to_f32(x[e]);
        }
        if (tid == CT - 1) {      // while they are on their way
            s_setup = setup_of(t, row_min_p(a, row));
            s_best = 0x7fffffff;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const T* r = reinterpret_cast<const T*>(&raw[k]);
#pragma unroll
            for (int i = 0; i < VE; ++i) w[k * VE + i] = k * CT + tid < n ? to_f32(r[i]) : -INFINITY;
        }
    }
    float m = no_nan(extra);                       // fmaxf leaves NaN out
#pragma unroll
    for (int i = 0; i < K * VE; ++i) m = fmaxf(m, w[i]);
    m = over_cluster(s_max, s_warps[0], warp_max(m), ranks, rank, true, [](float x, float y) { return fmaxf(x, y); });
    if (t == 0.f || m == -INFINITY) {     // (a NaN m, of a wait that ran out, makes the row NaN)
        int best = 0x7fffffff;
        if (m != -INFINITY) {
#pragma unroll
            for (int k = K - 1; k >= 0; --k)
#pragma unroll
                for (int i = VE - 1; i >= 0; --i)
                    if (w[k * VE + i] == m) best = head + (v0 + k * CT + tid) * VE + i;
            if (extra == m) best = min(best, e);
        }
        best = (int)__reduce_min_sync(0xffffffffu, (unsigned)best);
        if ((tid & 31) == 0) atomicMin(&s_best, best);
        __syncthreads();
        best = s_best;
        if (ranks > 1 && trade(s_sum, (uint32_t)best, ranks, rank))
            for (int i = 0; i < ranks; ++i) best = min(best, (int)s_sum.all[i]);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i) w[k * VE + i] = head + (v0 + k * CT + tid) * VE + i == best ? 1.f : 0.f;
        extra = e == best ? 1.f : 0.f;
    } else {
        float sum;
        if (m < INFINITY) {
            const RowRule r = rule_of(m, s_setup);
            sum = extra = weight(r, extra);
#pragma unroll
            for (int i = 0; i < K * VE; ++i) {
                w[i] = weight(r, w[i]);
                sum += w[i];
            }
        } else {
            sum = extra = extra == INFINITY ? 1.f : 0.f;
#pragma unroll
            for (int i = 0; i < K * VE; ++i) {
                w[i] = w[i] == INFINITY ? 1.f : 0.f;
                sum += w[i];
            }
        }
        sum = over_cluster(s_sum, s_warps[1], warp_sum(sum), ranks, rank, false, [](float x, float y) { return x + y; });
        const float inv = 1.f / sum;
        extra *= inv;
#pragma unroll
        for (int i = 0; i < K * VE; ++i) w[i] *= inv;
    }
    if (e >= 0) p[e] = extra;
    float* pv = p + head + (long long)v0 * VE;
    if ((reinterpret_cast<uintptr_t>(pv) & 15) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * CT + tid < n)
#pragma unroll
                for (int i = 0; i < VE; i += 4)
                    reinterpret_cast<float4*>(pv)[(k * CT + tid) * (VE / 4) + i / 4] =
                        make_float4(w[k * VE + i], w[k * VE + i + 1], w[k * VE + i + 2], w[k * VE + i + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * CT + tid < n)
#pragma unroll
                for (int i = 0; i < VE; ++i) pv[(k * CT + tid) * VE + i] = w[k * VE + i];
    }
}

// ---- rows of any length

constexpr int PT = 1024;

template <typename T>
__global__ void __launch_bounds__(PT) probs_rows_kernel(const __grid_constant__ ProbsArgs a) {
    __shared__ float red[32];
    __shared__ unsigned long long red_key;
    __shared__ RowSetup s_setup;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const float t = a.temperature[row];
    if (!(t >= 0.f) || t == INFINITY) return;
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
    float sum = 0.f;
    for (int i = tid; i < a.vocab; i += PT) sum += weigh(to_f32(x[i]));
    sum = warp_sum(sum);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = warp_sum(red[lane]);
    const float inv = 1.f / sum;
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

template <typename T, int K>
int launch_cluster(const ProbsArgs& a, int ranks, cudaStream_t s) {
    const void* kern = reinterpret_cast<const void*>(probs_cluster_kernel<T, K>);
    if (ranks > 8) {
        const cudaError_t e = allow_cluster(kern);
        if (e != cudaSuccess) return (int)e;
    }
    return (int)launch_cluster_k(probs_cluster_kernel<T, K>, dim3((unsigned)((long long)a.rows * ranks)), dim3(CT), ranks, s,
                                 0, a, ranks);
}

template <typename T>
int launch_t(const ProbsArgs& a, int sms, cudaStream_t s) {
    constexpr int VE = per_vec<T>(), MOST = 40 / VE;      // vectors of a thread
    const long long vecs = ((long long)a.vocab + VE - 1) / VE + 1;      // and one for a row that begins between two
    int ranks = 1;
    while (ranks < 16 && (vecs + ranks - 1) / ranks > CT * MOST) ranks *= 2;
    const long long left = (vecs + ranks - 1) / ranks;
    if (left > CT * MOST || (long long)a.rows * ranks > 0x7fffffffll)
        return (int)launch_k(probs_rows_kernel<T>, dim3((unsigned)a.rows), dim3(PT), 0, s, a);
    // few rows: more CTAs each, while all are resident at once
    while (ranks < 8 && (long long)a.rows * ranks * 2 <= sms && (vecs + ranks - 1) / ranks > CT) ranks *= 2;
    const int k = (int)(((vecs + ranks - 1) / ranks + CT - 1) / CT);
    if (k <= 1) return launch_cluster<T, 1>(a, ranks, s);
    if (k <= 2) return launch_cluster<T, 2>(a, ranks, s);
    if (k <= 3) return launch_cluster<T, 3>(a, ranks, s);
    if (k <= 5) return launch_cluster<T, 5>(a, ranks, s);
    if (VE == 4 && k <= 7) return launch_cluster<T, VE == 4 ? 7 : 5>(a, ranks, s);
    return launch_cluster<T, MOST>(a, ranks, s);
}

}  // namespace

int launch_probs(const ProbsArgs& a, int sms, cudaStream_t s) {
    if (a.dtype == 0) return launch_t<float>(a, sms, s);
    if (a.dtype == 1) return launch_t<__nv_bfloat16>(a, sms, s);
    return launch_t<__half>(a, sms, s);
}

}  // namespace dfl
