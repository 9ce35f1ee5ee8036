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

// What a row's temperature and min_p come to, by one thread: fp64 is slow here.
struct RowSetup {
    float c, c_lo;        // log2(e) / T
    float cut, cut_lo;    // T ln(min_p)
};

__device__ __forceinline__ RowSetup setup_of(float t, float min_p) {
    RowSetup r;
    const double c = fmin(1.4426950408889634 / (double)t, 1e38);    // no 0 * inf at the smallest T
    r.c = (float)c;
    r.c_lo = (float)(c - (double)r.c);
    const double cut = min_p > 0.f ? (double)t * log((double)fminf(min_p, 1.f)) : -INFINITY;
    r.cut = (float)cut;
    r.cut_lo = isinf(r.cut) ? 0.f : (float)(cut - (double)r.cut);
    return r;
}

struct RowRule {
    float m, border;      // maximum, smallest logit that counts
    float c, c_lo;
};

__device__ __forceinline__ RowRule rule_of(float m, const RowSetup& u) {
    RowRule r{m, -INFINITY, u.c, u.c_lo};
    // m + cut as s + e, exactly, then rounded up
    const float s = __fadd_rn(m, u.cut), b = __fsub_rn(s, m);
    const float e = __fadd_rn(__fsub_rn(m, __fsub_rn(s, b)), __fsub_rn(u.cut, b));
    if (fabsf(s) < INFINITY) r.border = __fadd_ru(s, __fadd_rn(e, u.cut_lo));
    return r;
}

__device__ __forceinline__ float weight(const RowRule& r, float x) {
    const float d = x == r.m ? 0.f : x - r.m;      // inf - inf
    // -inf * c_lo may be inf: the sum's NaN is a weight of nothing
    const float y = fmaxf(fmaf(d, r.c, d * r.c_lo), -256.f);
    return x >= r.border && x > -INFINITY ? ex2(y) : 0.f;
}

__device__ __forceinline__ float row_min_p(const ProbsArgs& a, long long row) { return a.min_p ? a.min_p[row] : 0.f; }

// ---- rows held by a cluster

constexpr int CT = 512, CW = CT / 32;

template <typename T> constexpr int per_vec() { return 16 / (int)sizeof(T); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// A word of another CTA's shared memory, at the place of this CTA's p.
__device__ __forceinline__ void put_remote(void* p, uint32_t rank, uint32_t v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

struct Trade {
    uint32_t warp[CW];
    uint32_t all[16];
};

// The largest / the sum of a warp value over the cluster, the same everywhere.
// `first`: the cluster's opening barrier is still to be waited for.
template <typename F>
__device__ __forceinline__ float trade(Trade& t, float v, int ranks, uint32_t rank, bool first, F op) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) t.warp[warp] = __float_as_uint(v);
    __syncthreads();
    if (first && ranks > 1) cluster_wait();
    float r = __uint_as_float(t.warp[0]);
#pragma unroll
    for (int i = 1; i < CW; ++i) r = op(r, __uint_as_float(t.warp[i]));
    if (ranks == 1) return r;
    if ((int)threadIdx.x < ranks) put_remote(&t.all[rank], threadIdx.x, __float_as_uint(r));
    cluster_arrive();
    cluster_wait();
    r = __uint_as_float(t.all[0]);
    for (int i = 1; i < ranks; ++i) r = op(r, __uint_as_float(t.all[i]));
    return r;
}

// K vectors of 16 bytes a thread.  WIDE: full vectors of probabilities are
// 16-byte aligned where the logits' are.
template <typename T, int K>
__global__ void __launch_bounds__(CT, K * per_vec<T>() > 12 ? 2 : 3)
probs_cluster_kernel(const __grid_constant__ ProbsArgs a, int ranks) {
    constexpr int VE = per_vec<T>();
    __shared__ Trade s_max, s_sum;
    __shared__ RowSetup s_setup;
    __shared__ int s_best;
    pdl_trigger();
    const int tid = threadIdx.x;
    const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
    const long long row = blockIdx.x / (unsigned)ranks;
    pdl_wait();
    const float t = a.temperature[row];
    if (!(t >= 0.f) || t == INFINITY) return;      // such a row is left as it was, by all of the cluster
    if (ranks > 1) cluster_arrive();
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_row;
    float* p = a.p + row * a.p_row;
    // vectors begin at 16-byte boundaries: the first may begin before the row
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int vecs = (int)(((long long)a.vocab + off + VE - 1) / VE), per = (vecs + ranks - 1) / ranks;
    const int v0 = (int)rank * per, v1 = min(v0 + per, vecs);
    float w[K * VE];
    {
        uint4 raw[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = v0 + k * CT + tid;
            const int e = v * VE - off;
            if (v < v1 && e >= 0 && e + VE <= a.vocab) raw[k] = *reinterpret_cast<const uint4*>(x + e);
        }
        if (tid == 0) {      // while they are on their way
            s_setup = setup_of(t, row_min_p(a, row));
            s_best = 0x7fffffff;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = v0 + k * CT + tid;
            const int e = v * VE - off;
            const T* r = reinterpret_cast<const T*>(&raw[k]);
            const bool full = v < v1 && e >= 0 && e + VE <= a.vocab;
#pragma unroll
            for (int i = 0; i < VE; ++i) w[k * VE + i] = full ? no_nan(to_f32(r[i])) : -INFINITY;
            if (v < v1 && !full)
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (e + i >= 0 && e + i < a.vocab) w[k * VE + i] = no_nan(to_f32(x[e + i]));
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < K * VE; ++i) m = fmaxf(m, w[i]);
    m = trade(s_max, warp_max(m), ranks, rank, true, [](float x, float y) { return fmaxf(x, y); });
    if (t == 0.f || m == -INFINITY) {
        int best = 0x7fffffff;
        if (m != -INFINITY)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (w[k * VE + i] == m) best = min(best, (v0 + k * CT + tid) * VE - off + i);
        best = (int)__reduce_min_sync(0xffffffffu, (unsigned)best);
        if ((tid & 31) == 0) atomicMin(&s_best, best);
        __syncthreads();
        best = s_best;
        if (ranks > 1) {
            if (tid < ranks) put_remote(&s_sum.all[rank], tid, (uint32_t)best);
            cluster_arrive();
            cluster_wait();
            for (int i = 0; i < ranks; ++i) best = min(best, (int)s_sum.all[i]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i) w[k * VE + i] = (v0 + k * CT + tid) * VE - off + i == best ? 1.f : 0.f;
    } else {
        const RowRule r = rule_of(m, s_setup);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < K * VE; ++i) {
            w[i] = weight(r, w[i]);
            sum += w[i];
        }
        sum = trade(s_sum, warp_sum(sum), ranks, rank, false, [](float x, float y) { return x + y; });
        const float inv = 1.f / sum;
#pragma unroll
        for (int i = 0; i < K * VE; ++i) w[i] *= inv;
    }
    const bool wide = ((reinterpret_cast<uintptr_t>(p) / 4 - off) & 3) == 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = v0 + k * CT + tid;
        const int e = v * VE - off;
        if (v >= v1) continue;
        if (wide && e >= 0 && e + VE <= a.vocab) {
#pragma unroll
            for (int i = 0; i < VE; i += 4)
                *reinterpret_cast<float4*>(p + e + i) =
                    make_float4(w[k * VE + i], w[k * VE + i + 1], w[k * VE + i + 2], w[k * VE + i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (e + i >= 0 && e + i < a.vocab) p[e + i] = w[k * VE + i];
        }
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
    float sum = 0.f;
    for (int i = tid; i < a.vocab; i += PT) sum += weight(r, no_nan(to_f32(x[i])));
    sum = warp_sum(sum);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = warp_sum(red[lane]);
    const float inv = 1.f / sum;
    for (int i = tid; i < a.vocab; i += PT) p[i] = weight(r, no_nan(to_f32(x[i]))) * inv;
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
    set_carveout_once(kern);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.rows * ranks));
    cfg.blockDim = dim3(CT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    ++g_launches;
    return (int)cudaLaunchKernelEx(&cfg, probs_cluster_kernel<T, K>, a, ranks);
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
