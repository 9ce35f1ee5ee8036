// Probabilities of rows of logits.
//
//   p_v = w_v / sum w,  w_v = exp((x_v - m) / T) where x_v >= m + T ln(min_p), else 0
// with m the row's maximum; T = 0: 1 at the first maximum.  NaN logits count as
// -inf; where the maximum is +inf its holders share the row.
//
// The border m + T ln(min_p) is taken in 64 bits and rounded up to the next
// fp32 value, so that comparing fp32 logits with it is exact.  Weights, sums
// and quotients are fp32.
//
// A row is read three times (maximum, sum, quotients), after the first from L2.

#include "gemm.cuh"
#include "sampling.cuh"

namespace dfl {
namespace {

constexpr int PT = 1024;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float no_nan(float x) { return x == x ? x : -INFINITY; }

struct RowRule {
    float m, c, border;   // maximum, log2(e) / T, smallest logit that counts
};

__device__ __forceinline__ RowRule rule_of(float m, float t, float min_p) {
    RowRule r;
    r.m = m;
    r.c = fminf(1.4426950408889634f / t, 3.402823466e38f);   // no 0 * inf at the smallest T
    r.border = -INFINITY;
    if (min_p > 0.f) r.border = __double2float_ru((double)m + (double)t * log((double)fminf(min_p, 1.f)));
    return r;
}

__device__ __forceinline__ float weight(const RowRule& r, float x) {
    const float d = x == r.m ? 0.f : x - r.m;      // inf - inf
    return x >= r.border ? ex2(d * r.c) : 0.f;
}

template <typename T>
__global__ void __launch_bounds__(PT) probs_rows_kernel(ProbsArgs a) {
    __shared__ float red[32];
    __shared__ unsigned long long red_key;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const float t = a.temperature[row];
    if (!(t >= 0.f) || t == INFINITY) return;      // such a row is left as it was
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_row;
    float* p = a.p + row * a.p_row;
    if (tid == 0) red_key = 0;
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
    const RowRule r = rule_of(m, t, a.min_p ? a.min_p[row] : 0.f);
    float sum = 0.f;
    for (int i = tid; i < a.vocab; i += PT) sum += weight(r, no_nan(to_f32(x[i])));
    sum = warp_sum(sum);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = warp_sum(red[lane]);
    const float inv = 1.f / sum;
    for (int i = tid; i < a.vocab; i += PT) p[i] = weight(r, no_nan(to_f32(x[i]))) * inv;
}

}  // namespace

int launch_probs(const ProbsArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)a.rows), block(PT);
    if (a.dtype == 0) return (int)launch_k(probs_rows_kernel<float>, grid, block, 0, s, a);
    if (a.dtype == 1) return (int)launch_k(probs_rows_kernel<__nv_bfloat16>, grid, block, 0, s, a);
    return (int)launch_k(probs_rows_kernel<__half>, grid, block, 0, s, a);
}

}  // namespace dfl
