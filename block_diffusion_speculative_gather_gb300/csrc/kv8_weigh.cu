// Accumulated attention weight of the 8-bit paged cache's positions.
//
//   weight[j] (+)= sum over the counted rows i and their q heads h of
//                  exp(scale q_ih . k_j - lse_ih)    where row i sees position j
// with lse the log of the row's softmax sum that the attention has left, so
// every term is the weight that the attention gave the position.
//
// A CTA has a page of one sequence, all its kv heads: no two CTAs add to the
// same position, so there are no atomics, and the order of the terms is fixed.

#include "gemm.cuh"
#include "kv8.cuh"
#include "kv8_attn_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;

constexpr int WT = 256;
constexpr int WG = WT / KV8_PAGE;     // rows dealt to this many threads of a position

template <typename T, int HD>
__global__ void __launch_bounds__(WT) kv8_weigh_kernel(Kv8WeighArgs a) {
    __shared__ float red[WG][KV8_PAGE];
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.y, page = blockIdx.x, tid = threadIdx.x;
    const int r0 = a.row_start[s], n = a.row_start[s + 1] - r0, kv = a.kv_len[s];
    if (r0 < 0 || n < 0 || r0 + n > a.rows || kv < 0 || kv > (long long)a.max_pages * KV8_PAGE) {
        if (page == 0 && tid == 0) report(a.err, DERR_INDEX, SITE_LEN);
        return;
    }
    if (page * KV8_PAGE >= kv) return;
    const int pg = a.table[(size_t)s * a.max_pages + page];
    if (pg < 0 || pg >= a.n_pages) {
        if (tid == 0) report(a.err, DERR_INDEX, SITE_PAGE);
        return;
    }
    int i1 = n;
    if (a.count) i1 = min(max(a.count[s], 0), n);
    const int i0 = a.observe > 0 ? max(i1 - a.observe, 0) : 0;
    const int first = kv - n, k = tid % KV8_PAGE, g = tid / KV8_PAGE, j = page * KV8_PAGE + k;
    float total = 0.f;
    for (int h = 0; h < a.n_kv; ++h) {
        const size_t at = (size_t)pg * a.n_kv + h;
        const float f = a.k_scale[at] * a.scale_log2;
        float kf[HD];
        const uint4* src = reinterpret_cast<const uint4*>(a.k_codes + (at * KV8_PAGE + k) * HD);
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
            const uint4 w = src[c];
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t two = f16_of_codes(x[e / 2] >> (16 * (e % 2)));
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&two));
                kf[16 * c + 2 * e] = v.x;
                kf[16 * c + 2 * e + 1] = v.y;
            }
        }
        for (int r = i0 * a.group + g; r < i1 * a.group; r += WG) {
            const int i = r / a.group, hq = h * a.group + r % a.group, p = first + i;
            bool seen;
            if (a.causal) seen = j <= p && (a.window <= 0 || (long long)j > (long long)p - a.window);
            else seen = j < kv && (a.window <= 0 || (long long)j >= (long long)first - a.window);
            const T* q = reinterpret_cast<const T*>(a.q) + (long long)(r0 + i) * a.q_row + (long long)hq * a.q_head;
            float dot = 0.f;
#pragma unroll 8
            for (int d = 0; d < HD; ++d) dot = fmaf(to_f32(q[d]), kf[d], dot);
            const float lse = a.lse[(long long)(r0 + i) * a.n_q + hq];
            if (seen && lse > -INFINITY) total += ex2(fmaf(dot, f, -lse * 1.4426950408889634f));
        }
    }
    red[g][k] = total;
    __syncthreads();
    if (g == 0 && j < kv) {
        float* w = a.weights + (size_t)pg * KV8_PAGE + k;
        const float old = a.fresh && j >= first ? 0.f : *w;
        *w = old + ((red[0][k] + red[1][k]) + (red[2][k] + red[3][k]));
    }
}

}  // namespace

int launch_kv8_weigh(const Kv8WeighArgs& a, int head_dim, cudaStream_t s) {
    const dim3 grid((unsigned)a.max_pages, (unsigned)a.S), block(WT);
    if (a.dtype == 1)
        return (int)(head_dim == 128 ? launch_k(kv8_weigh_kernel<__nv_bfloat16, 128>, grid, block, 0, s, a)
                                     : launch_k(kv8_weigh_kernel<__nv_bfloat16, 64>, grid, block, 0, s, a));
    return (int)(head_dim == 128 ? launch_k(kv8_weigh_kernel<__half, 128>, grid, block, 0, s, a)
                                 : launch_k(kv8_weigh_kernel<__half, 64>, grid, block, 0, s, a));
}

}  // namespace dfl
