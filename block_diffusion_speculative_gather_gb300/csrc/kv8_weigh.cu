// Accumulated attention weight of the 8-bit paged cache's positions.
//
//   weight[j] (+)= sum over the counted rows i and their q heads h of
//                  exp(scale q_ih . k_j - lse_ih)    where row i sees position j
// with lse the log of the row's softmax sum that the attention has left, so
// every term is the weight that the attention gave the position.
//
// Scores are K q^T in mma.sync tiles with the cached keys as the M side: 16 keys
// of one page a warp, 8 (row, q head) pairs of one kv head a step, so a key's
// sum runs over the columns: in the registers of a lane, over the quad at the
// end.  q enters as f16, a row scaled by the power of two that brings its largest
// element into [1, 2) (as the attention does), e4m3 codes are exact in f16;
// scores, exponents and sums are fp32.  tcgen05 would need the scores moved out
// of tensor memory for the same exponentials, which are what many rows cost.
//
// An item is 128 keys of one sequence, all kv heads, 8 warps: no two CTAs add to
// the same position, so there are no atomics, and the order of the terms is
// fixed.  The rows pass through shared memory, 64 at a time, and serve all 8
// warps; keys go straight to registers, two heads ahead.

#include "gemm.cuh"
#include "kv8.cuh"
#include "kv8_attn_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;

constexpr int WT = 256;
constexpr int WW = WT / 32;
constexpr int WKEYS = 16 * WW;        // keys of an item
constexpr int WROWS = 8 * WW;         // packed rows of a stage
constexpr int WSEQS = 4096;

// A sequence's counted rows [i0, i1) and the positions [lo, hi) to go through.
struct Span {
    int r0, i0, i1, first, kv, lo, hi;
};

__device__ __forceinline__ Span span_of(const Kv8WeighArgs& a, int s, bool tell) {
    Span q{};
    const int r0 = a.row_start[s], r1 = a.row_start[s + 1], kv = a.kv_len[s];
    if (r0 < 0 || r1 < r0 || r1 > a.rows || kv < 0 || kv > (long long)a.max_pages * KV8_PAGE) {
        if (tell) report(a.err, DERR_INDEX, SITE_LEN);    // such a sequence is left out
        return q;
    }
    const int n = r1 - r0;
    q.r0 = r0;
    q.kv = kv;
    q.first = kv - n;
    q.i1 = a.count ? min(max(a.count[s], 0), n) : n;
    q.i0 = a.observe > 0 ? max(q.i1 - a.observe, 0) : 0;
    if (q.i1 > q.i0) {
        q.hi = a.causal ? max(q.first + q.i1, 0) : kv;
        const int end = a.causal ? q.first + q.i0 + 1 : q.first;
        if (a.window > 0 && end > a.window) q.lo = end - a.window;
    } else {
        q.lo = kv;
    }
    if (a.fresh && n > 0) {
        q.lo = min(q.lo, max(q.first, 0));
        q.hi = kv;
    }
    return q;
}

__device__ __forceinline__ int blocks_of(const Span& q) { return q.hi > q.lo ? (q.hi - 1) / WKEYS - q.lo / WKEYS + 1 : 0; }

template <int HD> struct WeighSmem {
    static constexpr int pitch = HD * 2 + 16;      // bytes: lanes of 8 read all banks
    alignas(16) uint8_t q[WROWS * pitch];
    float2 col[WROWS];           // score factor, lse in base 2 (inf: the column does not count)
    int row[WROWS];
    int before[WSEQS + 1];       // items before each sequence
    int warp[WW];
};

template <typename T, int HD>
__global__ void __launch_bounds__(WT, 2) kv8_weigh_kernel(const __grid_constant__ Kv8WeighArgs a) {
    using S_ = WeighSmem<HD>;
    __shared__ S_ sm;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    // items before each sequence
    const int per = (a.S + WT - 1) / WT;
    int mine = 0;
    for (int s = tid * per; s < a.S && s < (tid + 1) * per; ++s) mine = add_counts(mine, blocks_of(span_of(a, s, blockIdx.x == 0)));
    const int inc = warp_inclusive(mine, lane);
    if (lane == 31) sm.warp[warp] = inc;
    __syncthreads();
    int run = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WW; ++w) {
        if (w < warp) run = add_counts(run, sm.warp[w]);
        total = add_counts(total, sm.warp[w]);
    }
    run = add_counts(run, inc - mine);
    for (int s = tid * per; s < a.S && s < (tid + 1) * per; ++s) {
        sm.before[s] = run;
        if (per > 1) run = add_counts(run, blocks_of(span_of(a, s, false)));
    }
    if (tid == 0) sm.before[a.S] = total;
    __syncthreads();

    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        int s = 0;
        for (int len = a.S; len > 1;) {        // the last sequence that begins at or before the item
            const int st = (len + 31) / 32, at = lane * st;
            const int m = __popc(__ballot_sync(0xffffffffu, at < len && sm.before[s + at] <= item)) - 1;
            s += m * st;
            len = min(st, len - m * st);
        }
        const Span q = span_of(a, s, false);
        const int key0 = (q.lo / WKEYS + (item - sm.before[s])) * WKEYS + 16 * warp;   // the warp's first key
        int pg = -1;
        if (key0 < q.hi && key0 + 16 > q.lo) {
            pg = a.table[(size_t)s * a.max_pages + key0 / KV8_PAGE];
            if (pg < 0 || pg >= a.n_pages) {
                report(a.err, DERR_INDEX, SITE_PAGE);
                pg = -1;
            }
        }
        const bool active = pg >= 0;
        const int off = key0 % KV8_PAGE;
        uint4 ahead[2][HD / 32];
        float ahead_scale[2];
        auto fetch = [&](int h, uint4 (&x)[HD / 32], float* scale) {
            if (!active || h >= a.n_kv) return;
            const size_t at = (size_t)pg * a.n_kv + h;
            const uint8_t* src = a.k_codes + (at * KV8_PAGE + off + g) * HD + 16 * c;
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) {
                x[2 * i] = *reinterpret_cast<const uint4*>(src + 64 * i);
                x[2 * i + 1] = *reinterpret_cast<const uint4*>(src + 8 * HD + 64 * i);
            }
            *scale = a.k_scale[at];
        };
        fetch(0, ahead[0], ahead_scale);
        fetch(1, ahead[1], ahead_scale + 1);
        float* wp = a.weights + (size_t)max(pg, 0) * KV8_PAGE + off + g;
        float old[2] = {0.f, 0.f};
        if (active && c == 0)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = key0 + g + 8 * e;
                if (j < q.kv && !(a.fresh && j >= q.first)) old[e] = wp[8 * e];
            }

        const int packed = (q.i1 - q.i0) * a.group, per_head = (packed + 7) / 8, blocks = per_head * a.n_kv;
        // keys that every row sees, and keys that some row sees
        const int last = key0 + 15;
        bool whole = last < q.kv, none = !active;
        if (a.causal) {
            whole = whole && last <= q.first + q.i0 && (a.window <= 0 || key0 > (long long)q.first + q.i1 - 1 - a.window);
            none = none || key0 > q.first + q.i1 - 1;
        } else if (a.window > 0) {
            whole = whole && key0 >= (long long)q.first - a.window;
        }
        uint32_t k[HD / 16][4];
        float scale = 0.f, sum[2] = {0.f, 0.f};
        int head = -1;
        for (int b0 = 0; b0 < blocks; b0 += WW) {
            __syncthreads();       // the rows before have been used
            if (b0 + warp < blocks) {
                // this warp's 8 rows: a row by HD / 8 lanes, 16 bytes each
                constexpr int LANES = HD / 8, AT_ONCE = 32 / LANES;
                const int h = (b0 + warp) / per_head, p0 = (b0 + warp - h * per_head) * 8;
                uint4 x[8 / AT_ONCE];
                float lse = 0.f;
#pragma unroll
                for (int r = 0; r < 8; r += AT_ONCE) {
                    const int p = p0 + r + lane / LANES;
                    x[r / AT_ONCE] = make_uint4(0, 0, 0, 0);
                    if (p < packed)
                        x[r / AT_ONCE] = *reinterpret_cast<const uint4*>(
                            reinterpret_cast<const T*>(a.q) + (long long)(q.r0 + q.i0 + p / a.group) * a.q_row +
                            (long long)(h * a.group + p % a.group) * a.q_head + (lane % LANES) * 8);
                }
                if (lane < 8) {
                    const int p = p0 + lane;
                    lse = INFINITY;
                    if (p < packed) {
                        const float v = a.lse[(long long)(q.r0 + q.i0 + p / a.group) * a.n_q + h * a.group + p % a.group];
                        if (v > -INFINITY) lse = v * 1.4426950408889634f;
                    }
                    sm.row[8 * warp + lane] = q.i0 + p / a.group;
                }
#pragma unroll
                for (int r = 0; r < 8; r += AT_ONCE) {
                    const T* e = reinterpret_cast<const T*>(&x[r / AT_ONCE]);
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float v = fabsf(to_f32(e[i]));
                        top = fmaxf(top, v < INFINITY ? v : 0.f);
                    }
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    float inv, back;
                    row_factor(top, &inv, &back);
                    uint4 y;
                    y.x = pack_f16x2(to_f32(e[0]) * inv, to_f32(e[1]) * inv);
                    y.y = pack_f16x2(to_f32(e[2]) * inv, to_f32(e[3]) * inv);
                    y.z = pack_f16x2(to_f32(e[4]) * inv, to_f32(e[5]) * inv);
                    y.w = pack_f16x2(to_f32(e[6]) * inv, to_f32(e[7]) * inv);
                    const int row = 8 * warp + r + lane / LANES;
                    *reinterpret_cast<uint4*>(sm.q + row * S_::pitch + (lane % LANES) * 16) = y;
                    const float l = __shfl_sync(0xffffffffu, lse, r + lane / LANES);
                    if (lane % LANES == 0) sm.col[row] = make_float2(back * a.scale_log2, l);
                }
            }
            __syncthreads();
            if (none) continue;
            const int most = min(WW, blocks - b0);
            for (int b = 0; b < most; ++b) {
                const int h = (b0 + b) / per_head;
                if (h != head) {
                    head = h;
#pragma unroll
                    for (int i = 0; i < HD / 64; ++i) {
                        const uint32_t lo[4] = {ahead[0][2 * i].x, ahead[0][2 * i].y, ahead[0][2 * i].z, ahead[0][2 * i].w};
                        const uint32_t up[4] = {ahead[0][2 * i + 1].x, ahead[0][2 * i + 1].y, ahead[0][2 * i + 1].z,
                                                ahead[0][2 * i + 1].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            k[4 * i + j][0] = f16_of_codes(lo[j]);
                            k[4 * i + j][1] = f16_of_codes(up[j]);
                            k[4 * i + j][2] = f16_of_codes(lo[j] >> 16);
                            k[4 * i + j][3] = f16_of_codes(up[j] >> 16);
                        }
                    }
                    scale = ahead_scale[0];
                    if (!(scale >= 0.f && scale < INFINITY)) {
                        report(a.err, DERR_INDEX, SITE_SCALE);
                        scale = __int_as_float(0x7fffffff);     // scores that add nothing
                    }
#pragma unroll
                    for (int i = 0; i < HD / 32; ++i) ahead[0][i] = ahead[1][i];
                    ahead_scale[0] = ahead_scale[1];
                    fetch(head + 2, ahead[1], ahead_scale + 1);
                }
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                const uint8_t* qp = sm.q + (8 * b + g) * S_::pitch + 32 * c;
#pragma unroll
                for (int i = 0; i < HD / 64; ++i) {
                    const uint4 lo = lds128(qp + 128 * i), hi = lds128(qp + 128 * i + 16);
                    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t bb[2] = {w[2 * j], w[2 * j + 1]};
                        mma_f16_16816(d, k[4 * i + j], bb);
                    }
                }
                const float4 col = *reinterpret_cast<const float4*>(sm.col + 8 * b + 2 * c);
                // a NaN score (a NaN code) adds nothing: 2^-200 is 0
                float x[4];
                const float f0 = col.x * scale, f1 = col.z * scale;
                x[0] = fmaxf(fmaf(d[0], f0, -col.y), -200.f);
                x[1] = fmaxf(fmaf(d[1], f1, -col.w), -200.f);
                x[2] = fmaxf(fmaf(d[2], f0, -col.y), -200.f);
                x[3] = fmaxf(fmaf(d[3], f1, -col.w), -200.f);
                if (!whole) {
                    const int i0 = sm.row[8 * b + 2 * c], i1 = sm.row[8 * b + 2 * c + 1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = key0 + g + 8 * (e >> 1), p = q.first + (e & 1 ? i1 : i0);
                        bool seen;
                        if (a.causal) seen = j <= p && (a.window <= 0 || j > (long long)p - a.window);
                        else seen = j < q.kv && (a.window <= 0 || j >= (long long)q.first - a.window);
                        if (!seen) x[e] = -200.f;
                    }
                }
                sum[0] += ex2(x[0]) + ex2(x[1]);
                sum[1] += ex2(x[2]) + ex2(x[3]);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
            sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
            const int j = key0 + g + 8 * e;
            if (active && c == 0 && j < q.kv) wp[8 * e] = old[e] + sum[e];
        }
    }
}

}  // namespace

int launch_kv8_weigh(const Kv8WeighArgs& a, int head_dim, int sms, cudaStream_t s) {
    // items there can be: 128 keys each
    const long long most = (long long)a.S * ((a.max_pages + 1) / 2);
    const dim3 grid((unsigned)(most < 2 * sms ? most : 2 * sms)), block(WT);
    if (a.dtype == 1)
        return (int)(head_dim == 128 ? launch_k(kv8_weigh_kernel<__nv_bfloat16, 128>, grid, block, 0, s, a)
                                     : launch_k(kv8_weigh_kernel<__nv_bfloat16, 64>, grid, block, 0, s, a));
    return (int)(head_dim == 128 ? launch_k(kv8_weigh_kernel<__half, 128>, grid, block, 0, s, a)
                                 : launch_k(kv8_weigh_kernel<__half, 64>, grid, block, 0, s, a));
}

}  // namespace dfl
