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
// end.  q enters as f16, a bf16 row scaled by the power of two that brings its
// largest element into [1, 2) (as the attention does), e4m3 codes are exact in f16;
// scores, exponents and sums are fp32.  Many rows go by tcgen05 (kv8_weigh_tc.cu).
//
// An item is 128 keys, 16 a warp, all kv heads: no two CTAs add to the same
// position, so there are no atomics, and the order of the terms is fixed.  A CTA
// has a run of neighbouring items.  Their rows pass through shared memory, 8 a warp
// at a time, and stay there from item to item where a sequence has no more.  A warp's
// keys come by asynchronous copies, three heads ahead, from one item into the
// next; a lane reads what it copied itself, so that no barrier stands between.
//
// 32 single tokens over 10000 positions each on average (32 heads on 8) take 63 us for
// 345 MB, 5.5 TB/s: DRAM, beside the conversion of the codes (half of the issue slots).
// One token over 1088 takes 8.3 us, a chain of trips to memory: lengths, table, keys,
// with the rows and their lse beside, then the exponentials of eight heads.

#include <type_traits>

#include "copy_dev.cuh"
#include "gemm.cuh"
#include "kv8.cuh"
#include "kv8_attn_dev.cuh"
#include "kv8_weigh_dev.cuh"

namespace dfl {
namespace {

using namespace kv8;

constexpr int W = 8, WT = 32 * W, KEYS = 16 * W;
constexpr int RING = 4;              // heads of a warp's keys, on their way or at hand

template <int HD> struct WeighSmem {
    static constexpr int pitch = HD * 2 + 16;      // bytes: 8 lanes' rows fall on all banks
    uint8_t q[8 * W * pitch];
    uint4 keys[W][RING][HD / 32][32];
    float scale[W][RING];
    float2 col[8 * W];           // score factor, lse in base 2 (inf: the column does not count)
    int row[8 * W];
    int before[WSEQS + 1];       // items before each sequence
    int warp[W];
};

template <typename T, int HD>
__global__ void __launch_bounds__(WT, 2) kv8_weigh_kernel(const __grid_constant__ Kv8WeighArgs a) {
    using S_ = WeighSmem<HD>;
    extern __shared__ __align__(16) uint8_t raw[];
    S_& sm = *reinterpret_cast<S_*>(raw);
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const Run run = my_items<KEYS, WT>(a, sm.before, sm.warp);
    if (run.first >= run.last) return;
    int s = run.s;
    bool begins = true;                  // the item is the first of its sequence here
    bool fresh_rows = true;
    Span q = span_of(a, s, false);
    const int* table = nullptr;
    const int off = 16 * warp % KV8_PAGE + g;        // of the lane's first key in its page
    // the copies: head `h` of item `at` comes next, from `src`; `pg` its page (-1: none),
    // `ahead` the table's entry for the item behind it, `end` the sequence's last here
    int at = 0, h_next = 0, pg_next = -1, ahead = -1, end = 0;
    unsigned step = 0, fetched = 0;                  // heads used, asked for
    const uint8_t* src = nullptr;
    auto key_of_item = [&](int item) { return (q.lo / KEYS + (item - sm.before[s])) * KEYS + 16 * warp; };
    auto entry = [&](int item) {                     // raw: not looked at before it has arrived
        const int key = key_of_item(item);
        return item < end && key < q.hi && key + 16 > q.lo ? table[key / KV8_PAGE] : -0x7fffffff;
    };
    auto page = [&](int e) {
        if (e >= 0 && e < a.n_pages) return e;
        if (e != -0x7fffffff) report(a.err, DERR_INDEX, SITE_PAGE);
        return -1;
    };
    auto fetch = [&]() {
        const int slot = fetched % RING;
        if (at < end && pg_next >= 0) {
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) {
                copy_async16(&sm.keys[warp][slot][2 * i][lane], src + 64 * i);
                copy_async16(&sm.keys[warp][slot][2 * i + 1][lane], src + 8 * HD + 64 * i);
            }
            if (lane == 0) copy_async4(&sm.scale[warp][slot], a.k_scale + (size_t)pg_next * a.n_kv + h_next);
        }
        copy_commit();
        ++fetched;
        src += KV8_PAGE * HD;
        if (++h_next == a.n_kv) {
            h_next = 0;
            ++at;
            pg_next = page(ahead);
            src = a.k_codes + ((size_t)max(pg_next, 0) * a.n_kv * KV8_PAGE + off) * HD + 16 * c;
            ahead = entry(at + 1);
        }
    };
    for (int item = run.first; item < run.last; ++item) {
        if (item >= sm.before[s + 1]) {
            do ++s;
            while (item >= sm.before[s + 1]);
            q = span_of(a, s, false);
            begins = true;
        }
        if (begins) {
            begins = false;
            fresh_rows = true;
            table = a.table + (size_t)s * a.max_pages;
            end = min(run.last, sm.before[s + 1]);
            copy_wait<0>();              // (all groups are empty: nothing is asked for behind a sequence's end)
            __syncwarp();
            step = fetched = 0;
            at = item;
            h_next = 0;
            pg_next = page(entry(item));
            src = a.k_codes + ((size_t)max(pg_next, 0) * a.n_kv * KV8_PAGE + off) * HD + 16 * c;
            ahead = entry(item + 1);
            for (int i = 0; i < RING - 1; ++i) fetch();
        }
        const int key0 = key_of_item(item);          // the warp's first key
        int pg = -1;
        if (key0 < q.hi && key0 + 16 > q.lo) {
            pg = table[key0 / KV8_PAGE];
            if (pg < 0 || pg >= a.n_pages) pg = -1;  // reported with the copies
        }
        const bool active = pg >= 0;
        float* wp = a.weights + (size_t)max(pg, 0) * KV8_PAGE + off;
        float old[2] = {0.f, 0.f};
        if (active && c == 0)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = key0 + g + 8 * e;
                if (j < q.kv && !(a.fresh && j >= q.first)) old[e] = wp[8 * e];
            }

        const int packed = (q.i1 - q.i0) * a.group, per_head = (packed + 7) / 8, blocks = per_head * a.n_kv;
        // keys that every row sees, and keys that no row sees
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
        int in_head = per_head;          // of the next block: its head's first in_head have been done
        const unsigned done = step + a.n_kv;
        for (int b0 = 0; b0 < blocks; b0 += W) {
            if (fresh_rows) {
                __syncthreads();                   // the rows before have been used
                if (b0 + warp < blocks) {
                    // this warp's 8 rows: a row by HD / 8 lanes, 16 bytes each
                    constexpr int LANES = HD / 8, AT_ONCE = 32 / LANES;
                    const int h = (b0 + warp) / per_head, p0 = (b0 + warp - h * per_head) * 8;
                    uint4 x[8 / AT_ONCE];
                    float lse = 0.f;
#pragma unroll
                    for (int r = 0; r < 8; r += AT_ONCE) {
                        const int p = p0 + r + lane / LANES, i = p / a.group;
                        x[r / AT_ONCE] = make_uint4(0, 0, 0, 0);
                        if (p < packed)
                            x[r / AT_ONCE] = *reinterpret_cast<const uint4*>(
                                reinterpret_cast<const T*>(a.q) + (long long)(q.r0 + q.i0 + i) * a.q_row +
                                (long long)(h * a.group + p - i * a.group) * a.q_head + (lane % LANES) * 8);
                    }
                    if (lane < 8) {
                        const int p = p0 + lane, i = p / a.group;
                        lse = INFINITY;
                        if (p < packed) {
                            const float v = a.lse[(long long)(q.r0 + q.i0 + i) * a.n_q + h * a.group + p - i * a.group];
                            if (v > -INFINITY) lse = v * 1.4426950408889634f;
                        }
                        sm.row[8 * warp + lane] = q.i0 + i;
                    }
#pragma unroll
                    for (int r = 0; r < 8; r += AT_ONCE) {
                        uint4 y = x[r / AT_ONCE];
                        float back = 1.f;
                        if constexpr (!std::is_same<T, __half>::value) {
                            const T* e = reinterpret_cast<const T*>(&x[r / AT_ONCE]);
                            float top = 0.f, inv;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float v = fabsf(to_f32(e[i]));
                                top = fmaxf(top, v < INFINITY ? v : 0.f);
                            }
#pragma unroll
                            for (int o = LANES / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            row_factor(top, &inv, &back);
                            y.x = pack_f16x2(to_f32(e[0]) * inv, to_f32(e[1]) * inv);
                            y.y = pack_f16x2(to_f32(e[2]) * inv, to_f32(e[3]) * inv);
                            y.z = pack_f16x2(to_f32(e[4]) * inv, to_f32(e[5]) * inv);
                            y.w = pack_f16x2(to_f32(e[6]) * inv, to_f32(e[7]) * inv);
                        }
                        const int row = 8 * warp + r + lane / LANES;
                        *reinterpret_cast<uint4*>(sm.q + row * S_::pitch + (lane % LANES) * 16) = y;
                        const float l = __shfl_sync(0xffffffffu, lse, r + lane / LANES);
                        if (lane % LANES == 0) sm.col[row] = make_float2(back * a.scale_log2, l);
                    }
                }
                __syncthreads();
                fresh_rows = blocks > W;           // else they stay for the sequence's next items
            }
            if (none) continue;
            // scores of block b (8 columns) of the stage, two accumulators each
            auto score = [&](int b, float (&d)[2][4]) {
                const uint8_t* qp = sm.q + (8 * b + g) * S_::pitch + 32 * c;
#pragma unroll
                for (int i = 0; i < HD / 64; ++i) {
                    const uint4 lo = lds128(qp + 128 * i), hi = lds128(qp + 128 * i + 16);
                    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t bb[2] = {w[2 * j], w[2 * j + 1]};
                        mma_f16_16816(d[j & 1], k[4 * i + j], bb);
                    }
                }
            };
            auto add_up = [&](int b, const float (&d)[2][4]) {
                const float4 col = *reinterpret_cast<const float4*>(sm.col + 8 * b + 2 * c);
                // a NaN score (a NaN code) adds nothing: 2^-200 is 0
                const float f0 = col.x * scale, f1 = col.z * scale;
                float x[4];
                x[0] = fmaxf(fmaf(d[0][0] + d[1][0], f0, -col.y), -200.f);
                x[1] = fmaxf(fmaf(d[0][1] + d[1][1], f1, -col.w), -200.f);
                x[2] = fmaxf(fmaf(d[0][2] + d[1][2], f0, -col.y), -200.f);
                x[3] = fmaxf(fmaf(d[0][3] + d[1][3], f1, -col.w), -200.f);
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
            };
            const int most = min(W, blocks - b0);
            for (int b = 0; b < most;) {
                if (in_head == per_head) {         // the next head's keys
                    in_head = 0;
                    __syncwarp();                  // the scale's place has been read
                    fetch();
                    copy_wait<RING - 1>();
                    __syncwarp();                  // lane 0's copy of the scale
                    const int slot = step++ % RING;
#pragma unroll
                    for (int i = 0; i < HD / 64; ++i) {
                        const uint4 x = sm.keys[warp][slot][2 * i][lane], y = sm.keys[warp][slot][2 * i + 1][lane];
                        const uint32_t lo[4] = {x.x, x.y, x.z, x.w}, up[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            k[4 * i + j][0] = f16_of_codes(lo[j]);
                            k[4 * i + j][1] = f16_of_codes(up[j]);
                            k[4 * i + j][2] = f16_of_codes(lo[j] >> 16);
                            k[4 * i + j][3] = f16_of_codes(up[j] >> 16);
                        }
                    }
                    scale = sm.scale[warp][slot];
                    if (!(scale >= 0.f && scale < INFINITY)) {
                        report(a.err, DERR_INDEX, SITE_SCALE);
                        scale = __int_as_float(0x7fffffff);     // scores that add nothing
                    }
                }
                float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                if (b + 1 < most && in_head + 1 < per_head) {
                    float e[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                    score(b, d);
                    score(b + 1, e);
                    add_up(b, d);
                    add_up(b + 1, e);
                    b += 2;
                    in_head += 2;
                } else {
                    score(b, d);
                    add_up(b, d);
                    ++b;
                    ++in_head;
                }
            }
        }
        while (step != done) {           // heads that were not looked at: their places are free once written
            fetch();
            copy_wait<RING - 1>();
            ++step;
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

template <typename T, int HD>
int launch_t(const Kv8WeighArgs& a, int sms, cudaStream_t s) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv8_weigh_kernel<T, HD>));
    if (e != cudaSuccess) return (int)e;
    const long long most = (long long)a.S * ((a.max_pages + 1) / 2);   // items
    return (int)launch_k(kv8_weigh_kernel<T, HD>, dim3((unsigned)(most < 2 * sms ? most : 2 * sms)), dim3(WT),
                         sizeof(WeighSmem<HD>), s, a);
}

}  // namespace

int launch_kv8_weigh(const Kv8WeighArgs& a, int head_dim, int sms, cudaStream_t s) {
    if (a.dtype == 1)
        return head_dim == 128 ? launch_t<__nv_bfloat16, 128>(a, sms, s) : launch_t<__nv_bfloat16, 64>(a, sms, s);
    return head_dim == 128 ? launch_t<__half, 128>(a, sms, s) : launch_t<__half, 64>(a, sms, s);
}

}  // namespace dfl
