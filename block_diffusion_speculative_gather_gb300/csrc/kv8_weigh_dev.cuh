// What the two forms of the accumulated weights share: a sequence's span, and
// which of its items are a CTA's.
#pragma once

#include "kv8.cuh"
#include "kv8_attn_dev.cuh"

namespace dfl {
namespace kv8 {

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

// Items of KEYS positions.
template <int KEYS> __device__ __forceinline__ int items_of(const Span& q) {
    return q.hi > q.lo ? (q.hi - 1) / KEYS - q.lo / KEYS + 1 : 0;
}

// A run of neighbouring items [first, last) for this CTA, the sequence that the
// first belongs to, and in `before` (a.S + 1 ints of shared memory) the items before
// each sequence.  By all THREADS threads of the CTA; `sums`: THREADS / 32 ints.
struct Run {
    int first, last, s;
};

template <int KEYS, int THREADS>
__device__ __forceinline__ Run my_items(const Kv8WeighArgs& a, int* before, int* sums) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int each = (a.S + THREADS - 1) / THREADS;
    int mine = 0;
    for (int s = tid * each; s < a.S && s < (tid + 1) * each; ++s)
        mine = add_counts(mine, items_of<KEYS>(span_of(a, s, blockIdx.x == 0)));
    const int inc = warp_inclusive(mine, lane);
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int run = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) run = add_counts(run, sums[w]);
        total = add_counts(total, sums[w]);
    }
    run = add_counts(run, inc - mine);
    for (int s = tid * each; s < a.S && s < (tid + 1) * each; ++s) {
        before[s] = run;
        if (each > 1) run = add_counts(run, items_of<KEYS>(span_of(a, s, false)));
    }
    if (tid == 0) before[a.S] = total;
    __syncthreads();
    Run r;
    r.first = (int)((long long)total * blockIdx.x / gridDim.x);
    r.last = (int)((long long)total * (blockIdx.x + 1) / gridDim.x);
    r.s = 0;
    for (int len = a.S; len > 1;) {        // the last sequence that begins at or before the first item
        const int st = (len + 31) / 32, at = lane * st;
        const int m = __popc(__ballot_sync(0xffffffffu, at < len && before[r.s + at] <= r.first)) - 1;
        r.s += m * st;
        len = min(st, len - m * st);
    }
    return r;
}

}  // namespace kv8
}  // namespace dfl
