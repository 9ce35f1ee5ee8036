// Verification of drafted tokens against the target's probabilities.
//
// Sequence s has n rows of the step; row i >= 1 holds draft d_i, drawn from q_i,
// and p_{i-1} is the target's distribution of the token behind row i - 1.
// d_i is accepted where u_i q_i(d_i) < p_{i-1}(d_i); a is the number accepted
// before the first refusal.  The last token is drawn from
//   w = max(p_a - q_{a+1}, 0)  after a refusal (p_a where that has no weight),
//   w = p_a                    where every draft was accepted,
// as the first v with w_0 + .. + w_v > u_0 * sum w.  So every emitted token is
// distributed as the target's.
//
// Which token a uniform number falls on is a matter of sums of up to a vocabulary
// of terms: differences are taken exactly (two fp32 numbers each), sums are kept
// as pairs of fp32 numbers within a warp and in fp64 above, in a fixed order.
//
// Only one row of p and q is read whole.  A CTA takes 4096 tokens of it (and
// finds by itself, from two numbers a draft, which row that is); the last of a
// sequence's CTAs finds the 4096 tokens that u_0 falls into and reads them again.
// No CTA waits for another.

#include "sampling.cuh"

namespace dfl {
namespace {

constexpr int VT = 256;                        // threads
constexpr int VW = VT / 32;
constexpr int PER = VERIFY_CHUNK / VT;         // tokens of a thread

// A sum as hi + lo, |lo| below half a step of hi.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair add(Pair a, float x, float e) {
    const float s = __fadd_rn(a.hi, x), b = __fsub_rn(s, a.hi);
    const float err = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, b)), __fsub_rn(x, b));
    return {s, __fadd_rn(a.lo, __fadd_rn(err, e))};
}

__device__ __forceinline__ double value(Pair a) { return (double)a.hi + (double)a.lo; }

__device__ __forceinline__ Pair warp_total(Pair a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Pair b{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
        // the same operands in the same order on both sides
        const bool first = !(threadIdx.x & o);
        const Pair x = first ? a : b, y = first ? b : a;
        a = add(x, y.hi, y.lo);
    }
    return a;
}

// What counts of a probability: negative and NaN ones are 0, and those of 2^100 or
// more, so that no sum leaves fp32.
__device__ __forceinline__ float clean(float p) { return p > 0.f && p < 0x1p100f ? p : 0.f; }

// Weight of a token: p - q where that is positive, exactly.
__device__ __forceinline__ Pair weight(float p, float q) {
    p = clean(p);
    q = clean(q);
    if (!(p > q)) return {0.f, 0.f};
    const float d = __fsub_rn(p, q), b = __fsub_rn(d, p);
    return {d, __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b))};
}

__device__ __forceinline__ void report(int* err, int info) {
    if (atomicCAS(err, 0, DERR_INDEX) == 0) err[1] = info;
}

// What the drafts of a sequence come to.
struct Verdict {
    int a;          // drafts accepted before the first refusal
    int draft;      // the refused token, -1: none (the last token comes from p alone)
};

// By a whole warp, the same in all lanes.
__device__ __forceinline__ Verdict judge(const VerifyArgs& a, int r0, int n, bool tell) {
    const int lane = threadIdx.x & 31;
    for (int b = 1; b < n; b += 32) {
        const int i = b + lane;
        bool refused = false;
        int d = -1;
        if (i < n) {
            d = a.ids[r0 + i];
            if (d >= a.vocab) {
                if (tell) report(a.err, r0 + i);
                d = -1;
            }
            refused = true;
            if (d >= 0) {
                const float p = clean(a.p[(long long)(r0 + i - 1) * a.p_row + d]);
                const float q = a.q ? clean(a.q[(long long)(r0 + i) * a.q_row + d]) : 1.f;
                refused = !((double)a.u[r0 + i] * (double)q < (double)p);
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, refused);
        if (m) {
            const int l = __ffs(m) - 1;
            const int id = __shfl_sync(0xffffffffu, d, l);
            return {b + l - 1, id < 0 ? -1 : id};
        }
    }
    return {n - 1, -1};
}

// The row that the last token is drawn from.
struct Row {
    const float* p;
    const float* q;     // NULL: nothing is taken off,
    int certain;        // but for this token (-1: none), which has no weight
};

template <bool WIDE>
__device__ __forceinline__ int token_of(int base, int k) {
    return WIDE ? base + (k / 4) * (VT * 4) + threadIdx.x * 4 + k % 4 : base + k * VT + threadIdx.x;
}

// Weights of the thread's tokens of a chunk, in the order of token_of.
template <bool WIDE>
__device__ __forceinline__ void load_chunk(const Row& r, int vocab, int base, Pair (&w)[PER]) {
    float p[PER], q[PER];
    if (WIDE) {
#pragma unroll
        for (int k = 0; k < PER; k += 4) {
            const int v = token_of<true>(base, k);
            const bool in = v < vocab;          // vocab is a multiple of 4
            const float4 x = in ? *reinterpret_cast<const float4*>(r.p + v) : make_float4(0.f, 0.f, 0.f, 0.f);
            p[k] = x.x, p[k + 1] = x.y, p[k + 2] = x.z, p[k + 3] = x.w;
            const float4 y = in && r.q ? *reinterpret_cast<const float4*>(r.q + v) : make_float4(0.f, 0.f, 0.f, 0.f);
            q[k] = y.x, q[k + 1] = y.y, q[k + 2] = y.z, q[k + 3] = y.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int v = token_of<false>(base, k);
            p[k] = v < vocab ? r.p[v] : 0.f;
            q[k] = v < vocab && r.q ? r.q[v] : 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) w[k] = weight(token_of<WIDE>(base, k) == r.certain ? 0.f : p[k], q[k]);
}

// Sum of a chunk's weights, the same in all threads.
template <bool WIDE>
__device__ __forceinline__ double chunk_sum(const Row& r, int vocab, int base, double* red) {
    Pair w[PER], s{0.f, 0.f};
    load_chunk<WIDE>(r, vocab, base, w);
#pragma unroll
    for (int k = 0; k < PER; ++k) s = add(s, w[k].hi, w[k].lo);
    s = warp_total(s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = value(s);
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < VW; ++i) t += red[i];
    return t;
}

// First token of the chunk whose running sum, from `before` on, passes `goal`;
// -1: none.  Its last token with weight where `last` is set.
template <bool WIDE>
__device__ int find_token(const Row& r, int vocab, int base, double before, double goal, bool last, double* red,
                          int* s_v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int STEP = WIDE ? 4 : 1;        // tokens of a thread that stand together
    Pair w[PER];
    load_chunk<WIDE>(r, vocab, base, w);
    if (threadIdx.x == 0) *s_v = last ? -1 : 0x7fffffff;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; k += STEP) {
        double own = 0.0;
#pragma unroll
        for (int j = 0; j < STEP; ++j) own += value(w[k + j]);
        double inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) red[warp] = inc;
        __syncthreads();
        double run = before;
        for (int i = 0; i < warp; ++i) run += red[i];
        for (int i = 0; i < VW; ++i) before += red[i];
        run += inc - own;
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
            run += value(w[k + j]);
            if (w[k + j].hi > 0.f) {
                if (last) atomicMax(s_v, token_of<WIDE>(base, k + j));
                else if (run > goal) atomicMin(s_v, token_of<WIDE>(base, k + j));
            }
        }
        __syncthreads();
    }
    const int v = *s_v;
    __syncthreads();
    return v == 0x7fffffff ? -1 : v;
}

// The last token of a row whose chunks' sums are `part`; -1: it has no weight.
template <bool WIDE>
__device__ int draw(const VerifyArgs& a, const Row& r, const double* part, float u, double* red, int* s_v) {
    __shared__ double s_total, s_before;
    __shared__ int s_c, s_end;
    if (threadIdx.x == 0) {
        double total = 0.0;
        int end = -1;
        for (int c = 0; c < a.chunks; ++c) {
            const double x = __ldcg(part + c);
            total += x;
            if (x > 0.0) end = c;
        }
        const double goal = (double)u * total;
        double run = 0.0;
        int at = -1;
        for (int c = 0; c < a.chunks && at < 0; ++c) {
            const double x = __ldcg(part + c);
            if (x > 0.0 && run + x > goal) at = c;
            else run += x;
        }
        s_total = total;
        s_before = run;
        s_c = at;
        s_end = end;
    }
    __syncthreads();
    const double goal = (double)u * s_total, before = s_before;
    const int at = s_c, end = s_end;
    __syncthreads();
    if (end < 0) return -1;
    int v = -1;
    // a running sum can fall short of the chunk's by its last bits: then the
    // token is the chunk's last one with weight
    if (at >= 0) v = find_token<WIDE>(r, a.vocab, at * VERIFY_CHUNK, before, goal, false, red, s_v);
    if (v < 0) v = find_token<WIDE>(r, a.vocab, (at >= 0 ? at : end) * VERIFY_CHUNK, 0.0, 0.0, true, red, s_v);
    return v;
}

template <bool WIDE>
__global__ void __launch_bounds__(VT) verify_kernel(VerifyArgs a) {
    __shared__ double red[VW];
    __shared__ int s_v, s_last;
    __shared__ Verdict s_verdict;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, s = blockIdx.y, chunk = blockIdx.x;
    const int r0 = a.row_start[s], n = a.row_start[s + 1] - r0;
    const bool fine = r0 >= 0 && n >= 0 && r0 + n <= a.rows;
    if (!fine || n == 0) {
        if (chunk == 0 && tid == 0) {
            if (!fine) report(a.err, s);
            a.n_tokens[s] = 0;
            if (a.new_len) a.new_len[s] = a.kv_len[s];
        }
        return;
    }
    if (tid < 32) {
        const Verdict v = judge(a, r0, n, chunk == 0);
        if (tid == 0) s_verdict = v;
    }
    __syncthreads();
    const Verdict ve = s_verdict;
    Row row{a.p + (long long)(r0 + ve.a) * a.p_row, nullptr, -1};
    if (ve.draft >= 0) {
        if (a.q) row.q = a.q + (long long)(r0 + ve.a + 1) * a.q_row;
        else row.certain = ve.draft;
    }
    double* part = a.part + (long long)s * a.chunks;
    const double sum = chunk_sum<WIDE>(row, a.vocab, chunk * VERIFY_CHUNK, red);
    if (tid == 0) {
        __stcg(part + chunk, sum);
        __threadfence();
        s_last = atomicAdd(a.tickets + s, 1) == a.chunks - 1;
    }
    __syncthreads();
    if (!s_last) return;
    if (tid == 0) a.tickets[s] = 0;
    __threadfence();
    const float u = a.u[r0];
    int v = draw<WIDE>(a, row, part, u, red, &s_v);
    if (v < 0 && ve.draft >= 0) {
        // nothing is left of p behind q: p itself
        row.q = nullptr;
        row.certain = -1;
        for (int c = 0; c < a.chunks; ++c) {
            const double x = chunk_sum<WIDE>(row, a.vocab, c * VERIFY_CHUNK, red);
            if (tid == 0) __stcg(part + c, x);
        }
        __syncthreads();
        v = draw<WIDE>(a, row, part, u, red, &s_v);
    }
    const int out = ve.a + (v >= 0);
    for (int i = tid; i < n; i += VT) a.tokens[r0 + i] = i < ve.a ? a.ids[r0 + i + 1] : (i == ve.a ? v : -1);
    if (tid == 0) {
        a.n_tokens[s] = out;
        if (a.new_len) a.new_len[s] = a.kv_len[s] - (n - 1 - ve.a);
    }
}

}  // namespace

int launch_verify_drafts(const VerifyArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)a.chunks, (unsigned)a.S), block(VT);
    return (int)(a.wide ? launch_k(verify_kernel<true>, grid, block, 0, s, a)
                        : launch_k(verify_kernel<false>, grid, block, 0, s, a));
}

}  // namespace dfl
