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
// Only one row of p and q is read whole.  Its tokens are dealt in units of 512 to
// warps (each CTA finds by itself, from two numbers a draft, which row that is),
// a unit's sum goes to memory, and the last of a sequence's CTAs finds the unit
// that u_0 falls into and reads it again.  No CTA waits for another.

#include "sampling.cuh"

namespace dfl {
namespace {

constexpr int VT = 256;                        // threads
constexpr int VW = VT / 32;
constexpr int PER = VERIFY_UNIT / 32;          // tokens of a lane

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

// The lane's k-th token of a unit: in order of k / 4, then of lanes, then of k.
__device__ __forceinline__ int token_of(int unit, int k) {
    return unit * VERIFY_UNIT + (k / 4) * 128 + (threadIdx.x & 31) * 4 + k % 4;
}

struct Tokens {
    float p[PER], q[PER];
};

template <bool WIDE, bool Q>
__device__ __forceinline__ void load_unit(const Row& r, int vocab, int unit, Tokens& t) {
    if (WIDE) {
#pragma unroll
        for (int k = 0; k < PER; k += 4) {
            const int v = token_of(unit, k);
            const bool in = v < vocab;          // vocab is a multiple of 4
            const float4 x = in ? *reinterpret_cast<const float4*>(r.p + v) : make_float4(0.f, 0.f, 0.f, 0.f);
            t.p[k] = x.x, t.p[k + 1] = x.y, t.p[k + 2] = x.z, t.p[k + 3] = x.w;
            if (!Q) continue;
            const float4 y = in && r.q ? *reinterpret_cast<const float4*>(r.q + v) : make_float4(0.f, 0.f, 0.f, 0.f);
            t.q[k] = y.x, t.q[k + 1] = y.y, t.q[k + 2] = y.z, t.q[k + 3] = y.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int v = token_of(unit, k);
            t.p[k] = v < vocab ? r.p[v] : 0.f;
            if (Q) t.q[k] = v < vocab && r.q ? r.q[v] : 0.f;
        }
    }
}

// Weights of the tokens, and their sum over the warp (the same in all lanes).
template <bool Q>
__device__ __forceinline__ Pair weigh_unit(const Row& r, int unit, const Tokens& t, Pair (&w)[PER]) {
    Pair s{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (Q) w[k] = weight(t.p[k], t.q[k]);
        else w[k] = {token_of(unit, k) == r.certain ? 0.f : clean(t.p[k]), 0.f};
        s = add(s, w[k].hi, w[k].lo);
    }
    return warp_total(s);
}

// By a warp: sums of units `unit`, unit + step, .. into part.  The next unit is on
// its way while one is summed.
template <bool WIDE, bool Q>
__device__ __forceinline__ void sum_units(const VerifyArgs& a, const Row& r, int unit, int step, float2* part) {
    Tokens t;
    if (unit < a.units) load_unit<WIDE, Q>(r, a.vocab, unit, t);
    for (; unit < a.units; unit += step) {
        const Tokens now = t;
        if (unit + step < a.units) load_unit<WIDE, Q>(r, a.vocab, unit + step, t);
        Pair w[PER];
        const Pair s = weigh_unit<Q>(r, unit, now, w);
        if ((threadIdx.x & 31) == 0) __stcg(part + unit, make_float2(s.hi, s.lo));
    }
}

// By a warp: the first token of the unit whose running sum, from `before` on,
// passes `goal`, else its last token with weight (a running sum can fall short of
// the unit's by its last bits); -1: it has none.
template <bool WIDE, bool Q>
__device__ int find_token(const VerifyArgs& a, const Row& r, int unit, double before, double goal) {
    const int lane = threadIdx.x & 31;
    constexpr int STEP = 4;        // tokens of a lane that stand together
    Tokens t;
    Pair w[PER];
    load_unit<WIDE, Q>(r, a.vocab, unit, t);
    weigh_unit<Q>(r, unit, t, w);
    // sums before each of the lane's groups: PER / STEP scans side by side
    double own[PER / STEP], inc[PER / STEP];
#pragma unroll
    for (int k = 0; k < PER / STEP; ++k) {
        Pair x{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < STEP; ++j) x = add(x, w[STEP * k + j].hi, w[STEP * k + j].lo);
        own[k] = inc[k] = value(x);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < PER / STEP; ++k) {
            const double x = __shfl_up_sync(0xffffffffu, inc[k], o);
            if (lane >= o) inc[k] += x;
        }
    int first = 0x7fffffff, last = -1;
#pragma unroll
    for (int k = 0; k < PER / STEP; ++k) {
        double run = before + (inc[k] - own[k]);
        before += __shfl_sync(0xffffffffu, inc[k], 31);
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
            run += value(w[STEP * k + j]);
            if (w[STEP * k + j].hi > 0.f) {
                const int v = token_of(unit, STEP * k + j);
                last = max(last, v);
                if (run > goal) first = min(first, v);
            }
        }
    }
    first = (int)__reduce_min_sync(0xffffffffu, (unsigned)first);
    last = __reduce_max_sync(0xffffffffu, last);
    return first != 0x7fffffff ? first : last;
}

__device__ __forceinline__ double unit_sum(const float2* p) {
    const float2 s = __ldcg(p);
    return value(Pair{s.x, s.y});
}

// By the whole CTA: the token that u draws from a row whose units' sums are
// `part`; -1: it has no weight.
template <bool WIDE, bool Q>
__device__ int draw(const VerifyArgs& a, const Row& r, const float2* part, float u, double* red, int* s_v) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // each thread a run of units
    const int per = (a.units + VT - 1) / VT, b0 = tid * per, b1 = min(b0 + per, a.units);
    double own = 0.0;
    int end = -1;                      // last unit with weight
    for (int c = b0; c < b1; ++c) {
        const double x = unit_sum(part + c);
        own += x;
        if (x > 0.0) end = c;
    }
    double inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) red[warp] = inc;
    if (tid == 0) s_v[0] = 0x7fffffff, s_v[1] = -1;
    __syncthreads();
    double total = 0.0, before = 0.0;
#pragma unroll
    for (int i = 0; i < VW; ++i) {
        if (i < warp) before += red[i];
        total += red[i];
    }
    const double goal = (double)u * total;
    before += inc - own;
    // the first run that passes the goal, and in it the first unit
    if (end >= 0) {
        atomicMax(s_v + 1, end);
        if (before + own > goal) atomicMin(s_v, tid);
    }
    __syncthreads();
    const int at = s_v[0], last = s_v[1];
    __syncthreads();
    if (last < 0) return -1;
    if (at == 0x7fffffff ? warp == 0 : warp == at / 32) {
        int unit = last;
        double run = 0.0, g = INFINITY;            // past the goal: the last token with weight
        if (at != 0x7fffffff) {
            unit = end;
            run = before;
            g = goal;
            for (int c = b0; c < b1; ++c) {        // in the lane whose run it is
                const double x = unit_sum(part + c);
                if (x > 0.0) {
                    unit = c;
                    if (run + x > goal) break;
                    if (c < end) run += x;
                }
            }
            unit = __shfl_sync(0xffffffffu, unit, at % 32);
            run = __shfl_sync(0xffffffffu, run, at % 32);
        }
        const int v = find_token<WIDE, Q>(a, r, unit, run, g);
        if (lane == 0) s_v[0] = v;
    }
    __syncthreads();
    const int v = s_v[0];
    __syncthreads();
    return v;
}

template <bool WIDE, bool Q>
__global__ void __launch_bounds__(VT, Q ? 3 : 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ double red[VW];
    __shared__ int s_v[2], s_last;
    __shared__ Verdict s_verdict;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, s = blockIdx.y;
    const int r0 = a.row_start[s], n = a.row_start[s + 1] - r0;
    const bool fine = r0 >= 0 && n >= 0 && r0 + n <= a.rows;
    if (!fine || n == 0) {
        if (blockIdx.x == 0 && tid == 0) {
            if (!fine) report(a.err, s);
            a.n_tokens[s] = 0;
            if (a.new_len) a.new_len[s] = a.kv_len[s];
        }
        return;
    }
    Verdict ve{0, -1};
    if (n > 1) {
        if (tid < 32) {
            const Verdict v = judge(a, r0, n, blockIdx.x == 0);
            if (tid == 0) s_verdict = v;
        }
        __syncthreads();
        ve = s_verdict;
    }
    Row row{a.p + (long long)(r0 + ve.a) * a.p_row, nullptr, -1};
    if (ve.draft >= 0) {
        if (Q) row.q = a.q + (long long)(r0 + ve.a + 1) * a.q_row;
        else row.certain = ve.draft;
    }
    float2* part = a.part + (long long)s * a.units;
    sum_units<WIDE, Q>(a, row, blockIdx.x * VW + warp, gridDim.x * VW, part);
    __threadfence();
    __syncthreads();
    if (gridDim.x > 1) {
        if (tid == 0) s_last = atomicAdd(a.tickets + s, 1) == (int)gridDim.x - 1;
        __syncthreads();
        if (!s_last) return;
        if (tid == 0) a.tickets[s] = 0;
        __threadfence();
    }
    const float u = a.u[r0];
    int v = draw<WIDE, Q>(a, row, part, u, red, s_v);
    if (v < 0 && ve.draft >= 0) {
        // nothing is left of p behind q: p itself
        row.q = nullptr;
        row.certain = -1;
        sum_units<WIDE, Q>(a, row, warp, VW, part);
        __threadfence();
        __syncthreads();
        v = draw<WIDE, Q>(a, row, part, u, red, s_v);
    }
    const int out = ve.a + (v >= 0);
    for (int i = tid; i < n; i += VT) a.tokens[r0 + i] = i < ve.a ? a.ids[r0 + i + 1] : (i == ve.a ? v : -1);
    if (tid == 0) {
        a.n_tokens[s] = out;
        if (a.new_len) a.new_len[s] = a.kv_len[s] - (n - 1 - ve.a);
    }
}

}  // namespace

int launch_verify_drafts(const VerifyArgs& a, int sms, cudaStream_t s) {
    // a unit a warp while they are few, up to four in a row where there are many:
    // CTAs come and go less often
    int x = (a.units + VW - 1) / VW;
    const long long all = (long long)x * a.S, room = 8LL * sms;
    const int each = all >= 4 * room ? 4 : (all >= 2 * room ? 2 : 1);
    x = (x + each - 1) / each;
    const dim3 grid((unsigned)x, (unsigned)a.S), block(VT);
    if (a.q)
        return (int)(a.wide ? launch_k(verify_kernel<true, true>, grid, block, 0, s, a)
                            : launch_k(verify_kernel<false, true>, grid, block, 0, s, a));
    return (int)(a.wide ? launch_k(verify_kernel<true, false>, grid, block, 0, s, a)
                        : launch_k(verify_kernel<false, false>, grid, block, 0, s, a));
}

}  // namespace dfl
