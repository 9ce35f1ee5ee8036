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
// as pairs of fp32 numbers, in a fixed order.  The k-th addition of a chain leaves up
// to 2^-24 of the sum to the low part, which then holds up to k 2^-24 of it and is
// rounded by k 2^-48: n additions are off by at most n (n + 3) / 2 of 2^-48, a lane's 32 of
// a unit by 2^-38.8.  With the joins of lanes, units (one a thread up to 262144 tokens,
// else up to 64) and warps, and the search in the unit, a running sum is within 2^-36
// of the whole up to 262144 tokens and 2^-34 at 2^24, if all roundings are at their
// largest and go one way.  A uniform number's own step is 2^-24.
//
// Only one row of p and q is read whole.  Its tokens are dealt in units of 1024 to
// warps (each CTA finds by itself, from two numbers a draft, which row that is),
// a unit's sum goes to memory, and the last of a sequence's CTAs finds the unit
// that u_0 falls into and reads it again.  No CTA waits for another.
//
// With 151936 tokens and 16 rows a sequence one takes 7.1 us, a chain of trips to
// memory: row starts, ids, p and q of the drafts, the row, the ticket, the sums, the unit.
// 32 take 14.5 us for 38.9 MB, the same chain around the reads (11.5 from L2); 480 rows
// without drafts 57 us, 5.1 TB/s, where a pair's additions (7 instructions a token) and
// the chain at each CTA's end stand beside the reads.

#include "sampling.cuh"

namespace dfl {
namespace {

constexpr int VT = 256;                        // threads
constexpr int VW = VT / 32;
// Tokens of a lane and of a warp at a time: as many again are on their way, 2 KB a warp
// with q or without.
template <bool Q> constexpr int per() { return Q ? 8 : 16; }
template <bool Q> constexpr int block() { return 32 * per<Q>(); }
static_assert(VERIFY_UNIT == 4 * VT && VERIFY_UNIT % block<false>() == 0, "four tokens a thread of the search");

// A sum as hi + lo: the rounded sum, and what its roundings have left over.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair add(Pair a, float x, float e) {
    const float s = __fadd_rn(a.hi, x), b = __fsub_rn(s, a.hi);
    const float err = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, b)), __fsub_rn(x, b));
    return {s, __fadd_rn(a.lo, __fadd_rn(err, e))};
}

__device__ __forceinline__ Pair plus(Pair a, Pair b) { return add(a, b.hi, b.lo); }
// The sign of the difference is the rounded one's: where the high parts are close
// theirs is exact.
__device__ __forceinline__ bool above(Pair a, Pair b) { return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) > 0.f; }
__device__ __forceinline__ Pair shfl(Pair a, int from) {
    return {__shfl_sync(0xffffffffu, a.hi, from), __shfl_sync(0xffffffffu, a.lo, from)};
}
// Sums over this and the lower lanes of the warp.
__device__ __forceinline__ Pair warp_running(Pair a, int lanes = 32) {
    const int lane = threadIdx.x & 31;
    for (int o = 1; o < lanes; o <<= 1) {
        const Pair b{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
        if (lane >= o) a = plus(b, a);
    }
    return a;
}

// The same in all lanes: a sum's rounding error does not depend on the operands' order.
__device__ __forceinline__ Pair warp_total(Pair a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, a.hi, o), lo = __fadd_rn(a.lo, __shfl_xor_sync(0xffffffffu, a.lo, o));
        a = add(Pair{a.hi, lo}, hi, 0.f);
    }
    return a;
}

// What counts of a probability: negative and NaN ones are 0, and those of 2^100 or
// more, so that no sum leaves fp32.
__device__ __forceinline__ float clean(float p) { return p > 0.f && p < 0x1p100f ? p : 0.f; }

// Weight of a token: p - q where that is positive, exactly.
__device__ __forceinline__ Pair less(float p, float q) {
    const float d = __fsub_rn(p, q), b = __fsub_rn(d, p);
    const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
    return p > q ? Pair{d, e} : Pair{0.f, 0.f};
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

// Four tokens from v on (v < vocab); those behind the vocabulary are 0.
template <bool WIDE>
__device__ __forceinline__ void load4(const float* row, int vocab, int v, float* x) {
    if (WIDE) {                                 // vocab is a multiple of 4
        const float4 f = *reinterpret_cast<const float4*>(row + v);
        x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = v + j < vocab ? row[v + j] : 0.f;
    }
}

template <bool Q> struct Tokens {
    float p[per<Q>()], q[Q ? per<Q>() : 1];
};

// A warp's tokens from v0 on.
template <bool WIDE, bool Q>
__device__ __forceinline__ void load_block(const Row& r, int vocab, int v0, Tokens<Q>& t) {
#pragma unroll
    for (int k = 0; k < per<Q>(); k += 4) {
        const int v = v0 + k * 32 + (threadIdx.x & 31) * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            t.p[k + j] = 0.f;
            if (Q) t.q[k + j] = 0.f;
        }
        if (v < vocab) {
            load4<WIDE>(r.p, vocab, v, t.p + k);
            if (Q && r.q) load4<WIDE>(r.q, vocab, v, t.q + k);
        }
    }
}

// CLEAN false: numbers of 2^100 and more are left in; a sum below it holds none.
template <bool Q, bool CLEAN>
__device__ __forceinline__ Pair add_block(const Row& r, int v0, const Tokens<Q>& t, Pair s) {
    const int mine = r.certain - v0 - (threadIdx.x & 31) * 4;      // where the refused token is the lane's
#pragma unroll
    for (int k = 0; k < per<Q>(); ++k) {
        float p = CLEAN ? clean(t.p[k]) : fmaxf(t.p[k], 0.f);      // fmaxf: NaN is 0
        if constexpr (Q) {
            const Pair w = less(p, clean(t.q[k]));
            s = add(s, w.hi, w.lo);
        } else {
            if (r.certain >= 0 && mine == (k / 4) * 128 + k % 4) p = 0.f;
            s = add(s, p, 0.f);
        }
    }
    return s;
}

// By a warp: the sum of a unit's weights, read anew.
template <bool WIDE, bool Q>
__device__ __noinline__ Pair sum_unit(const Row& r, int vocab, int unit) {
    Pair s{0.f, 0.f};
    for (int v0 = unit * VERIFY_UNIT; v0 < min((unit + 1) * VERIFY_UNIT, vocab); v0 += block<Q>()) {
        Tokens<Q> t;
        load_block<WIDE, Q>(r, vocab, v0, t);
        s = add_block<Q, true>(r, v0, t, s);
    }
    return warp_total(s);
}

// By a warp: sums of units `unit`, unit + step, .. into part.  The next tokens are
// on their way while these are summed.
template <bool WIDE, bool Q>
__device__ __forceinline__ void sum_units(const VerifyArgs& a, const Row& r, int unit, int step, float2* part) {
    Tokens<Q> t;
    constexpr int BLOCK = block<Q>();
    if (unit < a.units) load_block<WIDE, Q>(r, a.vocab, unit * VERIFY_UNIT, t);
    for (; unit < a.units; unit += step) {
        Pair s{0.f, 0.f};
#pragma unroll
        for (int b = 0; b < VERIFY_UNIT / BLOCK; ++b) {
            const Tokens<Q> now = t;
            const int v0 = unit * VERIFY_UNIT + b * BLOCK;
            if (b + 1 < VERIFY_UNIT / BLOCK) load_block<WIDE, Q>(r, a.vocab, v0 + BLOCK, t);
            else if (unit + step < a.units) load_block<WIDE, Q>(r, a.vocab, (unit + step) * VERIFY_UNIT, t);
            s = add_block<Q, Q>(r, v0, now, s);
        }
        s = warp_total(s);
        if (!Q && !(s.hi < 0x1p100f)) {
            const Row copy = r;      // what a call names lies in memory
            s = sum_unit<WIDE, Q>(copy, a.vocab, unit);
        }
        if ((threadIdx.x & 31) == 0) __stcg(part + unit, make_float2(s.hi, s.lo));
    }
}

__device__ __forceinline__ Pair unit_sum(const float2* p) {
    const float2 s = __ldcg(p);
    return {s.x, s.y};
}

// Sums before each thread of the CTA, and the total.
__device__ __forceinline__ Pair block_before(Pair v, Pair* total, float2* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Pair run = warp_running(v);
    if (lane == 31) red[warp] = make_float2(run.hi, run.lo);
    __syncthreads();
    const float2 w = red[lane % VW];
    const Pair warps = warp_running(Pair{w.x, w.y}, VW);      // its first VW lanes
    *total = shfl(warps, VW - 1);
    const Pair lower = shfl(warps, warp ? warp - 1 : 0);
    Pair up{__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
    if (lane == 0) up = {0.f, 0.f};
    return warp ? plus(lower, up) : up;
}

struct Search {
    float2 red[2][VW];
    Pair run;
    int thread, last, unit, token;
};

// By the whole CTA: the token that u draws from a row whose units' sums are
// `part`; -1: it has no weight.  In pairs of fp32 numbers throughout (fp64 sums
// took 6 us of a call).
template <bool WIDE, bool Q>
__device__ int draw(const VerifyArgs& a, const Row& r, const float2* part, float u, Search& sm) {
    const int tid = threadIdx.x;
    // each thread a run of units
    const int per = (a.units + VT - 1) / VT, b0 = tid * per, b1 = min(b0 + per, a.units);
    Pair own{0.f, 0.f};
    int end = -1;                      // last unit with weight
    for (int c = b0; c < b1; ++c) {
        const Pair x = unit_sum(part + c);
        own = plus(own, x);
        if (x.hi > 0.f) end = c;
    }
    if (tid == 0) sm.thread = 0x7fffffff, sm.last = -1;
    Pair total;
    const Pair before = block_before(own, &total, sm.red[0]);
    // u * total: the product of the high parts exactly, and the low one's
    const float prod = __fmul_rn(u, total.hi);
    const Pair goal{prod, fmaf(u, total.lo, fmaf(u, total.hi, -prod))};
    // the first run that passes the goal
    const bool past = end >= 0 && above(plus(before, own), goal);
    const unsigned m = __ballot_sync(0xffffffffu, past);
    const int top = __reduce_max_sync(0xffffffffu, end);
    if ((tid & 31) == 0) {
        if (m) atomicMin(&sm.thread, tid + __ffs(m) - 1);
        if (top >= 0) atomicMax(&sm.last, top);
    }
    __syncthreads();
    const int last = sm.last, thread = sm.thread;
    __syncthreads();
    if (last < 0) return -1;
    const bool none = thread == 0x7fffffff;          // u at or above 1, or NaN: the last token with weight
    if (tid == (none ? 0 : thread)) {
        // the run's first unit that passes it (by rounding maybe none: its last one with weight)
        int unit = none ? last : end;
        Pair run = none ? Pair{0.f, 0.f} : before;
        for (int c = b0; c < b1 && !none && b1 - b0 > 1; ++c) {
            const Pair x = unit_sum(part + c), next = plus(run, x);
            if (x.hi > 0.f && above(next, goal)) {
                unit = c;
                break;
            }
            if (c < end) run = next;
        }
        sm.unit = unit;
        sm.run = run;
        sm.token = 0x7fffffff;
        sm.last = -1;
    }
    __syncthreads();
    // the unit's tokens, four a thread
    const int v = sm.unit * VERIFY_UNIT + 4 * tid;
    float p[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
    if (v < a.vocab) {
        load4<WIDE>(r.p, a.vocab, v, p);
        if (Q && r.q) load4<WIDE>(r.q, a.vocab, v, q);
    }
    Pair w[4], s{0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = Q ? less(clean(p[j]), clean(q[j])) : Pair{v + j == r.certain ? 0.f : clean(p[j]), 0.f};
        s = plus(s, w[j]);
    }
    Pair run = plus(sm.run, block_before(s, &total, sm.red[1]));
    int hit = 0x7fffffff, any = -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        run = plus(run, w[j]);
        if (w[j].hi > 0.f) {
            any = v + j;
            if (!none && above(run, goal)) hit = min(hit, v + j);
        }
    }
    hit = (int)__reduce_min_sync(0xffffffffu, (unsigned)hit);
    any = __reduce_max_sync(0xffffffffu, any);
    if ((tid & 31) == 0) {
        if (hit != 0x7fffffff) atomicMin(&sm.token, hit);
        if (any >= 0) atomicMax(&sm.last, any);
    }
    __syncthreads();
    const int token = sm.token != 0x7fffffff ? sm.token : sm.last;
    __syncthreads();
    return token;
}

template <bool WIDE, bool Q>
__global__ void __launch_bounds__(VT, 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Search s_search;
    __shared__ int s_last;
    __shared__ Verdict s_verdict;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, s = blockIdx.y;
    const int r0 = a.row_start[s], r1 = a.row_start[s + 1];
    const bool fine = r0 >= 0 && r1 >= r0 && r1 <= a.rows;
    const int n = fine ? r1 - r0 : 0;
    if (n == 0) {
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
    float u = a.u[r0];
    u = u < 0.f ? -1.f : (u < 1.f ? u : 2.f);      // outside [0, 1), and NaN: the ends
    int v = draw<WIDE, Q>(a, row, part, u, s_search);
    if (v < 0 && ve.draft >= 0) {
        // nothing is left of p behind q: p itself
        row.q = nullptr;
        row.certain = -1;
        sum_units<WIDE, Q>(a, row, warp, VW, part);
        __threadfence();
        __syncthreads();
        v = draw<WIDE, Q>(a, row, part, u, s_search);
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
    // a unit a warp while all CTAs run at once (four an SM), else as many CTAs a sequence as
    // do; many sequences: about four rounds of them, so that the last one is short (151936
    // tokens: 100 sequences 17.4 us, with a unit a warp 19.4; 480 in four rounds 57, in one
    // 64, with a unit a warp 65)
    const int most = (a.units + VW - 1) / VW;
    const long long room = 4LL * sms;
    long long x = most;
    if (x * a.S > room) x = a.S <= room / 2 ? room / a.S : (4 * room + a.S - 1) / a.S;
    if (x > most) x = most;
    const dim3 grid((unsigned)x, (unsigned)a.S), block(VT);
    if (a.q)
        return (int)(a.wide ? launch_k(verify_kernel<true, true>, grid, block, 0, s, a)
                            : launch_k(verify_kernel<false, true>, grid, block, 0, s, a));
    return (int)(a.wide ? launch_k(verify_kernel<true, false>, grid, block, 0, s, a)
                        : launch_k(verify_kernel<false, false>, grid, block, 0, s, a));
}

}  // namespace dfl
