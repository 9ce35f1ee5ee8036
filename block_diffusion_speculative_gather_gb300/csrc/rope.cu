// Rotary positions as an operator: y = scale * R(pos * f) x on the first
// rotary dimensions of each head, the others copied.
//
// Angles.  f / (2 pi) is kept as a 64-bit fraction of a turn, so pos * f
// modulo a whole turn is one integer multiply that wraps, without the 64-bit
// floating point this part has little of.  What is off is the table itself, by
// its fp64 arithmetic (about 2^-52 of a turn, so pos * 2^-52 turns), and the
// angle's rounding to fp32 (2^-28 turns).
//
// A warp takes one row and some of its heads; a lane keeps its pairs' cosines
// and sines in registers for all heads it visits.  Bound by the rows' bytes
// (read once, written once) at many rows and by latency at few, where a row's
// heads are spread over more warps.  16384 rows of 40 heads of 128, bf16, half of
// the head rotated: 60 us, 5.6 TB/s; 16 rows: 2.5 us.

#include "gemm.cuh"
#include "kv8.cuh"

namespace dfl {
namespace {

constexpr double TWO_PI = 6.283185307179586476925286766559;

__global__ void rope_turns_kernel(RopeTurnsArgs a) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.half) return;
    double f = pow(a.theta, -(double)i / (double)a.half);
    if (a.scaling == 1) {
        f /= a.factor;
    } else if (a.scaling == 2) {
        // by parts: pairs that turn often over the original length keep their
        // frequency, pairs that turn less than alpha times are stretched
        const double r = a.original_len * f / TWO_PI;
        double g = (r - a.alpha) / (a.beta - a.alpha);
        g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
        f = (1.0 - g) * f / a.factor + g * f;
    }
    double t = f / TWO_PI;
    t -= floor(t);
    // 2^64 t in two 32-bit steps (t < 1): the product with 2^32 is exact
    const double hi = floor(t * 4294967296.0);
    const double lo = rint((t * 4294967296.0 - hi) * 4294967296.0);
    a.turns[i] = ((unsigned long long)hi << 32) + (unsigned long long)lo;
}

// The turn is split exactly into a quarter and a remainder of at most an
// eighth of a turn, so the fp32 angle is off by 2^-28 turns or less and
// sincospif sees no large argument.
__device__ __forceinline__ void angle_of(unsigned long long turn, int pos, float scale, float* c, float* s) {
    const unsigned long long t = turn * (unsigned long long)(unsigned)pos;
    const unsigned q = (unsigned)((t + (1ull << 61)) >> 62);            // nearest quarter
    const long long r = (long long)(t - ((unsigned long long)q << 62)); // 2^-64 turns, |r| <= 2^61
    float sn, cs;
    sincospif((float)r * 0x1p-63f, &sn, &cs);
    const float a = (q & 1) ? -sn : cs, b = (q & 1) ? cs : sn;
    *c = ((q & 2) ? -a : a) * scale;
    *s = ((q & 2) ? -b : b) * scale;
}

template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// Two neighbouring elements rounded in one conversion.
__device__ __forceinline__ void put2(float* p, float a, float b) { p[0] = a; p[1] = b; }
__device__ __forceinline__ void put2(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void put2(__half* p, float a, float b) {
    *reinterpret_cast<__half2*>(p) = __floats2half2_rn(a, b);
}

// The heads of one tensor that this lane visits: first, then every step-th.
// V elements at i0 (and, halves, at i1) of each head; HB heads' loads are in
// flight together, the first before `angles` finds the cosines and sines.
// (16384 rows of 40 heads: HB 1, 2, 4: 72, 60, 61 us.)
template <typename T, int V, bool IL, int P, typename A>
__device__ __forceinline__ void rotate_heads(const RopeHeads& t, long long row, int first, int step, int i0, int i1,
                                             bool rot, const float (&c)[P], const float (&s)[P], A angles) {
    constexpr int HB = V > 1 ? 2 : 1;
    const T* x = reinterpret_cast<const T*>(t.x) + row * t.x_row + first * t.x_head + i0;
    T* y = reinterpret_cast<T*>(t.out) + row * t.out_row + first * t.out_head + i0;
    const long long xs = step * t.x_head, ys = step * t.out_head;
    const int d = i1 - i0;
    Vec<T, V> e[HB], f[HB];
    auto load = [&](int h) {
#pragma unroll
        for (int b = 0; b < HB; ++b) {
            if (h + b * step >= t.heads) break;
            e[b] = *reinterpret_cast<const Vec<T, V>*>(x + b * xs);
            if (rot && !(IL && V > 1)) f[b] = *reinterpret_cast<const Vec<T, V>*>(x + b * xs + d);
        }
    };
    load(first);
    angles();
    for (int h = first; h < t.heads; h += HB * step) {
        if (h > first) load(h);
#pragma unroll
        for (int b = 0; b < HB; ++b) {
            if (h + b * step >= t.heads) break;
            if (rot) {
                if (V == 1) {
                    const float p = to_f32(e[b].v[0]), q = to_f32(f[b].v[0]);
                    y[b * ys + d] = from_f32<T>(q * c[0] + p * s[0]);
                    e[b].v[0] = from_f32<T>(p * c[0] - q * s[0]);
                } else if (IL) {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        const float p = to_f32(e[b].v[2 * j]), q = to_f32(e[b].v[2 * j + 1]);
                        put2(e[b].v + 2 * j, p * c[j] - q * s[j], q * c[j] + p * s[j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float p0 = to_f32(e[b].v[j]), q0 = to_f32(f[b].v[j]);
                        const float p1 = to_f32(e[b].v[j + 1]), q1 = to_f32(f[b].v[j + 1]);
                        put2(e[b].v + j, p0 * c[j] - q0 * s[j], p1 * c[j + 1] - q1 * s[j + 1]);
                        put2(f[b].v + j, q0 * c[j] + p0 * s[j], q1 * c[j + 1] + p1 * s[j + 1]);
                    }
                    *reinterpret_cast<Vec<T, V>*>(y + b * ys + d) = f[b];
                }
            }
            *reinterpret_cast<Vec<T, V>*>(y + b * ys) = e[b];
        }
        x += HB * xs;
        y += HB * ys;
    }
}

// V elements (16 bytes, or one element where alignment or the dims forbid
// more) are a unit.  Half layout: a rotary unit is V elements of the first
// half and the V elements rotary/2 behind them.  Interleaved: V elements,
// V/2 pairs (one pair of single elements when V is 1).
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(64) rope_kernel(RopeArgs a, int splits, int units, int rot_units,
                                                  int per_iter) {
    constexpr int P = IL ? (V > 1 ? V / 2 : 1) : V;   // pairs of a rotary unit
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long row = w / splits;
    const int part = (int)(w % splits);
    if (row >= a.rows) return;
    const int pos = a.positions[row];
    if (pos < 0) return;    // padding: the row stays as it was
    const int sub = units <= 32 ? lane / units : 0;   // which head of an iteration
    if (sub >= per_iter) return;
    const int step = splits * per_iter, first = part * per_iter + sub;
    // heads are dealt over both tensors in a row: the second goes on where the first ends
    int second = first - a.t[0].heads;
    if (second < 0) second = (second % step + step) % step;
    for (int u = units <= 32 ? lane % units : lane; u < units; u += 32) {
        const bool rot = u < rot_units;
        int i0, i1 = 0;          // element offsets in the head
        float c[P], s[P];
        const int p0 = u * P;
        if (rot) {
            i0 = IL ? 2 * p0 : p0;
            i1 = IL ? i0 + 1 : p0 + (a.rotary >> 1);
        } else {
            i0 = a.rotary + (u - rot_units) * V;
        }
        rotate_heads<T, V, IL, P>(a.t[0], row, first, step, i0, i1, rot, c, s, [&] {
            if (rot) {
#pragma unroll
                for (int j = 0; j < P; ++j) angle_of(a.turns[p0 + j], pos, a.scale, &c[j], &s[j]);
            }
        });
        rotate_heads<T, V, IL, P>(a.t[1], row, second, step, i0, i1, rot, c, s, [] {});
    }
}

template <typename T, int V, bool IL>
int launch_rope_t(const RopeArgs& a, cudaStream_t s) {
    const int per = IL ? (V > 1 ? V : 2) : 2 * V;   // elements of a rotary unit
    const int rot_units = a.rotary / per, units = rot_units + (a.head_dim - a.rotary) / V;
    const int per_iter = units <= 32 ? 32 / units : 1;
    const int heads = a.t[0].heads + a.t[1].heads;
    // warps of a row: one while there are rows enough to fill the device
    // (2048 warps), else as many as leave each one step over the heads
    int splits = (heads + per_iter - 1) / per_iter;
    const long long want = (2048 + a.rows - 1) / a.rows;
    if (splits > want) splits = (int)want;
    const long long warps = (long long)a.rows * splits;
    // small CTAs: few warps spread over the SMs, and many leave little of an SM
    // empty (16384 rows of 40 heads: 256 threads 66 us, 128 61 us, 64 60 us)
    constexpr int tpb = 64;
    const long long blocks = (warps * 32 + tpb - 1) / tpb;
    return (int)launch_k(rope_kernel<T, V, IL>, dim3((unsigned)blocks), dim3(tpb), 0, s, a, splits, units,
                         rot_units, per_iter);
}

template <typename T>
int launch_rope_d(const RopeArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (a.wide) return a.interleaved ? launch_rope_t<T, V, true>(a, s) : launch_rope_t<T, V, false>(a, s);
    return a.interleaved ? launch_rope_t<T, 1, true>(a, s) : launch_rope_t<T, 1, false>(a, s);
}

}  // namespace

int launch_rope_turns(const RopeTurnsArgs& a, cudaStream_t s) {
    return (int)launch_k(rope_turns_kernel, dim3((a.half + 127) / 128), dim3(128), 0, s, a);
}

int launch_rope(const RopeArgs& a, cudaStream_t s) {
    if (a.dtype == 0) return launch_rope_d<float>(a, s);
    if (a.dtype == 1) return launch_rope_d<__nv_bfloat16>(a, s);
    return launch_rope_d<__half>(a, s);
}

}  // namespace dfl
