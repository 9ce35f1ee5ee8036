// Rotary positions as an operator: y = scale * R(pos * f) x on the first
// rotary dimensions of each head, the others copied.
//
// Angles.  f / (2 pi) is kept as a 64-bit fraction of a turn, so pos * f
// modulo a whole turn is one integer multiply that wraps: exact to
// pos * 2^-65 turns at any position, without the 64-bit floating point this
// part has little of.
//
// A warp takes one row and some of its heads; a lane keeps its pairs' cosines
// and sines in registers for all heads it visits.  Bound by the rows' bytes
// (read once, written once) at many rows and by latency at few, where a row's
// heads are spread over more warps.

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
// eighth of a turn, so the fp32 angle is off by 2^-26 of it or less and
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

// V elements (16 bytes, or one element where alignment or the dims forbid
// more) are a unit.  Half layout: a rotary unit is V elements of the first
// half and the V elements rotary/2 behind them.  Interleaved: V elements,
// V/2 pairs (one pair of single elements when V is 1).
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a, int splits, int units, int rot_units,
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
    const int heads = a.t[0].heads + a.t[1].heads;
    const int half = a.rotary >> 1;
    const int sub = units <= 32 ? lane / units : 0;   // which head of an iteration
    if (sub >= per_iter) return;
    for (int u = units <= 32 ? lane % units : lane; u < units; u += 32) {
        const bool rot = u < rot_units;
        int i0, i1 = 0;          // element offsets in the head
        float c[P], s[P];
        if (rot) {
            const int p0 = u * P;
            i0 = IL ? 2 * p0 : p0;
            i1 = IL ? i0 + 1 : p0 + half;
#pragma unroll
            for (int j = 0; j < P; ++j) angle_of(a.turns[p0 + j], pos, a.scale, &c[j], &s[j]);
        } else {
            i0 = a.rotary + (u - rot_units) * V;
        }
        for (int h = part * per_iter + sub; h < heads; h += splits * per_iter) {
            const bool second = h >= a.t[0].heads;
            const RopeHeads& t = a.t[second ? 1 : 0];
            const int hh = second ? h - a.t[0].heads : h;
            const T* x = reinterpret_cast<const T*>(t.x) + row * t.x_row + hh * t.x_head;
            T* y = reinterpret_cast<T*>(t.out) + row * t.out_row + hh * t.out_head;
            if (!rot) {
                *reinterpret_cast<Vec<T, V>*>(y + i0) = *reinterpret_cast<const Vec<T, V>*>(x + i0);
            } else if (IL && V > 1) {
                Vec<T, V> e = *reinterpret_cast<const Vec<T, V>*>(x + i0);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float p = to_f32(e.v[2 * j]), q = to_f32(e.v[2 * j + 1]);
                    e.v[2 * j] = from_f32<T>(p * c[j] - q * s[j]);
                    e.v[2 * j + 1] = from_f32<T>(q * c[j] + p * s[j]);
                }
                *reinterpret_cast<Vec<T, V>*>(y + i0) = e;
            } else {
                Vec<T, V> e = *reinterpret_cast<const Vec<T, V>*>(x + i0);
                Vec<T, V> f = *reinterpret_cast<const Vec<T, V>*>(x + i1);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float p = to_f32(e.v[j]), q = to_f32(f.v[j]);
                    e.v[j] = from_f32<T>(p * c[j] - q * s[j]);
                    f.v[j] = from_f32<T>(q * c[j] + p * s[j]);
                }
                *reinterpret_cast<Vec<T, V>*>(y + i0) = e;
                *reinterpret_cast<Vec<T, V>*>(y + i1) = f;
            }
        }
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
    // few warps: small CTAs, so that they spread over the SMs
    const int tpb = warps >= 4096 ? 256 : 64;
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
