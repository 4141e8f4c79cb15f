// Rotary positions with three axes (t, y, x): the rotation itself and rope_apply_kernel, which rotates token tensors
// while it moves them between layouts (a projection's token-major output and the head-major padded layout the attention
// kernels read).
//
// A token at (t, y, x) turns pair i of an axis of m dimensions by pos * theta^(-2i/m). Angles are kept in turns as 64-bit
// fixed-point fractions: the host rounds theta^(-2i/m) / 2 pi to a multiple of 2^-64, and pos * step wraps modulo one
// turn by itself, so the reduction of a far position's angle is one exact integer product (the error is pos times
// the step's, see rope_args). The nearest quarter turn is split off, and the rest, at most an eighth of a turn, goes through
// sincospif.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "ptx.cuh"

namespace losa {

constexpr int kRopeMaxPairs = 128;  // head_dim <= 256

// The rotation of one call: pairs 0 .. end[2] - 1 in axis order, each axis's first pair and dimension.
struct RopeArgs {
    uint64_t step[kRopeMaxPairs];  // turns * 2^64 per unit of position
    int end[3];                    // first dimension behind each axis's section
    int half[3];                   // pairs of each axis
    int gy, gx;                    // the token grid
    int off[3];                    // added to (t, y, x)
};

struct RopePos {
    int p[3];
};

// The quotient rounded down; y > 0.
__device__ __forceinline__ int floor_div(int x, int y) {
    const int q = x / y;
    return q - (x - q * y < 0 ? 1 : 0);
}

// Position of token n of the grid (negative: before its first), or the caller's (t, y, x) triple.
__device__ __forceinline__ RopePos rope_position(const RopeArgs& r, const int32_t* triple, int n) {
    RopePos q;
    if (triple) {
        q.p[0] = triple[0];
        q.p[1] = triple[1];
        q.p[2] = triple[2];
    } else {
        const int row = floor_div(n, r.gx), t = floor_div(row, r.gy);
        q.p[0] = t;
        q.p[1] = row - t * r.gy;
        q.p[2] = n - row * r.gx;
    }
    q.p[0] += r.off[0];
    q.p[1] += r.off[1];
    q.p[2] += r.off[2];
    return q;
}

// cos and sin of pair `pair` (an index into step) at position pos.
__device__ __forceinline__ float2 rope_angle(uint64_t step, int pos) {
    const uint64_t turns = step * (uint64_t)(int64_t)pos;
    const uint32_t h = (uint32_t)((turns + 0x80000000ull) >> 32);
    const uint32_t quarter = (h + 0x20000000u) >> 30;             // nearest quarter turn
    const float x = (float)(int32_t)(h - (quarter << 30)) * 4.656612873077393e-10f;  // half turns, |x| <= 1/4
    float s, c;
    sincospif(x, &s, &c);
    const bool swap = quarter & 1u;
    const float cs = swap ? s : c, sn = swap ? c : s;
    return make_float2((quarter == 1u || quarter == 2u) ? -cs : cs, (quarter & 2u) ? -sn : sn);
}

// cos and sin of the pair whose first dimension (in axis order: twice its index) is e; (1, 0) behind the rotated ones.
__device__ __forceinline__ float2 rope_pair(const RopeArgs& r, const RopePos& q, int e) {
    if (e >= r.end[2]) return make_float2(1.0f, 0.0f);
    return rope_angle(r.step[e >> 1], e < r.end[0] ? q.p[0] : (e < r.end[1] ? q.p[1] : q.p[2]));
}

// How a row falls into units of work. Interleaved pairing (W = 0): 16 bytes of consecutive dimensions, pairs inside. Halves
// pairing: W consecutive dimensions of the first half of an axis's section and the W they are paired with; W is the
// largest of 4, 2, 1 that divides every half, so that both sides are aligned for one load of W. (Reading partners one
// element at a time instead took 1229 us on the 24-head 118800-token gradient; this takes 447 us.) What is not rotated comes in units
// of 2 W consecutive dimensions, whose second W may be missing.
struct RopeUnit {
    int first, second;  // first dimension of each side; second < 0: none
    int pair;           // twice the index of the first pair
};
template <int W>
__device__ __forceinline__ RopeUnit rope_unit(const RopeArgs& r, int d, int u) {
    RopeUnit x;
    x.first = x.pair = 2 * W * u;
    x.second = x.first + W;
    if (x.first >= r.end[2]) {
        if (x.second >= d) x.second = -1;
        return x;
    }
    const int a = x.first < r.end[0] ? 0 : (x.first < r.end[1] ? 1 : 2);
    const int base = a == 0 ? 0 : r.end[a - 1];
    x.first = base + (x.first - base) / 2;
    x.second = x.first + r.half[a];
    return x;
}

// One side of a copy: strides in elements; dimension d is contiguous.
struct TokenView {
    int64_t part, batch, token, head;
};

struct RopeApplyArgs {
    RopeArgs r;
    TokenView xs, ys;
    const int32_t* positions;  // [batch][n][3] or null
    const int32_t* start;      // [batch] or null
    int parts, batch, heads;
    int n, n_out;              // tokens rotated; rows written (rows n .. n_out - 1 become zero)
    int d;
    int units;                 // units of a row
    int per_cta;               // (part, head) rows each CTA walks
    uint32_t rotate;           // bit p: part p is rotated (else copied)
    float sign;                // -1 for the inverse rotation
};

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 6;  // rows in flight per thread

// N elements in one load or store.
template <int BYTES> struct RawVec;
template <> struct RawVec<2> { typedef uint16_t type; };
template <> struct RawVec<4> { typedef uint32_t type; };
template <> struct RawVec<8> { typedef uint2 type; };
template <> struct RawVec<16> { typedef uint4 type; };
template <typename T, int N> struct Pack {
    typedef typename RawVec<N * sizeof(T)>::type Raw;
    Raw raw;
    __device__ __forceinline__ void load(const T* p) { raw = __ldcg(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = raw; }
    __device__ __forceinline__ float get(int i) const {
        return to_float(reinterpret_cast<const T*>(&raw)[i]);
    }
    __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<T*>(&raw)[i] = from_float(f[i]);
    }
    static __device__ __forceinline__ float to_float(float x) { return x; }
    static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ T from_float(float x) {
        if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(x);
        else return x;
    }
};

// Every row is read once and written once; nothing else moves, so the kernel is bound by memory. A thread owns one unit of
// one token and walks that token's (part, head) rows with the unit's cosines and sines in registers: the angles are computed
// once per token instead of once per row, which would cost more than the copy. Measured: a 480p projection (12 heads, query,
// key and value, 604 MB) in 102 us, 5.9 TB/s; the 720p gradient (24 heads, query and key, 2.9 GB) in 447 us, 6.5 TB/s, on two
// sets of tensors in turn, in 483 on three. Loads that mark their lines for early eviction cost 3 % of that, rows by two or
// eight at a time 4 to 8 %.
template <typename T, int W>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const __grid_constant__ RopeApplyArgs a,
                                                                  const T* __restrict__ x, T* __restrict__ y) {
    constexpr int N = W ? W : 16 / sizeof(T);  // elements of a load
    constexpr int SIDES = W ? 2 : 1;
    constexpr int PAIRS = W ? W : N / 2;
    const int64_t unit = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    const int n = (int)(unit / a.units);
    if (n >= a.n_out) return;
    const int u = (int)(unit - (int64_t)n * a.units);
    RopeUnit at;
    if (W) {
        at = rope_unit<W ? W : 1>(a.r, a.d, u);
    } else {
        at.first = at.pair = u * N;
        at.second = -1;
    }
    const int b = blockIdx.z;
    const int rows = a.parts * a.heads;
    const int lo = blockIdx.y * a.per_cta, hi = min(rows, lo + a.per_cta);
    T* const yt = y + b * a.ys.batch + n * a.ys.token;
    const bool real = n < a.n, two = SIDES == 2 && at.second >= 0;
    const T* const xt = x + b * a.xs.batch + (real ? n : 0) * a.xs.token;
    float c[PAIRS], s[PAIRS];
    if (real) {
        const int32_t* triple = a.positions ? a.positions + 3 * ((int64_t)b * a.n + n) : nullptr;
        const RopePos q = rope_position(a.r, triple, (a.start ? a.start[b] : 0) + n);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            const float2 cs = rope_pair(a.r, q, at.pair + 2 * e);
            c[e] = cs.x;
            s[e] = cs.y * a.sign;
        }
    }
    const int turned = a.r.end[2] - at.pair;  // dimensions of this unit that are rotated
    int p = lo / a.heads, h = lo - p * a.heads;
    for (int i0 = lo; i0 < hi; i0 += kRopeRows) {
        Pack<T, N> w[kRopeRows][SIDES];
        int64_t out[kRopeRows];
        bool turn[kRopeRows];
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            w[k][0].raw = {};
            if (SIDES == 2) w[k][SIDES - 1].raw = {};
            out[k] = -1;
            turn[k] = false;
            if (i0 + k >= hi) continue;
            out[k] = p * a.ys.part + h * a.ys.head;
            turn[k] = real && ((a.rotate >> p) & 1u);
            const T* const row = xt + p * a.xs.part + h * a.xs.head;
            if (real) w[k][0].load(row + at.first);
            if (real && two) w[k][SIDES - 1].load(row + at.second);
            if (++h == a.heads) {
                h = 0;
                ++p;
            }
        }
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            if (out[k] < 0) continue;
            if (turn[k] && turned > 0) {
                if constexpr (W > 0) {
                    float f[N], g[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float z0 = w[k][0].get(e), z1 = w[k][1].get(e);
                        f[e] = fmaf(-s[e], z1, c[e] * z0);
                        g[e] = fmaf(s[e], z0, c[e] * z1);
                    }
                    w[k][0].set(f);
                    w[k][1].set(g);
                } else {
                    float f[N];
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float z0 = w[k][0].get(e), z1 = w[k][0].get(e + 1);
                        const bool on = e < turned;  // an unrotated dimension must not meet its neighbour's infinity
                        f[e] = on ? fmaf(-s[e / 2], z1, c[e / 2] * z0) : z0;
                        f[e + 1] = on ? fmaf(s[e / 2], z0, c[e / 2] * z1) : z1;
                    }
                    w[k][0].set(f);
                }
            }
            T* const dst = yt + out[k];
            w[k][0].store(dst + at.first);
            if (two) w[k][SIDES - 1].store(dst + at.second);
        }
    }
}

}  // namespace losa
