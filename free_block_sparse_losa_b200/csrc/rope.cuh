// Rotary positions with three axes (t, y, x): the rotation itself and rope_apply_kernel, which rotates token tensors
// while it moves them between layouts (a projection's token-major output and the head-major padded layout the attention
// kernels read).
//
// A token at (t, y, x) turns pair i of an axis of m dimensions by pos * theta^(-2i/m). Angles are kept in turns as 64-bit
// fixed-point fractions: the host rounds theta^(-2i/m) / 2 pi to a multiple of 2^-64, and pos * step wraps modulo one
// turn by itself, so the reduction of a far position's angle is one exact integer product (the error is pos * 2^-65
// turns). The nearest quarter turn is split off, and the rest, at most an eighth of a turn, goes through sincospif.
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

// Position of token n of the grid, or the caller's (t, y, x) triple.
__device__ __forceinline__ RopePos rope_position(const RopeArgs& r, const int32_t* triple, int n) {
    RopePos q;
    if (triple) {
        q.p[0] = triple[0];
        q.p[1] = triple[1];
        q.p[2] = triple[2];
    } else {
        const int row = n / r.gx, t = row / r.gy;
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

// Cosine and signed sine by which dimension e of a rotated row is formed: y[e] = c * x[e] + s * x[partner]; partner
// returns the partner's dimension (e itself where the dimension is not rotated: c = 1, s = 0).
template <bool HALVES>
__device__ __forceinline__ float2 rope_dim(const RopeArgs& r, const RopePos& q, int e, int& partner) {
    partner = e;
    if (e >= r.end[2]) return make_float2(1.0f, 0.0f);
    const int a = e < r.end[0] ? 0 : (e < r.end[1] ? 1 : 2);
    const int base = a == 0 ? 0 : r.end[a - 1];
    const int l = e - base, h = r.half[a];
    bool first;
    int pair;
    if (HALVES) {
        first = l < h;
        pair = first ? l : l - h;
        partner = first ? e + h : e - h;
    } else {
        first = (l & 1) == 0;
        pair = l >> 1;
        partner = e ^ 1;  // sections start at even dimensions
    }
    const float2 cs = rope_angle(r.step[(base >> 1) + pair], a == 0 ? q.p[0] : (a == 1 ? q.p[1] : q.p[2]));
    return make_float2(cs.x, first ? -cs.y : cs.y);
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
    int chunks;                // 16-byte chunks of a row
    int per_cta;               // (part, head) rows each CTA walks
    uint32_t rotate;           // bit p: part p is rotated (else copied)
    float sign;                // -1 for the inverse rotation
};

template <typename T> struct RopeVec;
template <> struct RopeVec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <> struct RopeVec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
};

constexpr int kRopeThreads = 256;

// Every row is read once and written once; nothing else moves, so the kernel is bound by memory. A thread owns one
// 16-byte chunk of one token and walks that token's (part, head) rows with the chunk's cosines and sines in registers:
// the angles are computed once per token instead of once per row, which would cost more than the copy. With the halves
// pairing a dimension's partner lies half a section away, in general in another chunk at no aligned distance; the eight
// partners are read one by one from L1, where the row already is.
template <typename T, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const __grid_constant__ RopeApplyArgs a,
                                                                  const T* __restrict__ x, T* __restrict__ y) {
    constexpr int V = RopeVec<T>::kN;
    const int64_t unit = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    const int n = (int)(unit / a.chunks);
    if (n >= a.n_out) return;
    const int e0 = (int)(unit - (int64_t)n * a.chunks) * V;
    const int b = blockIdx.z;
    const int rows = a.parts * a.heads;
    const int lo = blockIdx.y * a.per_cta, hi = min(rows, lo + a.per_cta);
    T* const yt = y + b * a.ys.batch + n * a.ys.token + e0;
    if (n >= a.n) {
        for (int i = lo; i < hi; ++i) {
            const int p = i / a.heads, h = i - p * a.heads;
            *reinterpret_cast<uint4*>(yt + p * a.ys.part + h * a.ys.head) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const T* const xt = x + b * a.xs.batch + n * a.xs.token;
    float c[V], s[V];
    int partner[V];
    {
        const int32_t* triple = a.positions ? a.positions + 3 * ((int64_t)b * a.n + n) : nullptr;
        const RopePos q = rope_position(a.r, triple, (a.start ? a.start[b] : 0) + n);
#pragma unroll
        for (int e = 0; e < V; e += HALVES ? 1 : 2) {
            const float2 cs = rope_dim<HALVES>(a.r, q, e0 + e, partner[e]);
            c[e] = cs.x;
            s[e] = cs.y * a.sign;
            if (!HALVES) {  // the pair's second member
                c[e + 1] = cs.x;
                s[e + 1] = -s[e];
            }
        }
    }
    const int turned = a.r.end[2] - e0;  // dimensions of this chunk that are rotated
    constexpr int U = 4;  // rows in flight
    for (int i0 = lo; i0 < hi; i0 += U) {
        uint4 w[U];
        float z[HALVES ? U : 1][HALVES ? V : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= hi) continue;
            const int p = i / a.heads, h = i - p * a.heads;
            const T* const row = xt + p * a.xs.part + h * a.xs.head;
            w[u] = HALVES ? *reinterpret_cast<const uint4*>(row + e0)
                          : __ldcs(reinterpret_cast<const uint4*>(row + e0));
            if (HALVES && ((a.rotate >> p) & 1u)) {
#pragma unroll
                for (int e = 0; e < V; ++e) z[u][e] = RopeVec<T>::one(row + partner[e]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= hi) continue;
            const int p = i / a.heads, h = i - p * a.heads;
            if ((a.rotate >> p) & 1u) {
                float f[V], g[V];
                RopeVec<T>::unpack(w[u], f);
#pragma unroll
                for (int e = 0; e < V; ++e)  // an unrotated dimension must not meet its neighbour's infinity
                    g[e] = e < turned ? fmaf(s[e], HALVES ? z[u][e] : f[e ^ 1], c[e] * f[e]) : f[e];
                w[u] = RopeVec<T>::pack(g);
            }
            *reinterpret_cast<uint4*>(yt + p * a.ys.part + h * a.ys.head) = w[u];
        }
    }
}

}  // namespace losa
