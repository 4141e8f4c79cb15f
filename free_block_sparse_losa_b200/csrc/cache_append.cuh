// Appending keys and values to the paged 8-bit cache, rotating the keys on the way: cache_append_kernel.
//
// The cache holds e4m3 codes in pages of C tokens, [page][kv head][C][d], with one fp32 scale per (page, kv head) for the
// keys and one for the values; a code stands for code * scale. A block's scale is the smallest power of two 2^e with
// max |x| <= 448 * 2^e over its tokens (e within [-40, 60]), or what the block already had if that is larger. With powers
// of two a scale that grows moves the held codes by an exact shift (only codes that become subnormal round again), so
// the result hardly depends on how the tokens were split into calls.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "rope.cuh"

namespace losa {

constexpr int kAppendThreads = 1024;
constexpr int kAppendDims = 16;  // dimensions of new rows that a thread holds
constexpr int kCacheExpMin = -40, kCacheExpMax = 60;

// A sequence's pages: the geometry every cache kernel shares.
struct CacheGeom {
    int kv_heads, page, n_pages;     // kv heads, tokens of a page, pages of the pool
    int table_stride;                // page-table entries of a sequence
    const int32_t* table;            // [seqs][table_stride]
    const int32_t* lens;             // [seqs]
};

struct AppendArgs {
    RopeArgs r;
    CacheGeom g;
    const int32_t* positions;  // [total][3] or null
    const int32_t* indptr;     // [seqs + 1] or null: new_tokens each
    int32_t* new_lens;         // may be null
    int64_t k_token, k_head, v_token, v_head;  // strides in elements
    int64_t total;             // rows of k and v
    int new_tokens;            // every sequence's count, or its upper bound
    int spans;                 // pages a sequence's new tokens can touch
    int heads_per_cta;
    int rotate;                // 0: keys are stored as they come
    uint8_t* code[2];          // keys, values
    float* scale[2];
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four values times s as codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, uint64_t s) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b64 x, y;\n\t.reg .f32 p, q, u, v;\n\t"
        "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
        "mul.rn.f32x2 x, x, %5;\n\tmul.rn.f32x2 y, y, %5;\n\t"
        "mov.b64 {p, q}, x;\n\tmov.b64 {u, v}, y;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, q, p;\n\tcvt.rn.satfinite.e4m3x2.f32 h, v, u;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d), "l"(s));
    return r;
}
// The largest magnitude of three (NaN is passed over).
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of_half2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

// 2^e for the smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), within the scales' range. amax's bits.
__device__ __forceinline__ float cache_scale(uint32_t amax_bits) {
    int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, kCacheExpMin), kCacheExpMax);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// One CTA takes the new tokens of one page, for the keys (blockIdx.z = 0) or the values, and walks a group of kv heads.
// K and V are read once and their codes written once, so the kernel is bound by memory. A thread holds the same 16
// dimensions of the page's rows for every head: their angles stay in registers, computed once (an angle per token and
// pair against six bytes of traffic per pair and head would cost more than the copy), and the values stay there between the
// maximum over the block and the rounding. The next head's values are fetched before this head's are used, so that the
// barrier of the maximum does not drain the memory pipe. A block of 1024 threads leaves 64 registers to each, of which every
// instance spills 24 to 104 bytes.
template <typename T, int D, int W>
__device__ __forceinline__ void append_page(const AppendArgs& a, const T* __restrict__ src, int64_t ts, int64_t hs,
                                            uint8_t* __restrict__ code, float* __restrict__ scale, bool keys) {
    constexpr int N = W ? W : 8;               // dimensions of a unit's side (see rope.cuh)
    constexpr int SIDES = W ? 2 : 1;
    constexpr int UNITS = D / (N * SIDES);     // of a row
    constexpr int P = kAppendDims / (N * SIDES);  // units of a thread
    constexpr int PAIRS = N * SIDES / 2;
    constexpr int LOADS = N * sizeof(T) / 16 > 1 ? N * sizeof(T) / 16 : 1;  // fp32, interleaved: two loads a side
    constexpr int LN = N / LOADS;
    __shared__ uint32_t part[2][kAppendThreads / 32];

    const int b = blockIdx.x / a.spans, span = blockIdx.x - b * a.spans;
    const int C = a.g.page;
    const int len = a.g.lens[b];
    int m = a.new_tokens;
    int64_t first = (int64_t)b * m;
    uint32_t bad = 0;
    if (a.indptr) {
        first = a.indptr[b];
        const int64_t count = (int64_t)a.indptr[b + 1] - first;
        bad |= count < 0 || count > m;
        m = (int)(count < 0 ? 0 : (count > m ? m : count));
    }
    if (first < 0 || first + m > a.total) {
        bad = 1;
        m = 0;
    }
    const int64_t room = (int64_t)a.g.table_stride * C - len;
    if (len < 0 || room < 0) {
        bad = 1;
        m = 0;
    } else if (m > room) {
        bad = 1;
        m = (int)room;
    }
    if (span == 0 && blockIdx.y == 0 && keys && threadIdx.x == 0) {
        if (a.new_lens) a.new_lens[b] = len + m;
        if (bad) atomicOr(&g_device_error, kDevErrBadData);
    }
    const int blk = (m > 0 ? len / C : 0) + span;
    const int lo = max(len - blk * C, 0);                       // first new slot of the page
    const int64_t end = (int64_t)len + m - (int64_t)blk * C;
    const int hi = (int)min((int64_t)C, end);                   // behind the last
    if (m <= 0 || hi <= lo) return;
    const int page = a.g.table[(int64_t)b * a.g.table_stride + blk];
    if (page < 0 || page >= a.g.n_pages) {
        if (threadIdx.x == 0) atomicOr(&g_device_error, kDevErrBadData);
        return;
    }
    const int64_t src0 = first + (int64_t)blk * C - len;        // source row of slot 0
    const bool rotate = keys && a.rotate;
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(a.g.kv_heads, h0 + a.heads_per_cta);
    const int warps = blockDim.x >> 5;

    // This thread's units: the same unit u of rows row, row + rows_pass, ... (the block's size is a multiple of UNITS).
    const int rows_pass = (int)blockDim.x / UNITS, row = (int)threadIdx.x / UNITS, u = (int)threadIdx.x - row * UNITS;
    int dim0 = u * N * SIDES, dim1 = dim0 + N, pair = dim0;
    if constexpr (W > 0) {  // only with a rotation
        const RopeUnit x = rope_unit<W>(a.r, D, u);
        dim0 = x.first;
        dim1 = x.second;
        pair = x.pair;
    }
    const bool turned = rotate && pair < a.r.end[2];
    const bool part_turned = turned && pair + 2 * PAIRS > a.r.end[2];  // an interleaved unit's last pairs may stay
    bool real[P];
    float2 cs[P][PAIRS];
    Pack<T, LN> next[P][SIDES][LOADS] = {};  // zeros where there is no row
    const T* from = src + (src0 + lo + row) * ts + h0 * hs + dim0;
    const int64_t step = rows_pass * ts;
    auto fetch = [&]() {
        const T* x = from;
#pragma unroll
        for (int p = 0; p < P; ++p, x += step)
            if (real[p]) {
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    next[p][0][j].load(x + j * LN);
                    if (SIDES == 2) next[p][SIDES - 1][j].load(x + (dim1 - dim0) + j * LN);
                }
            }
        from += hs;
    };
#pragma unroll
    for (int p = 0; p < P; ++p) real[p] = lo + row + p * rows_pass < hi;
    fetch();
    if (turned) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (real[p]) {
                const int slot = lo + row + p * rows_pass;
                const int32_t* triple = a.positions ? a.positions + 3 * (src0 + slot) : nullptr;
                const RopePos q = rope_position(a.r, triple, blk * C + slot);
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) cs[p][e] = rope_pair(a.r, q, pair + 2 * e);
            }
    }
    uint8_t* to = code + ((int64_t)page * a.g.kv_heads + h0) * C * D + (lo + row) * D + dim0;

    const int lane = threadIdx.x & 31;
    for (int h = h0; h < h1; ++h) {
        float f[P][SIDES][N];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int s = 0; s < SIDES; ++s)
#pragma unroll
                for (int e = 0; e < N; ++e) f[p][s][e] = next[p][s][e / LN].get(e % LN);
        if (h + 1 < h1) fetch();
        float top = 0.0f;  // NaN is passed over
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (turned) {
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) {
                    float& z0 = f[p][0][W ? e : 2 * e];
                    float& z1 = f[p][SIDES - 1][W ? e : 2 * e + 1];
                    const float x0 = z0, x1 = z1;
                    const float2 q = cs[p][e];
                    z0 = fmaf(-q.y, x1, q.x * x0);
                    z1 = fmaf(q.y, x0, q.x * x1);
                    // (1, 0) where the unit reaches behind the rotated dimensions: they must not meet their neighbour's
                    // infinity
                    if (W == 0 && part_turned && q.y == 0.0f && q.x == 1.0f) {
                        z0 = x0;
                        z1 = x1;
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < SIDES; ++s)
#pragma unroll
                for (int e = 0; e + 1 < N; e += 2) top = fmax3_abs(top, f[p][s][e], f[p][s][e + 1]);
            if (N == 1) top = fmax3_abs(top, f[p][0][0], f[p][SIDES - 1][0]);
        }
        uint32_t* const buf = part[h & 1];
        auto block_max = [&](float x) -> uint32_t {  // of non-negative numbers, as bits
            const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(x));
            if (lane == 0) buf[threadIdx.x >> 5] = w;
            __syncthreads();
            return __reduce_max_sync(0xffffffffu, lane < warps ? buf[lane] : 0u);
        };
        uint32_t amax = block_max(top);  // the other buffer is free: every thread read it before this barrier
        if (amax >= 0x7f800000u) {       // infinities saturate: the finite values set the scale
            top = 0.0f;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int s = 0; s < SIDES; ++s)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (fabsf(f[p][s][e]) < INFINITY) top = fmaxf(top, fabsf(f[p][s][e]));
            __syncthreads();
            amax = block_max(top);
        }
        const int64_t at = (int64_t)page * a.g.kv_heads + h;
        float sc = cache_scale(amax);
        uint8_t* const dst = code + at * C * D;
        if (lo > 0) {  // the block already holds tokens
            const float old = scale[at];
            if (sc > old) {
                const float ratio = old / sc;
                for (int i = threadIdx.x; i < lo * (D / 8); i += blockDim.x) {
                    uint2 w = *reinterpret_cast<const uint2*>(dst + i * 8);
                    uint32_t u[2] = {w.x, w.y};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t o = 0;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const uint32_t hh = half2_of_e4m3x2((u[j] >> (16 * s)) & 0xffffu);
                            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&hh));
                            o |= e4m3x2(z.x * ratio, z.y * ratio) << (16 * s);
                        }
                        u[j] = o;
                    }
                    *reinterpret_cast<uint2*>(dst + i * 8) = make_uint2(u[0], u[1]);
                }
            } else {
                sc = old;
            }
            __syncthreads();  // every thread has read the old scale
        }
        if (threadIdx.x == 0) scale[at] = sc;
        // a fresh scale's reciprocal is another power of two
        const float inv = lo > 0 ? 1.0f / sc : __uint_as_float((254u << 23) - __float_as_uint(sc));
        const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (!real[p]) continue;
#pragma unroll
            for (int s = 0; s < SIDES; ++s) {
                uint8_t* const out = to + p * rows_pass * D + (s ? dim1 - dim0 : 0);
                const float (&g)[N] = f[p][s];
                if constexpr (N == 8) {
                    *reinterpret_cast<uint2*>(out) =
                        make_uint2(e4m3x4(g[0], g[1], g[2], g[3], inv2), e4m3x4(g[4], g[5], g[6], g[7], inv2));
                } else if constexpr (N == 4) {
                    *reinterpret_cast<uint32_t*>(out) = e4m3x4(g[0], g[1], g[2], g[3], inv2);
                } else if constexpr (N == 2) {
                    *reinterpret_cast<uint16_t*>(out) = (uint16_t)e4m3x2(g[0] * inv, g[1] * inv);
                } else {
                    *out = (uint8_t)e4m3x2(g[0] * inv, 0.0f);
                }
            }
        }
        to += C * D;
    }
}

// Values, and keys that are not rotated, need no pairs: they take the widest loads whatever the pairing.
template <typename T, int D, int W>
__global__ void __launch_bounds__(kAppendThreads, 1) cache_append_kernel(const __grid_constant__ AppendArgs a,
                                                                         const T* __restrict__ k,
                                                                         const T* __restrict__ v) {
    if (blockIdx.z == 0) append_page<T, D, W>(a, k, a.k_token, a.k_head, a.code[0], a.scale[0], true);
    else append_page<T, D, 0>(a, v, a.v_token, a.v_head, a.code[1], a.scale[1], false);
}

}  // namespace losa
