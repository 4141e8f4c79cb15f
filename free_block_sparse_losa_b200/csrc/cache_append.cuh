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

constexpr int kAppendThreads = 512;
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

template <typename T> __device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
    RopeVec<__nv_bfloat16>::unpack(__ldcs(reinterpret_cast<const uint4*>(p)), f);
}
template <> __device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 w = __ldcs(reinterpret_cast<const float4*>(p) + i);
        f[4 * i] = w.x;
        f[4 * i + 1] = w.y;
        f[4 * i + 2] = w.z;
        f[4 * i + 3] = w.w;
    }
}

// One CTA takes the new tokens of one page, for the keys (blockIdx.z = 0) or the values, and walks a group of kv heads.
// K and V are read once and their codes written once, so the kernel is bound by memory; what could cost more is the
// angles (an angle per token and pair against six bytes of traffic per pair and head), so they are computed once per CTA
// into shared memory and used for all its heads. A head's rows of the page stay in registers between the maximum over
// the block and the rounding.
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kAppendThreads, 2) cache_append_kernel(const __grid_constant__ AppendArgs a,
                                                                         const T* __restrict__ k,
                                                                         const T* __restrict__ v) {
    constexpr int W = D / 8;                   // 8-element chunks of a row
    constexpr int ROWS = kAppendThreads / W;   // rows a pass covers
    constexpr int P = 128 / ROWS;              // passes over the largest page
    extern __shared__ float2 angle[];          // [new rows of the page][D / 2]: cos, sin
    __shared__ uint32_t part[2][kAppendThreads / 32];

    const int b = blockIdx.x / a.spans, span = blockIdx.x - b * a.spans;
    const bool keys = blockIdx.z == 0;
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
    const int row0 = (int)threadIdx.x / W, e0 = ((int)threadIdx.x % W) * 8;
    const int64_t src0 = first + (int64_t)blk * C - len;        // source row of slot 0
    const bool rotate = keys && a.rotate;
    if (rotate) {
        for (int i = threadIdx.x; i < (hi - lo) * (D / 2); i += kAppendThreads) {
            const int row = i / (D / 2), pair = i - row * (D / 2);
            const int axis = 2 * pair < a.r.end[0] ? 0 : (2 * pair < a.r.end[1] ? 1 : 2);
            if (2 * pair < a.r.end[2]) {
                const int32_t* triple = a.positions ? a.positions + 3 * (src0 + lo + row) : nullptr;
                const RopePos q = rope_position(a.r, triple, blk * C + lo + row);
                angle[i] = rope_angle(a.r.step[pair], axis == 0 ? q.p[0] : (axis == 1 ? q.p[1] : q.p[2]));
            }
        }
        __syncthreads();
    }
    // where this thread's dimensions find their pair and partner
    const int turned = rotate ? a.r.end[2] - e0 : 0;
    int pair[HALVES ? 8 : 1], partner[HALVES ? 8 : 1];
    uint32_t second = 0;
    if (HALVES) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int x = e0 + e;
            const int ax = x < a.r.end[0] ? 0 : (x < a.r.end[1] ? 1 : 2);
            const int base = ax == 0 ? 0 : a.r.end[ax - 1], h = a.r.half[ax], l = x - base;
            const bool f = l < h;
            second |= f ? 0u : 1u << e;
            pair[e] = (base >> 1) + (f ? l : l - h);
            partner[e] = f ? x + h : x - h;
        }
    }

    const T* const src = keys ? k : v;
    const int64_t ts = keys ? a.k_token : a.v_token, hs = keys ? a.k_head : a.v_head;
    uint8_t* const code = a.code[keys ? 0 : 1];
    float* const scale = a.scale[keys ? 0 : 1];
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(a.g.kv_heads, h0 + a.heads_per_cta);
    for (int h = h0; h < h1; ++h) {
        float f[P][8];
        uint32_t amax = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int slot = lo + p * ROWS + row0;
            if (slot < hi) load8(src + (src0 + slot) * ts + h * hs + e0, f[p]);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int slot = lo + p * ROWS + row0;
            if (slot >= hi) continue;
            if (turned > 0) {
                const float2* const row = angle + (slot - lo) * (D / 2);
                if (HALVES) {
                    const T* const g = src + (src0 + slot) * ts + h * hs;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < turned) {
                            const float2 cs = row[pair[e]];
                            f[p][e] = fmaf((second >> e) & 1u ? cs.y : -cs.y, RopeVec<T>::one(g + partner[e]),
                                           cs.x * f[p][e]);
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        if (e < turned) {
                            const float2 cs = row[(e0 + e) >> 1];
                            const float x0 = f[p][e], x1 = f[p][e + 1];
                            f[p][e] = fmaf(-cs.y, x1, cs.x * x0);
                            f[p][e + 1] = fmaf(cs.y, x0, cs.x * x1);
                        }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t u = __float_as_uint(f[p][e]) & 0x7fffffffu;
                amax = max(amax, u < 0x7f800000u ? u : 0u);  // infinities saturate, NaN stays NaN: neither sets a scale
            }
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        uint32_t* const buf = part[h & 1];
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = amax;
        __syncthreads();  // the other buffer is free: every thread read it before this barrier
        amax = __reduce_max_sync(0xffffffffu, buf[threadIdx.x & (kAppendThreads / 32 - 1)]);
        const int64_t at = (int64_t)page * a.g.kv_heads + h;
        float sc = cache_scale(amax);
        uint8_t* const dst = code + at * C * D;
        if (lo > 0) {  // the block already holds tokens
            const float old = scale[at];
            if (sc > old) {
                const float ratio = old / sc;
                for (int i = threadIdx.x; i < lo * W; i += kAppendThreads) {
                    uint2 w = *reinterpret_cast<const uint2*>(dst + i * 8);
                    uint32_t u[2] = {w.x, w.y};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t o = 0;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const uint32_t hh = half2_of_e4m3x2(u[j] >> (16 * s));
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
        const float inv = 1.0f / sc;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int slot = lo + p * ROWS + row0;
            if (slot >= hi) continue;
            uint32_t u[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                u[j] = e4m3x2(f[p][4 * j] * inv, f[p][4 * j + 1] * inv) |
                       (e4m3x2(f[p][4 * j + 2] * inv, f[p][4 * j + 3] * inv) << 16);
            *reinterpret_cast<uint2*>(dst + (int64_t)slot * D + e0) = make_uint2(u[0], u[1]);
        }
    }
}

}  // namespace losa
