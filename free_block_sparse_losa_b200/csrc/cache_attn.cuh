// Attention of a few tokens over the paged 8-bit cache: cache_attn_kernel and, when a sequence's keys are split over
// several CTAs, cache_join_kernel.
//
// For one sequence and kv head the query rows are its tokens times the query heads that share the kv head. With codes k, v
// and their blocks' scales ks, vs, the logit of row r and key j in base 2 is t = c ks (q_r . k_j), c = scale log2 e, and
//   O_r = sum_j 2^t vs v_j / sum_j 2^t.
// The block's vs is folded into the exponent, x = t + log2 vs: the weights 2^(x - M) against the running maximum M of x
// multiply the codes v_j themselves, and the denominator adds 2^(x - M) / vs. So neither tile is ever scaled, and the
// weights are largest for the keys that matter most to O.
//
// Precision: e4m3 codes are exact in fp16. A query row is brought to a largest magnitude in [2^7, 2^8) by a power of two and
// is then exact in fp16 down to 2^-24 of its largest element. Weights are rounded to fp16 (11 bits) at 2^10 2^(x - M), so
// that weights down to 2^-34 of the largest are kept. Logits, sums and O are fp32.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "attn_tc.cuh"
#include "cache_append.cuh"

namespace losa {

constexpr int kCaWarps = 4;
constexpr int kCaStages = 3;   // tiles in flight per warp
constexpr int kCaKeys = 32;    // keys of a warp's tile: never more than one page
constexpr int kCaRows = 16;    // query rows of a CTA
constexpr int kCaMaxSplits = 128;
constexpr float kCaBias = 10.0f;

struct CacheAttnArgs {
    CacheGeom g;
    const float* k_scale;
    const float* v_scale;
    const __nv_bfloat16* q;
    __nv_bfloat16* o;
    float* lse;                // [seqs][tokens][heads] or null
    int64_t q_seq, q_token, q_head, o_seq, o_token, o_head;
    int heads, group, tokens, causal;
    int tiles;                 // 16-row tiles of a (sequence, kv head)
    int seqs;
    int splits;                // 0: one CTA per unit; else the most CTAs that share a unit
    float scale_log2;
    float* part_o;             // [row][split][D]
    float2* part_ml;           // [row][split]: maximum, denominator
    unsigned long long wait_limit_ns;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The power of two that brings a row's largest finite magnitude (its bits) into [2^7, 2^8); 1 for a zero row.
__device__ __forceinline__ float row_factor(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23);
    return e == 0 ? 1.0f : __uint_as_float((uint32_t)min(max(127 + 127 + 7 - e, 1), 254) << 23);
}

// The work of a call. A unit is a (sequence, kv head, row tile); its work is its sequence's 32-key tiles. The units' tiles,
// one behind the other, are cut into equal ranges, one per CTA, across the units' borders: ragged lengths and any number of
// heads load every SM alike (cutting each sequence by itself left a third of the time idle: 127 against 83 us on eight
// ragged streams). A unit that lies in several ranges is joined by cache_join_kernel. Every CTA finds its place in the
// lengths by itself.
struct CaWork {
    int64_t total, range;  // tiles of the call; of a CTA
};

__device__ __forceinline__ int ca_tiles_of(const CacheAttnArgs& a, int seq, int& len) {
    const int64_t room = (int64_t)a.g.table_stride * a.g.page;
    len = a.g.lens[seq];
    if (len < 0 || len > room) len = len < 0 ? 0 : (int)room;  // reported where the sequence's page table is read
    return (len + kCaKeys - 1) / kCaKeys;
}

// Total and range; with seq >= 0 also the tiles before that sequence. Called by a whole warp.
__device__ __forceinline__ CaWork ca_work(const CacheAttnArgs& a, int ctas, int seq, int64_t& before) {
    const int units = a.g.kv_heads * a.tiles;
    int64_t sum = 0, head = 0;
    int most = 0;
    for (int b = (int)lane_id(); b < a.seqs; b += 32) {
        int len;
        const int t = ca_tiles_of(a, b, len);
        sum += t;
        if (b < seq) head += t;
        most = max(most, t);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, x);
        head += __shfl_xor_sync(0xffffffffu, head, x);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, x));
    }
    before = head * units;
    CaWork w;
    w.total = sum * units;
    w.range = (w.total + ctas - 1) / ctas;
    // at least eight tiles for each warp pair of loads to pay, and no unit in more than `splits` ranges
    const int64_t least = a.splits > 2 ? ((int64_t)most + a.splits - 3) / (a.splits - 2) : most;
    w.range = max(max(w.range, least), (int64_t)(2 * kCaWarps));
    return w;
}

// Row of an 8-key group that column n of an S tile stands for. Any order is right as long as S, P and V agree; this one
// lets the eight lanes of a shared-memory phase read eight different 16-byte columns of the swizzled K and V tiles.
__device__ __forceinline__ int key_of_column(int n) { return (n & 1) ? ((n - 1) ^ 4) | 1 : n; }

template <int D> constexpr uint32_t kCaTile = kCaKeys * D;  // bytes of a warp's key or value tile
template <int D> constexpr uint32_t kCaSmem =
    kCaWarps * kCaStages * 2 * kCaTile<D> + kCaWarps * kCaStages * 16 + kCaWarps * kCaRows * 8 + 1024;

// Reads the codes once and does little else, so it is bound by memory. A warp owns a ring of 32-key tiles that TMA fills
// (one lane issues, one barrier per tile, no exchange between warps until the end): three tiles of 8 KB for each of eight
// warps keep 190 KB in flight per SM, several times what the latency asks for. S and P V run on mma.m16n8k16 with the
// query rows as the 16 rows of A: the contraction is two orders of magnitude below the tensor peak here, and operands in
// registers need no further copy through shared memory, which tcgen05 would.
template <int D>
__global__ void __launch_bounds__(kCaWarps * 32, 2)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CacheAttnArgs a) {
    constexpr uint32_t TILE = kCaTile<D>;
    constexpr int HK = D / 64;    // 16-byte pieces of a key row that a lane holds
    constexpr int VW = D / 32;    // 4-byte words of a value row that a lane holds
    constexpr int NT = D / 8;     // 8-column tiles of O
    extern __shared__ __align__(1024) uint8_t ca_smem[];
    const uint32_t raw = smem_addr(ca_smem);
    uint8_t* const smem = ca_smem + (((raw + 1023u) & ~1023u) - raw);  // swizzled tiles need 1024-byte alignment
    const uint32_t base = smem_addr(smem);
    constexpr uint32_t BARS = kCaWarps * kCaStages * 2 * TILE;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = base + warp * kCaStages * 2 * TILE;
    const uint32_t bar = base + BARS + warp * kCaStages * 8;
    float2* const tile_scale = reinterpret_cast<float2*>(smem + BARS + kCaWarps * kCaStages * 8) + warp * kCaStages;
    float2* const row_ml = reinterpret_cast<float2*>(smem + BARS + kCaWarps * kCaStages * 16);

    const int C = a.g.page;
    const int units = a.g.kv_heads * a.tiles;
    if (lane == 0) {
        for (int s = 0; s < kCaStages; ++s) mbar_init(bar + 8 * s, 1);
        fence_barrier_init();
    }
    __syncwarp();

    // This CTA's range of the call's tiles, and the sequence it starts in.
    int64_t pos, stop, range = 1, seq_pos = 0;  // seq_pos: first tile of sequence seq
    int seq = 0, len, n_tiles;
    if (a.splits == 0) {
        seq = blockIdx.x / units;
        n_tiles = ca_tiles_of(a, seq, len);
        seq_pos = 0;
        pos = (int64_t)(blockIdx.x - seq * units) * n_tiles;
        stop = pos + n_tiles;
        if (a.g.lens[seq] != len && threadIdx.x == 0) atomicOr(&g_device_error, kDevErrBadData);
        if (n_tiles == 0) stop = pos + 1;  // one round without keys writes the rows
    } else {
        const CaWork w = ca_work(a, gridDim.x, 0, seq_pos);
        range = w.range;
        pos = (int64_t)blockIdx.x * range;
        stop = min(w.total, pos + range);
        if (pos >= stop) return;
        // the sequence that holds tile pos < total: 32 sequences at a time
        seq_pos = 0;
        for (;; seq += 32) {
            int64_t upto = seq + (int)lane < a.seqs ? (int64_t)ca_tiles_of(a, seq + (int)lane, len) * units : 0;
            const int64_t own = upto;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, x);
                if ((int)lane >= x) upto += y;
            }
            const uint32_t behind = __ballot_sync(0xffffffffu, pos < seq_pos + upto);
            if (behind) {
                const int l = __ffs(behind) - 1;
                seq_pos += __shfl_sync(0xffffffffu, upto - own, l);
                seq += l;
                break;
            }
            seq_pos += __shfl_sync(0xffffffffu, upto, 31);
        }
        n_tiles = ca_tiles_of(a, seq, len);
    }
    uint32_t filled = 0;  // tiles this warp has issued so far: stage and phase of the next
    while (pos < stop) {
    while (a.splits != 0 && pos >= seq_pos + (int64_t)n_tiles * units) {
        seq_pos += (int64_t)n_tiles * units;
        n_tiles = ca_tiles_of(a, ++seq, len);
    }
    const int unit = n_tiles == 0 ? (int)(blockIdx.x % units) : (int)((pos - seq_pos) / n_tiles);
    const int tile = unit % a.tiles, kvh = unit / a.tiles;
    const int64_t unit_pos = seq_pos + (int64_t)unit * n_tiles;
    const int t0 = (int)(pos - unit_pos), t1 = n_tiles == 0 ? 0 : (int)min((int64_t)n_tiles, stop - unit_pos);
    const int mine = max(0, (t1 - t0 - warp + kCaWarps - 1) / kCaWarps);  // this warp's tiles: t0 + warp, + 4, ...

    // Page and scales of the next 32 tiles, one tile per lane; a bad page is reported and its keys do not exist.
    int at_row = 0;
    float at_ks = 1.0f, at_vs = 1.0f;
    const uint32_t base_fill = filled;
    auto issue = [&](int j) {
        if ((j & 31) == 0) {
            const int i = j + (int)lane;
            at_row = -1;
            at_ks = at_vs = 1.0f;
            if (i < mine) {
                const int key = (t0 + warp + i * kCaWarps) * kCaKeys, blk = key / C;
                const int page = a.g.table[(int64_t)seq * a.g.table_stride + blk];
                if (page < 0 || page >= a.g.n_pages) {
                    atomicOr(&g_device_error, kDevErrBadData);
                } else {
                    const int64_t ph = (int64_t)page * a.g.kv_heads + kvh;
                    at_row = (int)(ph * C + (key - blk * C));
                    at_ks = a.k_scale[ph];
                    at_vs = fmaxf(a.v_scale[ph], 1e-30f);
                }
            }
        }
        const int row = __shfl_sync(0xffffffffu, at_row, j & 31);
        const float ks = __shfl_sync(0xffffffffu, at_ks, j & 31), vs = __shfl_sync(0xffffffffu, at_vs, j & 31);
        const uint32_t s = (base_fill + j) % kCaStages;
        if (lane == 0) {
            tile_scale[s] = make_float2(row < 0 ? -1.0f : ks, vs);
            mbar_arrive_expect_tx(bar + 8 * s, 2 * TILE);
            tma_load_2d(ring + s * 2 * TILE, &tmK, 0, max(row, 0), bar + 8 * s);
            tma_load_2d(ring + s * 2 * TILE + TILE, &tmV, 0, max(row, 0), bar + 8 * s);
        }
        ++filled;
    };
    for (int j = 0; j < kCaStages && j < mine; ++j) issue(j);

    // Query rows g and g + 8 of the tile as A fragments: step (h, i) holds dimensions 64 h + 16 t + 4 i .. + 3.
    const int n_rows = a.tokens * a.group;
    uint32_t qa[HK * 4][4];
    float c[2];
    int lim[2];
    {
        uint32_t amax[2] = {0, 0};
        uint2 w[2][HK * 4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = tile * kCaRows + g + 8 * half;
            const int token = r / a.group, head = kvh * a.group + r % a.group;
            lim[half] = r < n_rows && a.causal ? len - (a.tokens - 1 - token) : len;
            const __nv_bfloat16* const src = a.q + seq * a.q_seq + token * a.q_token + head * a.q_head + 16 * t;
#pragma unroll
            for (int s = 0; s < HK * 4; ++s) {
                w[half][s] = r < n_rows ? *reinterpret_cast<const uint2*>(src + 64 * (s >> 2) + 4 * (s & 3))
                                        : make_uint2(0, 0);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t u = x ? w[half][s].y : w[half][s].x;
                    const uint32_t lo = (u & 0x7fffu) << 16, hi = u & 0x7fff0000u;
                    amax[half] = max(amax[half], max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
                }
            }
            amax[half] = max(amax[half], __shfl_xor_sync(0xffffffffu, amax[half], 1));
            amax[half] = max(amax[half], __shfl_xor_sync(0xffffffffu, amax[half], 2));
            const float f = row_factor(amax[half]);
            c[half] = a.scale_log2 / f;
#pragma unroll
            for (int s = 0; s < HK * 4; ++s) {
                const uint32_t u0 = w[half][s].x, u1 = w[half][s].y;
                qa[s][half] = pack_f16x2(__uint_as_float(u0 << 16) * f, __uint_as_float(u0 & 0xffff0000u) * f);
                qa[s][2 + half] = pack_f16x2(__uint_as_float(u1 << 16) * f, __uint_as_float(u1 & 0xffff0000u) * f);
            }
        }
    }

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int ka = key_of_column(2 * t), kb = key_of_column(2 * t + 1), kg = key_of_column(g);

    bool ok = true;
    int j = 0;
    for (; j < mine; ++j) {
        const uint32_t f = base_fill + j, s = f % kCaStages;
        if (!(ok = wait_bounded_warp(bar + 8 * s, (f / kCaStages) & 1u, a.wait_limit_ns))) break;
        const float2 sc = tile_scale[s];  // written before the arrival this wait has seen
        const uint32_t tk = ring + s * 2 * TILE, tv = tk + TILE;
        const int key0 = (t0 + warp + j * kCaWarps) * kCaKeys;
        const int have = sc.x < 0.0f ? 0 : min(kCaKeys, len - key0);  // keys of this tile that exist
        float sv[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sv[n][i] = 0.0f;
            const int row = 8 * n + kg;
#pragma unroll
            for (int h = 0; h < HK; ++h) {
                const uint32_t ch = (uint32_t)(4 * h + t);
                const uint32_t off = D == 128 ? row * 128u + ((ch ^ (row & 7u)) << 4)
                                              : row * 64u + ((ch ^ ((row >> 1) & 3u)) << 4);
                const uint4 w = ld_shared_v4(tk + off);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_f16(sv[n], qa[4 * h + i], half2_of_e4m3x2(u[i] & 0xffffu), half2_of_e4m3x2(u[i] >> 16));
            }
        }
        // x = t + log2 vs; keys a row does not see become -inf whatever their codes hold
        const float lv = __log2f(sc.y), inv_vs = 1.0f / sc.y;
        const float ck[2] = {c[0] * sc.x, c[1] * sc.x};
        const bool whole = have == kCaKeys && key0 + kCaKeys <= min(lim[0], lim[1]);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int half = i >> 1, key = 8 * n + ((i & 1) ? kb : ka);
                float x = fmaf(sv[n][i], ck[half], lv);
                if (!whole && (key >= have || key0 + key >= lim[half])) x = -INFINITY;
                sv[n][i] = x;
                mx[half] = fmaxf(mx[half], x);
            }
        float ref[2], alpha[2];
        bool moved = false;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 1));
            mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 2));
            const float top = fmaxf(m[half], mx[half]);
            moved |= top > m[half];
            alpha[half] = m[half] == -INFINITY ? 0.0f : ex2_approx(m[half] - top);
            m[half] = top;
            ref[half] = top == -INFINITY ? 0.0f : kCaBias - top;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int half = 0; half < 2; ++half) l[half] *= alpha[half];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] *= alpha[i >> 1];
        }
        uint32_t pa[2][4];
        float add[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = ex2_approx(sv[n][i] + ref[i >> 1]);
                add[i >> 1] += p[i];
            }
            pa[n >> 1][2 * (n & 1)] = pack_f16x2(p[0], p[1]);
            pa[n >> 1][2 * (n & 1) + 1] = pack_f16x2(p[2], p[3]);
        }
        l[0] = fmaf(add[0], inv_vs, l[0]);
        l[1] = fmaf(add[1], inv_vs, l[1]);
        // O += P V: value rows of keys that do not exist count as zero whatever they hold
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t u[4][VW];
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const int row = 16 * kk + 8 * (r4 >> 1) + ((r4 & 1) ? kb : ka);
                if (D == 128) {
                    const uint4 w = ld_shared_v4(tv + row * 128u + (((uint32_t)g ^ (row & 7u)) << 4));
                    u[r4][0] = w.x, u[r4][1] = w.y, u[r4][VW - 2] = w.z, u[r4][VW - 1] = w.w;
                } else {
                    const uint2 w = ld_shared_v2(tv + row * 64u + (((uint32_t)(g >> 1) ^ ((row >> 1) & 3u)) << 4) +
                                                 8u * (g & 1));
                    u[r4][0] = w.x, u[r4][1] = w.y;
                }
                if (have < kCaKeys && row >= have) {
#pragma unroll
                    for (int x = 0; x < VW; ++x) u[r4][x] = 0;
                }
            }
#pragma unroll
            for (int x = 0; x < VW; ++x) {
                const uint32_t ab0 = __byte_perm(u[0][x], u[1][x], 0x5140), ab1 = __byte_perm(u[0][x], u[1][x], 0x7362);
                const uint32_t cd0 = __byte_perm(u[2][x], u[3][x], 0x5140), cd1 = __byte_perm(u[2][x], u[3][x], 0x7362);
                mma_f16(acc[4 * x], pa[kk], half2_of_e4m3x2(ab0 & 0xffffu), half2_of_e4m3x2(cd0 & 0xffffu));
                mma_f16(acc[4 * x + 1], pa[kk], half2_of_e4m3x2(ab0 >> 16), half2_of_e4m3x2(cd0 >> 16));
                mma_f16(acc[4 * x + 2], pa[kk], half2_of_e4m3x2(ab1 & 0xffffu), half2_of_e4m3x2(cd1 & 0xffffu));
                mma_f16(acc[4 * x + 3], pa[kk], half2_of_e4m3x2(ab1 >> 16), half2_of_e4m3x2(cd1 >> 16));
            }
        }
        __syncwarp();  // every lane has read the tile
        if (j + kCaStages < mine) issue(j + kCaStages);
    }
    if (!ok)  // copies in flight land before the ring is used for anything else
        for (uint32_t x = base_fill + j; x != filled; ++x)
            wait_bounded_warp(bar + 8 * (x % kCaStages), (x / kCaStages) & 1u, kDrainLimitNs);

    // Join the four warps through their own rings: [16 rows][D] fp32 each.
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
        if (t == 0) row_ml[warp * kCaRows + g + 8 * half] = make_float2(m[half], l[half]);
    }
    float* const mine_o = reinterpret_cast<float*>(smem + warp * kCaStages * 2 * TILE);
    // column 2t (+1) of O tile n is dimension (D / 8) (2t (+1)) + n
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine_o[(g + 8 * (i >> 1)) * D + NT * (2 * t + (i & 1)) + n] = acc[n][i];
    __syncthreads();
    const bool shared = a.splits != 0 && t1 - t0 < n_tiles;  // other CTAs hold the rest of the unit
    for (int i = threadIdx.x; i < kCaRows * (D / 4); i += kCaWarps * 32) {
        const int r = i / (D / 4), d0 = (i - r * (D / 4)) * 4;
        const int row = tile * kCaRows + r;
        if (row >= n_rows) continue;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kCaWarps; ++w) top = fmaxf(top, row_ml[w * kCaRows + r].x);
        float den = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kCaWarps; ++w) {
            const float2 ml = row_ml[w * kCaRows + r];
            const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - top);
            const float4 v = *reinterpret_cast<const float4*>(smem + w * kCaStages * 2 * TILE + (r * D + d0) * 4);
            den = fmaf(ml.y, f, den);
            o[0] = fmaf(v.x, f, o[0]);
            o[1] = fmaf(v.y, f, o[1]);
            o[2] = fmaf(v.z, f, o[2]);
            o[3] = fmaf(v.w, f, o[3]);
        }
        const int token = row / a.group, head = kvh * a.group + row % a.group;
        const int64_t id = ((int64_t)seq * a.tokens + token) * a.heads + head;
        if (shared) {
            const int64_t at = id * a.splits + (int)(blockIdx.x - unit_pos / range);
            *reinterpret_cast<float4*>(a.part_o + at * D + d0) = make_float4(o[0], o[1], o[2], o[3]);
            if (d0 == 0) a.part_ml[at] = make_float2(top, den);
        } else {
            const float inv = top == -INFINITY ? 0.0f : 1.0f / den;
            *reinterpret_cast<uint2*>(a.o + seq * a.o_seq + token * a.o_token + head * a.o_head + d0) =
                make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
            if (a.lse && d0 == 0)
                a.lse[id] = top == -INFINITY ? -INFINITY : (top - kCaBias + __log2f(den)) * 0.6931471805599453f;
        }
    }
    pos += max(t1 - t0, 1);
    if (!__syncthreads_and(ok)) break;  // the rings are free again; after a timeout every warp stops
    fence_proxy_async_smem();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the ranges that share a unit, weighted by 2^(their maximum - the row's): one CTA per row, a warp for every fourth
// range. Rows of units in one range are done already; rows of empty sequences are in none and become zero here.
template <int D>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ CacheAttnArgs a, int ctas) {
    constexpr int E = D / 32;
    __shared__ float sum[4][D], dens[4];
    const int64_t id = blockIdx.x;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int64_t tok = id / a.heads;
    const int head = (int)(id - tok * a.heads), seq = (int)(tok / a.tokens), token = (int)(tok - (int64_t)seq * a.tokens);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int64_t unit_pos;
    const CaWork w = ca_work(a, ctas, seq, unit_pos);
    int len;
    const int n_tiles = ca_tiles_of(a, seq, len);
    if (a.g.lens[seq] != len && threadIdx.x == 0) atomicOr(&g_device_error, kDevErrBadData);
    const int row = token * a.group + head % a.group;
    unit_pos += (int64_t)(head / a.group * a.tiles + row / kCaRows) * n_tiles;
    const int64_t first = unit_pos / w.range;
    const int splits = n_tiles ? (int)((unit_pos + n_tiles - 1) / w.range - first) + 1 : 0;
    if (splits == 1) return;
    const float2* const ml = a.part_ml + id * a.splits;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, ml[s].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    float den = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
    for (int s = warp; s < splits; s += 4) {
        const float2 p = ml[s];
        const float f = p.x == -INFINITY ? 0.0f : ex2_approx(p.x - top);
        const float* const src = a.part_o + (id * a.splits + s) * D + lane;
        den = fmaf(p.y, f, den);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(src[32 * e], f, o[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sum[warp][lane + 32 * e] = o[e];
    if (lane == 0) dens[warp] = den;
    __syncthreads();
    den = (dens[0] + dens[1]) + (dens[2] + dens[3]);
    if (threadIdx.x < D / 2) {
        const int d = 2 * threadIdx.x;
        const float inv = top == -INFINITY ? 0.0f : 1.0f / den;
        const float u = (sum[0][d] + sum[1][d]) + (sum[2][d] + sum[3][d]);
        const float v = (sum[0][d + 1] + sum[1][d + 1]) + (sum[2][d + 1] + sum[3][d + 1]);
        *reinterpret_cast<uint32_t*>(a.o + seq * a.o_seq + token * a.o_token + head * a.o_head + d) =
            pack_bf16x2(u * inv, v * inv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[id] = top == -INFINITY ? -INFINITY : (top - kCaBias + __log2f(den)) * 0.6931471805599453f;
}

}  // namespace losa
