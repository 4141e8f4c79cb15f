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

constexpr int kCaWarps = 4;       // of a CTA that shares units with others
constexpr int kCaUnitWarps = 8;   // of a CTA that has a short unit to itself
constexpr int kCaKeys = 32;    // keys of a warp's tile: never more than one page
constexpr int kCaMaxSplits = 128;
constexpr float kCaBias = 10.0f;

struct CacheAttnArgs {
    CacheGeom g;
    const float* k_scale;
    const float* v_scale;
    const uint8_t* v8;
    const __nv_bfloat16* q;
    __nv_bfloat16* o;
    float* lse;                // [seqs][tokens][heads] or null
    int64_t q_seq, q_token, q_head, o_seq, o_token, o_head;
    int heads, group, tokens, causal;
    int tiles;                 // row tiles of a (sequence, kv head)
    int tile_rows;
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
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The 8 x 8 matrix of 16-bit elements whose row g lies in lanes 4 g .. 4 g + 3, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The power of two that brings a row's largest magnitude (its bits) into [2^7, 2^8), or as near as 2^127 brings it
// (subnormal numbers below 2). A row with an infinity or NaN has no softmax: its factor is NaN, which makes every element of
// the row NaN, and so o and lse where it sees a key.
__device__ __forceinline__ float row_factor(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23);
    if (e == 255) return __uint_as_float(0x7fffffffu);
    return __uint_as_float((uint32_t)min(max(127 + 127 + 7 - e, 1), 254) << 23);
}

// The work of a call. A unit is a (sequence, kv head, row tile); its work is its sequence's 32-key tiles. The units' tiles,
// one behind the other, are cut into equal ranges, one per CTA, across the units' borders: ragged lengths and any number of
// heads load every SM alike (cutting each sequence by itself: 110 against 94 us on eight ragged streams). A unit that lies
// in several ranges is joined by cache_join_kernel. Every CTA finds its place in the lengths by itself.
struct CaWork {
    int64_t total, range;  // tiles of the call; of a CTA
};

__device__ __forceinline__ int ca_tiles_of(const CacheAttnArgs& a, int seq, int& len) {
    const int64_t room = (int64_t)a.g.table_stride * a.g.page;
    len = a.g.lens[seq];
    if (len < 0 || len > room) len = len < 0 ? 0 : (int)room;  // reported where the sequence's page table is read
    return (len + kCaKeys - 1) / kCaKeys;
}

// A quotient of non-negative numbers; in 32 bits where they fit, which saves about half a microsecond each.
__device__ __forceinline__ int64_t ca_div(int64_t x, int64_t y) {
    return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
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
    w.range = ca_div(w.total + ctas - 1, ctas);
    // at least two tiles a warp, and no unit in more than `splits` ranges
    const int least = (most + a.splits - 3) / (a.splits - 2);  // splits > 2
    w.range = max(w.range, (int64_t)max(least, 2 * kCaWarps));
    return w;
}

// Row of an 8-key group that column n of an S tile stands for. Any order is right as long as S, P and V agree; this one
// lets the eight lanes of a shared-memory phase read eight different 16-byte columns of the swizzled K and V tiles.
__device__ __forceinline__ int key_of_column(int n) { return (n & 1) ? ((n - 1) ^ 4) | 1 : n; }

template <int D> constexpr uint32_t kCaTile = kCaKeys * D;  // bytes of a warp's key or value tile
// NB: 8-row groups of a CTA's row tile. Up to eight rows, half the accumulators and products are enough.
template <int NB> constexpr int kCaRows = 8 * NB;
// Tiles in flight per warp and CTAs per SM: 128 KB on their way to an SM with 128 dimensions, 64 KB with 64. At 128 dimensions
// more (three tiles, or three CTAs, which eight rows have room for) queue in the memory system and let some SMs finish well
// before others: 84..86 against 80 us on eight ragged streams of four rows, 95 against 92 us on two long ones of twelve.
constexpr int kCaStages = 2;
constexpr int kCaCtas = 2;
template <int D, int NB, int NW> constexpr uint32_t kCaSmem =
    NW * kCaStages * (2 * kCaTile<D> + 8) + NW * kCaRows<NB> * 8 + 1024;

// Reads the codes once and does little else: the memory rate bounds it, if enough warps share the latency of the
// conversions and products in between. A warp owns a ring of 32-key tiles that TMA fills (one lane issues, one barrier per
// tile, no exchange between warps until the end of a unit). The products are taken transposed, S^T = K Q^T and
// O^T = V^T P^T on mma.m16n8k16, with the codes as the 16-row operand: 8 query rows then fill the other side, where the
// usual orientation would leave half of 16 rows empty (92 against 87 us on eight ragged streams of four rows). P^T comes out of
// S^T by movmatrix. The contraction is two orders of magnitude below the tensor peak here, and operands in registers need
// no further copy through shared memory, which tcgen05 would.
template <int D, int NB, int NW>
__global__ void __launch_bounds__(NW * 32, kCaCtas * kCaWarps / NW)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CacheAttnArgs a) {
    constexpr int ROWS = kCaRows<NB>, STAGES = kCaStages;
    constexpr uint32_t TILE = kCaTile<D>;
    constexpr int HK = D / 64;    // 16-byte pieces of a key row that a lane holds
    constexpr int VW = D / 32;    // 4-byte words of a value row that a lane holds
    constexpr int MT = D / 16;    // 16-row tiles of O^T
    constexpr int VD = D / 8;     // dimensions of a value row that a lane holds
    extern __shared__ __align__(1024) uint8_t ca_smem[];
    const uint32_t raw = smem_addr(ca_smem);
    uint8_t* const smem = ca_smem + (((raw + 1023u) & ~1023u) - raw);  // swizzled tiles need 1024-byte alignment
    const uint32_t base = smem_addr(smem);
    constexpr uint32_t BARS = NW * STAGES * 2 * TILE;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = base + warp * STAGES * 2 * TILE;
    const uint32_t bar = base + BARS + warp * STAGES * 8;
    float2* const row_ml = reinterpret_cast<float2*>(smem + BARS + NW * STAGES * 8);

    const int C = a.g.page;
    const int units = a.g.kv_heads * a.tiles;
    // the join's CTAs may take the room that these leave one by one: they wait for the whole grid themselves
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        for (int s = 0; s < STAGES; ++s) mbar_init(bar + 8 * s, 1);
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
    const int unit = n_tiles == 0 ? (int)(blockIdx.x % units) : (int)ca_div(pos - seq_pos, n_tiles);
    const int tile = unit % a.tiles, kvh = unit / a.tiles;
    const int64_t unit_pos = seq_pos + (int64_t)unit * n_tiles;
    const int t0 = (int)(pos - unit_pos), t1 = n_tiles == 0 ? 0 : (int)min((int64_t)n_tiles, stop - unit_pos);
    const int mine = max(0, (t1 - t0 - warp + NW - 1) / NW);  // this warp's tiles: t0 + warp, + NW, ...

    // Raw query rows, row 8 nb + g of the tile: asked for before the copies of codes, which would hold them up.
    const int n_rows = a.tokens * a.group;
    uint2 qw[NB][HK * 4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int r = tile * ROWS + 8 * nb + g;
        const int token = r / a.group, head = kvh * a.group + r % a.group;
        const __nv_bfloat16* const src = a.q + seq * a.q_seq + token * a.q_token + head * a.q_head + 16 * t;
#pragma unroll
        for (int s = 0; s < HK * 4; ++s)
            qw[nb][s] = r < n_rows ? *reinterpret_cast<const uint2*>(src + 64 * (s >> 2) + 4 * (s & 3)) : make_uint2(0, 0);
    }

    // Page and scales of the next 32 tiles, one tile per lane; a bad page is reported and its keys do not exist. The scales
    // are first needed when a tile has arrived: the copies do not wait for them, but follow them.
    int at_row = -1, at_page = 0;
    float at_ks = 1.0f, at_vs = 1.0f;
    const uint32_t base_fill = filled;
    auto pages = [&](int j) {
        const int i = j + (int)lane;
        at_row = -1;
        if (i < mine) {
            const int key = (t0 + warp + i * NW) * kCaKeys, blk = key / C;
            at_page = a.g.table[(int64_t)seq * a.g.table_stride + blk];
            if (at_page < 0 || at_page >= a.g.n_pages) atomicOr(&g_device_error, kDevErrBadData);
            else at_row = (int)(((int64_t)at_page * a.g.kv_heads + kvh) * C + (key - blk * C));
        }
    };
    auto scales = [&]() {
        at_ks = at_row < 0 ? -1.0f : a.k_scale[(int64_t)at_page * a.g.kv_heads + kvh];
        at_vs = at_row < 0 ? 1.0f : a.v_scale[(int64_t)at_page * a.g.kv_heads + kvh];
    };
    auto issue = [&](int j) {
        const int row = __shfl_sync(0xffffffffu, at_row, j & 31);
        const uint32_t s = (base_fill + j) % STAGES;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar + 8 * s, 2 * TILE);
            tma_load_2d(ring + s * 2 * TILE, &tmK, 0, max(row, 0), bar + 8 * s);
            tma_load_2d(ring + s * 2 * TILE + TILE, &tmV, 0, max(row, 0), bar + 8 * s);
        }
        ++filled;
    };
    pages(0);
    scales();
    for (int j = 0; j < STAGES && j < mine; ++j) issue(j);

    // Query rows as B fragments, row 8 nb + g: step (h, i) holds dimensions 64 h + 16 t + 4 i .. + 3. A lane's columns of S^T
    // and O^T are rows 2 t and 2 t + 1.
    uint32_t qb[NB][HK * 4][2];
    float c[NB][2];
    int lim[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const uint2 (&w)[HK * 4] = qw[nb];
        uint32_t amax = 0;
#pragma unroll
        for (int s = 0; s < HK * 4; ++s) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t u = x ? w[s].y : w[s].x;
                amax = max(amax, max((u & 0x7fffu) << 16, u & 0x7fff0000u));
            }
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const float f = row_factor(amax);
#pragma unroll
        for (int s = 0; s < HK * 4; ++s) {
            qb[nb][s][0] = pack_f16x2(__uint_as_float(w[s].x << 16) * f, __uint_as_float(w[s].x & 0xffff0000u) * f);
            qb[nb][s][1] = pack_f16x2(__uint_as_float(w[s].y << 16) * f, __uint_as_float(w[s].y & 0xffff0000u) * f);
        }
        const float cf = a.scale_log2 / f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            c[nb][x] = __shfl_sync(0xffffffffu, cf, 4 * (2 * t + x));
            const int rr = tile * ROWS + 8 * nb + 2 * t + x;
            lim[nb][x] = rr < n_rows && a.causal ? len - (a.tokens - 1 - rr / a.group) : len;
        }
    }
    const int least = a.causal ? len - (a.tokens - 1) : len;  // keys that every row sees

    float acc[MT][NB][4];
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][nb][i] = 0.0f;
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.0f;
    }
    const int ka = key_of_column(2 * t), kb = key_of_column(2 * t + 1), kg = key_of_column(g);

    bool ok = true, veiled_nan = false;
    int j = 0;
    for (; j < mine; ++j) {
        const uint32_t f = base_fill + j, s = f % STAGES;
        if (!(ok = wait_bounded_warp(bar + 8 * s, (f / STAGES) & 1u, a.wait_limit_ns))) break;
        const float2 sc = make_float2(__shfl_sync(0xffffffffu, at_ks, j & 31),
                                      fmaxf(__shfl_sync(0xffffffffu, at_vs, j & 31), 1e-30f));
        const uint32_t tk = ring + s * 2 * TILE, tv = tk + TILE;
        const int key0 = (t0 + warp + j * NW) * kCaKeys;
        const int have = sc.x < 0.0f ? 0 : min(kCaKeys, len - key0);  // keys of this tile that exist
        if (key0 + have > least) {
            // Some keys are hidden from some rows, whose weight 0 must not meet a NaN in V: it becomes 0 here, and the rows
            // that see it get it behind the loop. (Given to them at once it costs 3 % of a long call in scheduling.)
            bool found = false;
            for (uint32_t at = tv + max(least - key0, 0) * D + 4 * lane; at < tv + have * D; at += 128) {
                const uint32_t w = ld_shared_u32(at), nan = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                if (nan) {
                    st_shared_u32(at, w & ~nan);
                    found = true;
                }
            }
            veiled_nan |= __any_sync(0xffffffffu, found) != 0;
            fence_proxy_async_smem();  // a copy writes the tile next
            __syncwarp();
        }
        // S^T: 16 keys x 8 rows at a time; a lane's keys are 16 i + kg and 16 i + 8 + kg
        float sv[2][NB][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) sv[i][nb][x] = 0.0f;
#pragma unroll
        for (int h = 0; h < HK; ++h) {
            uint32_t u[4][4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t row = 8 * y + kg, ch = 4 * h + t;
                const uint4 w = ld_shared_v4(tk + (D == 128 ? row * 128u + ((ch ^ (row & 7u)) << 4)
                                                           : row * 64u + ((ch ^ ((row >> 1) & 3u)) << 4)));
                u[y][0] = w.x, u[y][1] = w.y, u[y][2] = w.z, u[y][3] = w.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t ka4[4] = {
                        half2_of_e4m3x2(u[2 * i][x] & 0xffffu), half2_of_e4m3x2(u[2 * i + 1][x] & 0xffffu),
                        half2_of_e4m3x2(u[2 * i][x] >> 16), half2_of_e4m3x2(u[2 * i + 1][x] >> 16)};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        mma_f16(sv[i][nb], ka4, qb[nb][4 * h + x][0], qb[nb][4 * h + x][1]);
                }
        }
        // x = t + log2 vs; keys a row does not see become -inf whatever their codes hold
        const float lv = __log2f(sc.y), inv_vs = 1.0f / sc.y;
        const bool whole = have == kCaKeys && key0 + kCaKeys <= least;
        uint32_t pb[2][NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float mx[2] = {-INFINITY, -INFINITY};
            const float ck[2] = {c[nb][0] * sc.x, c[nb][1] * sc.x};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int key = 16 * i + 8 * (x >> 1) + kg;
                    float v = fmaf(sv[i][nb][x], ck[x & 1], lv);
                    if (!whole && (key >= have || key0 + key >= lim[nb][x & 1])) v = -INFINITY;
                    sv[i][nb][x] = v;
                    mx[x & 1] = fmaxf(mx[x & 1], v);
                }
            float ref[2], alpha[2], add[2] = {0.0f, 0.0f};
            bool moved = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], y));
                const float top = fmaxf(m[nb][x], mx[x]);
                moved |= top > m[nb][x];
                alpha[x] = m[nb][x] == -INFINITY ? 0.0f : ex2_approx(m[nb][x] - top);
                m[nb][x] = top;
                ref[x] = top == -INFINITY ? 0.0f : kCaBias - top;
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) l[nb][x] *= alpha[x];
#pragma unroll
                for (int n = 0; n < MT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[n][nb][x] *= alpha[x & 1];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float p0 = ex2_approx(sv[i][nb][2 * y] + ref[0]), p1 = ex2_approx(sv[i][nb][2 * y + 1] + ref[1]);
                    add[0] += p0;
                    add[1] += p1;
                    pb[i][nb][y] = transpose8x8(pack_f16x2(p0, p1));
                }
            l[nb][0] = fmaf(add[0], inv_vs, l[nb][0]);
            l[nb][1] = fmaf(add[1], inv_vs, l[nb][1]);
        }
        // O^T += V^T P^T: row g of 16-row tile n is dimension VD g + 2 n, row g + 8 the next. Value rows of keys that do not
        // exist count as zero whatever they hold.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t u[4][VW];
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const uint32_t row = 16 * i + 8 * (r4 >> 1) + ((r4 & 1) ? kb : ka);
                if (D == 128) {
                    const uint4 w = ld_shared_v4(tv + row * 128u + (((uint32_t)g ^ (row & 7u)) << 4));
                    u[r4][0] = w.x, u[r4][1] = w.y, u[r4][VW - 2] = w.z, u[r4][VW - 1] = w.w;
                } else {
                    const uint2 w = ld_shared_v2(tv + row * 64u + (((uint32_t)(g >> 1) ^ ((row >> 1) & 3u)) << 4) +
                                                 8u * (g & 1));
                    u[r4][0] = w.x, u[r4][1] = w.y;
                }
                if (have < kCaKeys && (int)row >= have) {
#pragma unroll
                    for (int x = 0; x < VW; ++x) u[r4][x] = 0;
                }
            }
#pragma unroll
            for (int x = 0; x < VW; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t ab = __byte_perm(u[0][x], u[1][x], y ? 0x7362 : 0x5140);
                    const uint32_t cd = __byte_perm(u[2][x], u[3][x], y ? 0x7362 : 0x5140);
                    const uint32_t va[4] = {half2_of_e4m3x2(ab & 0xffffu), half2_of_e4m3x2(ab >> 16),
                                            half2_of_e4m3x2(cd & 0xffffu), half2_of_e4m3x2(cd >> 16)};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_f16(acc[2 * x + y][nb], va, pb[i][nb][0], pb[i][nb][1]);
                }
        }
        __syncwarp();  // every lane has read the tile
        if (j + STAGES < mine) {
            // the last tile of the 32 is consumed STAGES tiles after it was issued: pages run ahead of the scales
            if (((j + STAGES) & 31) == 0) pages(j + STAGES);
            issue(j + STAGES);
        }
        if (((j + 1) & 31) == 0) scales();
    }
    if (!ok)  // copies in flight land before the ring is used for anything else
        for (uint32_t x = base_fill + j; x != filled; ++x)
            wait_bounded_warp(bar + 8 * (x % STAGES), (x / STAGES) & 1u, kDrainLimitNs);

    // Join the warps through their own rings: [ROWS][D] fp32 each.
    float* const mine_o = reinterpret_cast<float*>(smem + warp * STAGES * 2 * TILE);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = 8 * nb + 2 * t + x;
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], y);
            if (g == 0) row_ml[warp * ROWS + r] = make_float2(m[nb][x], l[nb][x]);
#pragma unroll
            for (int n = 0; n < MT; ++n)
                *reinterpret_cast<float2*>(mine_o + r * D + VD * g + 2 * n) = make_float2(acc[n][nb][x], acc[n][nb][2 + x]);
        }
    if (veiled_nan) {  // NaN codes of keys that some rows do not see, for the rows that do
        __syncwarp();
        for (int i = max(0, (least / kCaKeys - t0 - warp) / NW); i < mine; ++i) {
            const int key0 = (t0 + warp + i * NW) * kCaKeys;
            for (int key = max(key0, least); key < min(key0 + kCaKeys, len); ++key) {
                const int page = a.g.table[(int64_t)seq * a.g.table_stride + key / C];
                if (page < 0 || page >= a.g.n_pages) continue;
                const uint8_t* const v = a.v8 + (((int64_t)page * a.g.kv_heads + kvh) * C + key % C) * D;
                for (int e = (int)lane; e < D; e += 32) {
                    if ((v[e] & 0x7f) != 0x7f) continue;
                    for (int r = 0; r < ROWS && tile * ROWS + r < n_rows; ++r)
                        if (key < len - (a.tokens - 1 - (tile * ROWS + r) / a.group)) mine_o[r * D + e] = __uint_as_float(0x7fffffffu);
                }
            }
        }
    }
    __syncthreads();
    const bool shared = a.splits != 0 && t1 - t0 < n_tiles;  // other CTAs hold the rest of the unit
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += NW * 32) {
        const int r = i / (D / 4), d0 = (i - r * (D / 4)) * 4;
        const int row = tile * ROWS + r;
        if (row >= n_rows) continue;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, row_ml[w * ROWS + r].x);
        float den = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float2 ml = row_ml[w * ROWS + r];
            const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - top);
            const float4 v = *reinterpret_cast<const float4*>(smem + w * STAGES * 2 * TILE + (r * D + d0) * 4);
            den = fmaf(ml.y, f, den);
            o[0] = fmaf(v.x, f, o[0]);
            o[1] = fmaf(v.y, f, o[1]);
            o[2] = fmaf(v.z, f, o[2]);
            o[3] = fmaf(v.w, f, o[3]);
        }
        const int token = row / a.group, head = kvh * a.group + row % a.group;
        const int64_t id = ((int64_t)seq * a.tokens + token) * a.heads + head;
        if (shared) {
            const int64_t at = id * a.splits + (int)(blockIdx.x - ca_div(unit_pos, range));
            *reinterpret_cast<float4*>(a.part_o + at * D + d0) = make_float4(o[0], o[1], o[2], o[3]);
            if (d0 == 0) a.part_ml[at] = make_float2(top, den);
        } else {
            // zero only where no key was seen: a row of NaN has a maximum of -inf as well
            const float inv = den == 0.0f ? 0.0f : 1.0f / den;
            *reinterpret_cast<uint2*>(a.o + seq * a.o_seq + token * a.o_token + head * a.o_head + d0) =
                make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
            if (a.lse && d0 == 0)
                a.lse[id] = den == 0.0f ? -INFINITY : (top - kCaBias + __log2f(den)) * 0.6931471805599453f;
        }
    }
    pos += max(t1 - t0, 1);
    if (!__syncthreads_and(ok)) break;  // the rings are free again; after a timeout every warp stops
    fence_proxy_async_smem();
    }
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
    // lens was there before the grid this one follows began: only its results have to be waited for
    int64_t unit_pos;
    const CaWork w = ca_work(a, ctas, seq, unit_pos);
    int len;
    const int n_tiles = ca_tiles_of(a, seq, len);
    if (a.g.lens[seq] != len && threadIdx.x == 0) atomicOr(&g_device_error, kDevErrBadData);
    const int row = token * a.group + head % a.group;
    unit_pos += (int64_t)(head / a.group * a.tiles + row / a.tile_rows) * n_tiles;
    const int splits =
        n_tiles ? (int)(ca_div(unit_pos + n_tiles - 1, w.range) - ca_div(unit_pos, w.range)) + 1 : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // by every CTA: this grid must not end before that one
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
        const float inv = den == 0.0f ? 0.0f : 1.0f / den;
        const float u = (sum[0][d] + sum[1][d]) + (sum[2][d] + sum[3][d]);
        const float v = (sum[0][d + 1] + sum[1][d + 1]) + (sum[2][d + 1] + sum[3][d + 1]);
        *reinterpret_cast<uint32_t*>(a.o + seq * a.o_seq + token * a.o_token + head * a.o_head + d) =
            pack_bf16x2(u * inv, v * inv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[id] = den == 0.0f ? -INFINITY : (top - kCaBias + __log2f(den)) * 0.6931471805599453f;
}

}  // namespace losa
