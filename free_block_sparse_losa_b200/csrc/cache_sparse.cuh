// Attention of 128-row query blocks over listed blocks (or all blocks) of the paged 8-bit cache: cache_sparse_kernel.
//
// The mathematics is cache_attn.cuh's: with codes k, v and scales ks, vs of a block, x = c ks (q . k) + log2 vs, and O is the
// sum of 2^(x - M) v over the sum of 2^(x - M) / vs, so no tile is ever scaled. Both products run on the tensor cores
// without widening K: a bf16 query element has 8 significant bits and is split, after its row was brought to a largest
// magnitude in [2^7, 2^8) by a power of two, into two e4m3 numbers of 4 bits each, q = q1 + q2 (exact down to 2^-9 of the
// row's largest element, off by at most 2^-17 of it below), so Q K^T is two kind::f8f6f4 products that read the codes as
// they lie in the cache, at the cost of one bf16 product. P keeps fp16's 11 bits and its range (weights down to 2^-31 of
// the largest: the tail under an attention sink is not lost), so V is widened to fp16 on its way, which is exact; four
// warps do that next to the softmax.
//
// One persistent CTA per SM walks one stream of items in rounds over the work order (a snake, longest first); the tiles
// (128 keys: 1, 2 or 4 blocks) of all its items form one sequence n = 0, 1, 2, ...:
//   warp 3       reads order, lists, page table and scales eight tiles at a time (a lane per 32-key quarter, so that the
//                chain of dependent loads is paid once for eight tiles) into a ring of tile records.
//   warp 0 / 2   TMA: K / V codes, four 32-key boxes a tile, one per lane.
//   warps 24..27 split an item's Q into shared memory, an item ahead; the reader has its rows fetched into L2.
//   warps 20..23 widen V (zeroing keys that do not exist), and store an item's O from the V slot it was staged in before
//                refilling that slot.
//   warp 1       MMA: S_n = Q K^T into S buffer n & 1, then O += P V of tile n - 2 with P from TMEM.
//   warps 4..19  softmax in two pairs of groups. The pairs take the tiles in turn, a group half of a tile's keys: while one
//                pair waits for S or finds maxima, the other's exponentials keep the exp unit busy.
// A row's reference maximum moves only when a tile's maximum exceeds it by more than 2^8. Each group publishes its half's
// row maxima (M_READY), and every thread follows the reference of its row through the tiles by itself; the pair whose tile
// moves it rescales O in place, behind P V of the tile before. Each group keeps its own share of the denominator; the pair
// with the item's last tile adds them up, divides and stages O at once: O's next item waits for it, and the other pair works
// meanwhile.
// TMEM: S_0 0..127, S_1 128..255, O 256..383, P_0 384..447, P_1 448..511. An S buffer is free once its pair has it in
// registers, so Q K^T runs two tiles ahead of P V.
//
// Measured on a 4680-token chunk over 32760 keys (12 heads) and on a 480p layer with 16 listed 32-key blocks a row: 990 and
// 193 us, 963 and 535 TFLOP/s. Steps that brought it there: one softmax path, keys that do not exist as -inf, and V widened
// without register swaps (1523 -> 1175 us, 297 -> 252); groups that take tiles in turn instead of halving every tile
// (-> 1141); MMA issued from uniform registers, four groups and Q split by warps of its own (-> 1052, 259 -> 198); waits for
// two barriers at once, a pair that walks only its own tiles, the first rows split before their records (-> 990, 193). Leaving
// out half of the MMAs, the exponentials or the widening takes at most a tenth off, all three a fifth: no single unit bounds
// it, but the chain S -> maximum -> weights -> P of two tiles in flight, and with short lists 3 us an item. Slower: three
// groups of whole rows with P over S (1175, 214 us), rows whole in a warp by 16-lane TMEM loads (7 %), O written behind the
// next tile's maximum (a fifth; registers). No faster: warps of their own for each product, blocks taken from the grid as
// CTAs come free.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "attn_tc.cuh"
#include "cache_attn.cuh"

namespace losa {

constexpr int kCsThreads = 896;
constexpr uint32_t kCsTile8 = 128 * 128;                  // a tile of codes
constexpr int kCsKStages = 3;
constexpr uint32_t kCsQ = 0;                              // 2 x (q1, q2)
constexpr uint32_t kCsK = 4 * kCsTile8;                   // 3 K tiles
constexpr uint32_t kCsV8 = kCsK + kCsKStages * kCsTile8;  // 2 V tiles of codes
constexpr uint32_t kCsVf = kCsV8 + 2 * kCsTile8;          // 2 fp16 V tiles (second use: O staging)
constexpr uint32_t kCsBar = kCsVf + 2 * kTileBytes;       // 48 barrier slots; the last holds the TMEM address
constexpr uint32_t kCsRec = kCsBar + 384;                 // tile records
constexpr int kCsBatch = 8, kCsBatches = 3;

struct CsTile {
    int32_t row[4];     // pool row of each 32-key quarter
    float ks[4], lv[4], iv[4];  // scale of K, log2 and reciprocal of V's
    uint32_t kv4;       // keys that exist in each quarter, 8 bits each
    int32_t qrow;       // first row of the query block in [H * Np]
    int32_t flags;      // of the tile in its item; negative: past the end of this CTA's work
    int32_t item;       // number of the item in this CTA's work
};
constexpr int kCsFirst = 1, kCsSecond = 2, kCsPre = 4, kCsLast = 8;  // first, second, last but one, last tile of an item
static_assert(sizeof(CsTile) == 80, "tile record");

constexpr uint32_t kCsFac = kCsRec + kCsBatch * kCsBatches * sizeof(CsTile);  // [4][128] reciprocal row factors
constexpr uint32_t kCsTop = kCsFac + 4 * 128 * 4;    // [4 tiles][2 halves][128] row maxima
constexpr uint32_t kCsDen = kCsTop + 8 * 128 * 4;    // [2 items][4 groups][128] (denominator, its reference)
constexpr uint32_t kCsSmem = kCsDen + 8 * 128 * 8;
static_assert(kCsSmem <= 232448, "shared memory");

enum : uint32_t {
    C_Q_FULL0 = 0, C_Q_EMPTY0 = 2, C_K_FULL0 = 4, C_K_EMPTY0 = 7, C_V8_FULL0 = 10, C_V8_EMPTY0 = 12, C_VF_FULL0 = 14,
    C_S_FULL0 = 16, C_P_FULL0 = 18, C_PV_DONE0 = 20, C_STAGED0 = 22, C_FLUSHED0 = 24, C_REC_FULL0 = 26,
    C_REC_EMPTY0 = 29, C_S_FREE0 = 32, C_M_READY0 = 34, C_O_FREE = 36, C_MMA_DONE, C_COUNT
};

struct CacheSparseArgs {
    CacheGeom g;
    const float* k_scale;
    const float* v_scale;
    const __nv_bfloat16* q;
    float* lse;               // may be null
    int heads, group;         // query heads of one sequence; query heads that share a kv head
    int Np, nq, n_items;
    int sub;                  // blocks of a 128-key tile
    float scale_log2;
    const int32_t* indptr;    // null: every block of the sequence
    const int32_t* kv_idx;
    const int32_t* order;     // null: ascending
    unsigned long long wait_limit_ns;
};

// MMA and commit issued by one elected lane of a converged warp. Descriptors, addresses and barriers must be uniform over
// the warp and known to be (values from shared memory go through a broadcast shuffle): the operands then stay in uniform
// registers. Issued by a lone thread in divergent code, each operand is copied there anew, and the issuing thread, not the
// tensor cores, sets the pace (measured: 1159 us against 950 us on a 4680-token chunk over 32760 keys).
__device__ __forceinline__ void el_mma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void el_mma_ts_f16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void el_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar) : "memory");
}
// Start fetching `bytes` of global memory into L2.
__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Instruction descriptor with A and B of format 0 (fp16 for kind::f16, e4m3 for kind::f8f6f4) and fp32 D.
__host__ __device__ constexpr uint32_t idesc_fmt0_f32(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ bool cs_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
    return wait_bounded_warp(bar, parity, limit_ns);
}
// Two barriers, both tested before either answer is looked at.
__device__ __forceinline__ bool cs_wait2(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1,
                                         unsigned long long limit_ns) {
    const bool ok0 = mbar_try_wait(bar0, parity0), ok1 = mbar_try_wait(bar1, parity1);
    if (__all_sync(0xffffffffu, ok0 && ok1)) return true;
    return cs_wait(bar0, parity0, limit_ns) && cs_wait(bar1, parity1, limit_ns);
}

constexpr float kCsBias = 7.0f;   // weights are kept at 2^7 of their size: at most 2^15 when the reference lags by 2^8

__global__ void __launch_bounds__(kCsThreads, 1)
    cache_sparse_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CacheSparseArgs a) {
    extern __shared__ __align__(1024) uint8_t cs_smem[];
    const uint32_t base = smem_addr(cs_smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicOr(&g_device_error, kDevErrBadData);
        return;
    }
    auto BAR = [&](uint32_t s) { return base + kCsBar + 8u * s; };
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(cs_smem + kCsBar + 47 * 8);
    CsTile* const recs = reinterpret_cast<CsTile*>(cs_smem + kCsRec);
    float* const fac = reinterpret_cast<float*>(cs_smem + kCsFac);
    float* const tops = reinterpret_cast<float*>(cs_smem + kCsTop);
    float2* const dens = reinterpret_cast<float2*>(cs_smem + kCsDen);

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
    const uint32_t lane = lane_id();
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < C_COUNT; ++s) {
            uint32_t cnt = 1;
            if (s / 2 == C_P_FULL0 / 2 || s / 2 == C_STAGED0 / 2 || s / 2 == C_S_FREE0 / 2 || s / 2 == C_M_READY0 / 2 ||
                s == C_O_FREE)
                cnt = 256;  // the two softmax groups of a tile
            else if (s / 2 == C_Q_FULL0 / 2 || s / 2 == C_V8_EMPTY0 / 2 || s / 2 == C_VF_FULL0 / 2)
                cnt = 128;  // warps 20..23 or 24..27
            else if (s >= C_REC_EMPTY0 && s < C_REC_EMPTY0 + kCsBatches)
                cnt = 27;   // every warp but the reader
            mbar_init(BAR(s), cnt);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmO);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);
    const uint32_t tS = tmem, tO = tmem + 256u, tP = tmem + 384u;
    const unsigned long long lim = a.wait_limit_ns;

    // Record of tile n (null on a timeout); every lane of a warp calls it for every tile, in order. A warp gives a batch
    // back after its last tile.
    auto record = [&](uint32_t n) -> const CsTile* {
        const uint32_t k = n / kCsBatch, sl = k % kCsBatches;
        if (n % kCsBatch == 0 && !cs_wait(BAR(C_REC_FULL0 + sl), (k / kCsBatches) & 1u, lim)) return nullptr;
        return &recs[sl * kCsBatch + n % kCsBatch];
    };
    auto release = [&](uint32_t n) {
        if (n % kCsBatch == kCsBatch - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C_REC_EMPTY0 + (n / kCsBatch) % kCsBatches));
        }
    };

    // Registers: 384 x 40 + 512 x 96 is what 896 x 72 were launched with.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;" ::: "memory");
        if (warp == 3) {
            // ------------------------------------------------------------------------------------------ reader
            uint32_t bad = 0;
            int r = 0;                       // next round
            int w_id = -1, w_begin = 0, w_count = 0;  // this lane's item of the current window of 32 rounds
            int id = 0, begin = 0, count = 0, tiles = 0, t = 0;  // the current item
            int items = -1;                  // its number
            bool ended = false, seen = false;  // seen: both parities of tiles have an end record
            for (uint32_t k = 0; !seen; ++k) {
                const uint32_t sl = k % kCsBatches;
                if (!cs_wait(BAR(C_REC_EMPTY0 + sl), ((k / kCsBatches) & 1u) ^ 1u, lim)) break;
                int m_id = 0, m_begin = 0, m_count = 0, m_t = 0, m_flags = -1, m_item = 0;  // tile `lane` of the batch
                seen = ended;
                for (int i = 0; i < kCsBatch && !ended; ++i) {
                    while (t == tiles && !ended) {  // next item
                        if ((r & 31) == 0) {
                            const int rr = r + (int)lane, G = gridDim.x, b = blockIdx.x;
                            const int64_t w = (int64_t)rr * G + ((rr & 1) ? (G - 1 - b) : b);
                            w_id = -1;
                            w_count = 0;
                            if (w < a.n_items) {
                                w_id = a.order ? a.order[w] : (int)w;
                                if (w_id < 0 || w_id >= a.n_items) {
                                    bad = 1;
                                    w_id = -2;  // not an item: skipped
                                } else {
                                    // reported here: an item without entries has no tile that would look at its length
                                    const int len = a.g.lens[w_id / a.nq / a.heads], room = a.g.table_stride * a.g.page;
                                    if (len < 0 || len > room) bad = 1;
                                    if (a.indptr) {
                                        w_begin = a.indptr[w_id];
                                        w_count = a.indptr[w_id + 1] - w_begin;
                                        if (w_count < 0 || w_begin < 0) {
                                            bad = 1;
                                            w_count = 0;
                                        }
                                    } else {
                                        w_begin = 0;
                                        w_count = (min(max(len, 0), room) + a.g.page - 1) / a.g.page;
                                    }
                                }
                            }
                        }
                        id = __shfl_sync(0xffffffffu, w_id, r & 31);
                        begin = __shfl_sync(0xffffffffu, w_begin, r & 31);
                        count = __shfl_sync(0xffffffffu, w_count, r & 31);
                        ++r;
                        t = 0;
                        tiles = id == -2 ? 0 : max(1, (count + a.sub - 1) / a.sub);  // an empty list still writes its rows
                        if (tiles > 0) ++items;
                        if (id == -1) {
                            ended = true;
                            seen = i < kCsBatch - 1;
                        }
                    }
                    if ((int)lane == i && !ended) {
                        m_id = id;
                        m_begin = begin;
                        m_count = count;
                        m_t = t;
                        m_flags = (t == 0 ? kCsFirst : 0) | (t == 1 ? kCsSecond : 0) | (t == tiles - 2 ? kCsPre : 0) |
                                  (t == tiles - 1 ? kCsLast : 0);
                        m_item = items;
                    }
                    ++t;
                }
                const int src = (int)lane >> 2, g = (int)lane & 3;
                const int q_id = __shfl_sync(0xffffffffu, m_id, src), q_begin = __shfl_sync(0xffffffffu, m_begin, src);
                const int q_count = __shfl_sync(0xffffffffu, m_count, src), q_t = __shfl_sync(0xffffffffu, m_t, src);
                const int q_flags = __shfl_sync(0xffffffffu, m_flags, src), q_item = __shfl_sync(0xffffffffu, m_item, src);
                const int h = q_id / a.nq, seq = h / a.heads, kvh = (h - seq * a.heads) / a.group;
                int valid = 0, row = 0;
                float ks = 1.0f, vs = 1.0f;
                const int e = q_t * a.sub + ((g * a.sub) >> 2);
                if (q_flags >= 0 && e < q_count) {
                    const int off = (g & (4 / a.sub - 1)) * 32;
                    const int j = a.indptr ? a.kv_idx[q_begin + e] : e;
                    const int64_t len = min(max(a.g.lens[seq], 0), a.g.table_stride * a.g.page);
                    if (j < 0 || j >= a.g.table_stride) {
                        bad = 1;
                    } else {
                        valid = (int)min((int64_t)32, max((int64_t)0, len - ((int64_t)j * a.g.page + off)));
                        if (valid > 0) {
                            const int page = a.g.table[(int64_t)seq * a.g.table_stride + j];
                            if (page < 0 || page >= a.g.n_pages) {
                                bad = 1;
                                valid = 0;
                            } else {
                                const int64_t ph = (int64_t)page * a.g.kv_heads + kvh;
                                row = (int)(ph * a.g.page) + off;
                                ks = a.k_scale[ph];
                                vs = fmaxf(a.v_scale[ph], 1e-30f);
                            }
                        }
                    }
                }
                CsTile* const rec = &recs[sl * kCsBatch + src];
                rec->row[g] = row;
                rec->ks[g] = ks;
                rec->lv[g] = __log2f(vs);
                rec->iv[g] = 1.0f / vs;
                reinterpret_cast<uint8_t*>(&rec->kv4)[g] = (uint8_t)valid;
                if (g == 0) {
                    rec->qrow = h * a.Np + (q_id - h * a.nq) * kTcRows;
                    rec->flags = q_flags;
                    rec->item = q_item;
                    if (q_flags >= 0 && (q_flags & kCsFirst))  // warps 24..27 read it some tiles from now
                        l2_prefetch(a.q + (size_t)rec->qrow * kTcDim, kTileBytes);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(C_REC_FULL0 + sl));
            }
            if (bad) atomicOr(&g_device_error, kDevErrBadData);
        } else if (warp == 0 || warp == 2) {
            // ------------------------------------------------------------------------- TMA: K codes, V codes
            const bool keys = warp == 0;
            const uint64_t pol = l2_policy_evict_last();
            const uint32_t stages = keys ? kCsKStages : 2u;
            const uint32_t full = keys ? C_K_FULL0 : C_V8_FULL0, empty = keys ? C_K_EMPTY0 : C_V8_EMPTY0;
            const uint32_t ring = base + (keys ? kCsK : kCsV8);
            uint32_t n = 0, filled = 0;
            for (;; ++n) {
                const CsTile* const rec = record(n);
                if (!rec || rec->flags < 0) break;
                const uint32_t s = n % stages;
                if (!cs_wait(BAR(empty + s), ((n / stages) & 1u) ^ 1u, lim)) break;
                if (lane == 0) mbar_arrive_expect_tx(BAR(full + s), kCsTile8);
                __syncwarp();
                if (lane < 4)
                    tma_load_2d_hint(ring + s * kCsTile8 + lane * 4096u, keys ? &tmK : &tmV, 0, rec->row[lane],
                                     BAR(full + s), pol);
                filled = n + 1;
                release(n);
            }
            for (uint32_t i = 1; i <= stages && i <= filled; ++i) {  // copies in flight land before the CTA ends
                const uint32_t x = filled - i;
                wait_bounded(BAR(full + x % stages), (x / stages) & 1u, kDrainLimitNs);
            }
            __syncwarp();
        } else {
            // ---------------------------------------------------------------------------------- MMA issuer
            constexpr uint32_t kIdQK = idesc_fmt0_f32(128, 128, false);
            constexpr uint32_t kIdPV = idesc_fmt0_f32(128, 128, true);
            const uint64_t dQ0 = smem_desc(base + kCsQ, 16, 1024), dK0 = smem_desc(base + kCsK, 16, 1024);
            const uint64_t dV0 = smem_desc(base + kCsVf, kBoxBytes, 1024);
            uint32_t n = 0, items = 0, pv = 0, pv_items = 0;  // Q K^T and P V issued so far, and their items
            uint32_t firsts = 0;                              // bit n & 31: tile n is the first of its item
            auto issue_pv = [&]() -> bool {  // tile pv
                const uint32_t b = pv & 1u, par = (pv >> 1) & 1u;
                const bool first = (firsts >> (pv & 31u)) & 1u;
                if (!cs_wait2(BAR(C_P_FULL0 + b), par, BAR(C_VF_FULL0 + b), par, lim)) return false;
                if (first) {
                    if (pv_items > 0 && !cs_wait(BAR(C_O_FREE), (pv_items - 1) & 1u, lim)) return false;
                    ++pv_items;
                }
                tc_fence_after();
                const uint64_t dV = dV0 + b * (kTileBytes >> 4);
#pragma unroll
                for (uint32_t kk = 0; kk < 8; ++kk)
                    el_mma_ts_f16(tO, tP + b * 64u + kk * 8u, dV + kk * 128u, kIdPV, (first && kk == 0) ? 0u : 1u);
                el_commit(BAR(C_PV_DONE0 + b));
                ++pv;
                return true;
            };
            bool ok = true;
            int flags = -1;
            auto look = [&](uint32_t x) -> bool {  // flags of tile x
                const CsTile* const rec = record(x);
                if (!rec) return false;
                flags = __shfl_sync(0xffffffffu, rec->flags, 0);
                release(x);
                return true;
            };
            for (ok = look(0); ok && flags >= 0; ++n) {
                const uint32_t first = flags & kCsFirst, last = flags & kCsLast;
                firsts = (firsts & ~(1u << (n & 31u))) | (first << (n & 31u));
                if (first) {
                    ++items;
                    if (!(ok = cs_wait(BAR(C_Q_FULL0 + ((items - 1) & 1u)), ((items - 1) >> 1) & 1u, lim))) break;
                }
                const uint32_t qs = (items - 1) & 1u, ks = n % kCsKStages, b = n & 1u;
                if (!(ok = cs_wait2(BAR(C_K_FULL0 + ks), (n / kCsKStages) & 1u, BAR(C_S_FREE0 + b), ((n >> 1) & 1u) ^ 1u, lim)))
                    break;
                tc_fence_after();
                const uint64_t dQ = dQ0 + qs * (2 * kCsTile8 >> 4), dK = dK0 + ks * (kCsTile8 >> 4);
#pragma unroll
                for (uint32_t kk = 0; kk < 8; ++kk)  // four steps of q1, four of q2, over the same K
                    el_mma_ss_f8(tS + b * 128u, dQ + (kk >> 2) * (kCsTile8 >> 4) + (kk & 3u) * 2u, dK + (kk & 3u) * 2u,
                                 kIdQK, kk ? 1u : 0u);
                el_commit(BAR(C_S_FULL0 + b));
                el_commit(BAR(C_K_EMPTY0 + ks));
                if (last) el_commit(BAR(C_Q_EMPTY0 + qs));
                if (!(ok = look(n + 1))) break;
                if (n >= 2 && !(ok = issue_pv())) break;
            }
            while (ok && pv < n) ok = issue_pv();
            el_commit(BAR(C_MMA_DONE));
            cs_wait(BAR(C_MMA_DONE), 0, kDrainLimitNs);
        }
    } else if (warp >= 24) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;" ::: "memory");
        // ----------------------------------------------------------------------------------------- Q split
        // Rows of the block as q1 + q2, swizzled like a TMA tile. Four lanes hold a row, 16 bytes of every 64; the eight
        // rows of a warp's step are ordered so that 16 lanes' 8-byte stores meet 16 different bank pairs.
        const uint32_t q4 = lane & 3u, r8 = (((lane >> 2) & 3u) << 1) | (lane >> 4);
        uint32_t items = 0;
        auto split_q = [&](int32_t qrow) -> bool {
            const uint32_t qs = items & 1u;
            if (!cs_wait(BAR(C_Q_EMPTY0 + qs), ((items >> 1) & 1u) ^ 1u, lim)) return false;
            const uint32_t dst = base + kCsQ + qs * 2 * kCsTile8;
#pragma unroll 1
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t row = (uint32_t)(warp - 24) * 32u + i * 8u + r8;
                const __nv_bfloat16* const src = a.q + ((size_t)qrow + row) * kTcDim + q4 * 8u;
                uint32_t u[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src + 32 * j));
                    u[4 * j] = w.x;
                    u[4 * j + 1] = w.y;
                    u[4 * j + 2] = w.z;
                    u[4 * j + 3] = w.w;
                }
                // magnitudes of bf16 order as integers; the two halves of a word are compared side by side
                uint32_t mx = 0;
#pragma unroll
                for (int j = 0; j < 16; ++j) mx = __vmaxu2(mx, u[j] & 0x7fff7fffu);
                mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float s = row_factor(max(mx & 0xffff0000u, mx << 16));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t c1[2], c2[2];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t v = u[4 * j + x];
                        const uint32_t h = pack_f16x2(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
                        const uint32_t q1 = e4m3x2_of_half2(h);
                        const uint32_t back = half2_of_e4m3x2(q1);
                        const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&h),
                                                     *reinterpret_cast<const __half2*>(&back));
                        const uint32_t q2 = e4m3x2_of_half2(*reinterpret_cast<const uint32_t*>(&rest));
                        c1[x >> 1] = x & 1 ? c1[x >> 1] | q1 << 16 : q1;
                        c2[x >> 1] = x & 1 ? c2[x >> 1] | q2 << 16 : q2;
                    }
                    const uint32_t piece = q4 + 4u * j;  // 8 bytes of the row
                    const uint32_t at = dst + row * 128u + ((((piece >> 1) ^ (row & 7u)) << 4) | (8u * (piece & 1u)));
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(c1[0]), "r"(c1[1]) : "memory");
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + kCsTile8), "r"(c2[0]), "r"(c2[1])
                                 : "memory");
                }
                // four items deep: item k's slot is written again for item k + 4, whose split waits for Q K^T of item
                // k + 2, which waited until item k's last S had been read
                // (of a row of NaN 1: hidden keys must stay -inf)
                if (q4 == 0) fac[(items & 3u) * 128u + row] = s == s ? 1.0f / s : 1.0f;
            }
            fence_proxy_async_smem();
            mbar_arrive(BAR(C_Q_FULL0 + qs));
            ++items;
            return true;
        };
        // The first item is known without its lists, pages and scales: its rows need not wait for the first records.
        const int id0 = a.order ? a.order[blockIdx.x] : (int)blockIdx.x;
        const bool early = id0 >= 0 && id0 < a.n_items;  // else the reader skips it
        bool ok = !early || split_q((id0 / a.nq) * a.Np + id0 % a.nq * kTcRows);
        for (uint32_t n = 0; ok; ++n) {
            const CsTile* const rec = record(n);
            if (!rec || rec->flags < 0) break;
            const bool split = (rec->flags & kCsFirst) && !(early && rec->item == 0);
            const int32_t qrow = rec->qrow;
            release(n);
            if (split) ok = split_q(qrow);
        }
    } else if (warp >= 20) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;" ::: "memory");
        // ----------------------------------------------------------------------------- V widening, O stores
        const int wt = warp - 20;
        bool fin[2] = {false, false};
        int32_t fin_row[2] = {0, 0};
        uint32_t staged[2] = {0, 0}, flushed[2] = {0, 0};
        // The O staged in slot sl leaves for global memory; returns once the slot has been read.
        auto flush = [&](uint32_t sl) -> bool {
            if (!cs_wait(BAR(C_STAGED0 + sl), staged[sl] & 1u, lim)) return false;
            ++staged[sl];
            if (warp == 20 && lane == 0) {
                tma_store_2d(&tmO, base + kCsVf + sl * kTileBytes, 0, fin_row[sl]);
                tma_store_2d(&tmO, base + kCsVf + sl * kTileBytes + kBoxBytes, 64, fin_row[sl]);
                bulk_commit_group();
                bulk_wait_read_all();
                mbar_arrive(BAR(C_FLUSHED0 + sl));
            }
            __syncwarp();
            if (!cs_wait(BAR(C_FLUSHED0 + sl), flushed[sl] & 1u, lim)) return false;
            ++flushed[sl];
            fin[sl] = false;
            return true;
        };
        // Warp wt widens quarter wt. Eight lanes take four 16-byte pieces of two rows r and r ^ 5: in the swizzled tile of
        // codes and in the swizzled fp16 tile alike they meet eight different bank groups.
        const uint32_t c16 = (lane & 3u) | ((lane >> 3) & 1u) << 2;  // 16 dimensions of a key row
        const uint32_t r0 = (lane >> 4) ^ ((lane & 4u) ? 5u : 0u), r1 = r0 ^ 2u;  // rows of an 8-row group
        bool ok = true;
        uint32_t n = 0;
        for (;; ++n) {
            const CsTile* const rec = record(n);
            if (!(ok = rec != nullptr) || rec->flags < 0) break;
            const bool last = rec->flags & kCsLast;
            const uint32_t have = (rec->kv4 >> (8 * wt)) & 255u;
            const int32_t qrow = rec->qrow;
            release(n);
            const uint32_t b = n & 1u, par = (n >> 1) & 1u;
            if (n >= 2) {
                if (fin[b]) ok = flush(b);
                else ok = cs_wait(BAR(C_PV_DONE0 + b), ((n - 2) >> 1) & 1u, lim);
                if (!ok) break;
            }
            if (!(ok = cs_wait(BAR(C_V8_FULL0 + b), par, lim))) break;
            const uint32_t src = base + kCsV8 + b * kCsTile8 + wt * 4096u;
            const uint32_t dst = base + kCsVf + b * kTileBytes + (c16 >> 2) * kBoxBytes + wt * 4096u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t r = i & 1 ? r1 : r0, at = (uint32_t)(i >> 1) * 1024u + r * 128u;
                uint4 w = ld_shared_v4(src + at + ((c16 ^ r) << 4));
                if (have < 32u && (uint32_t)(i >> 1) * 8u + r >= have) w = make_uint4(0, 0, 0, 0);
                const uint32_t j = 2u * (c16 & 3u);
                st_shared_v4(dst + at + ((j ^ r) << 4), half2_of_e4m3x2(w.x & 0xffffu), half2_of_e4m3x2(w.x >> 16),
                             half2_of_e4m3x2(w.y & 0xffffu), half2_of_e4m3x2(w.y >> 16));
                st_shared_v4(dst + at + (((j + 1u) ^ r) << 4), half2_of_e4m3x2(w.z & 0xffffu),
                             half2_of_e4m3x2(w.z >> 16), half2_of_e4m3x2(w.w & 0xffffu), half2_of_e4m3x2(w.w >> 16));
            }
            mbar_arrive(BAR(C_V8_EMPTY0 + b));
            fence_proxy_async_smem();
            mbar_arrive(BAR(C_VF_FULL0 + b));
            fin[b] = last;
            fin_row[b] = qrow;
        }
        for (uint32_t x = 0; ok && x < 2; ++x) {  // the last items' O, oldest slot first
            const uint32_t sl = (n + x) & 1u;
            if (fin[sl]) ok = flush(sl);
        }
        __syncwarp();  // flush has waited until the stores have read their slots; the grid's end waits for the rest
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 96;" ::: "memory");
        // ----------------------------------------------------------------------------- softmax warpgroups
        const uint32_t grp = (uint32_t)(warp - 4) >> 2;
        const uint32_t pair = grp >> 1, half = grp & 1u;  // tiles n with n & 1 == pair; keys 64 half .. 64 half + 63
        const uint32_t wl = (uint32_t)warp & 3u;
        const int row = (int)(wl * 32u + lane);
        const uint32_t lane_off = (wl * 32u) << 16;
        const uint32_t tSb = tS + pair * 128u + half * 64u + lane_off, tPb = tP + pair * 64u + half * 32u + lane_off;
        const uint32_t tOb = tO + half * 64u + lane_off;
        // A row's reference after a tile whose maximum is top: it moves when the row sees its first key, or when the
        // maximum exceeds it by more than 2^8. Every thread of a row follows it through all tiles by itself.
        auto moved = [](float m, float top) { return m == -INFINITY || top - m > 8.0f ? top : m; };
        float l = 0.0f, m = -INFINITY;  // this thread's share of the item's denominator, and its reference
        for (uint32_t n = pair;; n += 2) {
            const uint32_t k = n / kCsBatch, sl = k % kCsBatches;
            if (n % kCsBatch < 2 && !cs_wait(BAR(C_REC_FULL0 + sl), (k / kCsBatches) & 1u, lim)) break;
            const CsTile* const rec = &recs[sl * kCsBatch + n % kCsBatch];
            const int flags = rec->flags;
            if (flags < 0) break;
            const uint32_t item = (uint32_t)rec->item;
            const bool fresh = flags & (kCsFirst | kCsSecond);  // no tile of this item has come to this pair yet
            const uint32_t par = (n >> 1) & 1u;
            const int32_t qrow = rec->qrow;
            const uint32_t kv2 = (rec->kv4 >> (16 * half)) & 0xffffu;
            float ck[2], lv[2], iv[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                ck[x] = rec->ks[2 * half + x];
                lv[x] = rec->lv[2 * half + x];
                iv[x] = rec->iv[2 * half + x];
            }
            if (n % kCsBatch >= kCsBatch - 2) {  // this pair's last tile of the batch
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(C_REC_EMPTY0 + sl));
            }
            if (!cs_wait(BAR(C_S_FULL0 + pair), par, lim)) break;
            tc_fence_after();
            float s[64];
            tmem_ld32(tSb, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
            tmem_ld32(tSb + 32u, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
            // the row's factor was written before Q K^T could start
            const float c = a.scale_log2 * fac[(item & 3u) * 128u + (uint32_t)row];
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(BAR(C_S_FREE0 + pair));
            if (kv2 != 0x2020u) {  // keys that do not exist become -inf, whatever their codes gave
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    s[e] = (uint32_t)(e & 31) < ((kv2 >> (8 * (e >> 5))) & 255u) ? s[e] : -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float* const z = s + 32 * x;
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmax3(z[e], z[4 + e], z[8 + e]);
#pragma unroll
                for (int y = 12; y < 28; y += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmax3(mx[e], z[y + e], z[y + 4 + e]);
                const float q = fmaxf(fmax3(mx[0], mx[1], fmaxf(z[28], z[29])), fmax3(mx[2], mx[3], fmaxf(z[30], z[31])));
                // at least the smallest normal number: -inf times a factor that rounds to zero (a quiet row on a block of
                // zero keys, whose scale is 2^-40) would be NaN
                ck[x] *= c;
                ck[x] = ck[x] < 1.17549435e-38f ? 1.17549435e-38f : ck[x];
                top = fmaxf(top, fmaf(q, ck[x], lv[x]));
            }
            // The tile before first, then this one: a pair that published a tile before it had seen the other's could run
            // two phases ahead of a reader.
            if (n > 0 && !cs_wait(BAR(C_M_READY0 + (pair ^ 1u)), ((n - 1) >> 1) & 1u, lim)) break;
            float* const at = tops + (n & 3u) * 256u + (uint32_t)row;
            at[half * 128u] = top;
            mbar_arrive(BAR(C_M_READY0 + pair));
            float before = -INFINITY;
            if (!(flags & kCsFirst)) {
                const float* const was = tops + ((n - 1) & 3u) * 256u + (uint32_t)row;
                before = moved(fresh ? -INFINITY : m, fmaxf(was[0], was[128]));
            }
            if (!cs_wait(BAR(C_M_READY0 + pair), par, lim)) break;
            const float now = moved(before, fmaxf(top, at[(half ^ 1u) * 128u]));
            if (fresh) l = 0.0f;
            else if (now != m) l *= m == -INFINITY ? 0.0f : ex2_approx(m - now);
            const bool rescale = !(flags & kCsFirst) && now != before && before != -INFINITY;
            m = now;
            const float ref = m == -INFINITY ? 0.0f : kCsBias - m;
            // P's buffer was last read by P V of this pair's tile before
            if (n >= 2 && !cs_wait(BAR(C_PV_DONE0 + pair), ((n - 2) >> 1) & 1u, lim)) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float off = lv[x] + ref;
                const uint64_t c2 = f2_pack(ck[x], ck[x]), o2 = f2_pack(off, off);
                uint64_t l2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                uint32_t pw[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint64_t xx = f2_fma(f2_pack(s[32 * x + 2 * e], s[32 * x + 2 * e + 1]), c2, o2);
                    float x0, x1;
                    f2_unpack(xx, x0, x1);
                    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                    pw[e] = pack_f16x2(p0, p1);
                    l2[e & 1] = f2_add(l2[e & 1], f2_pack(p0, p1));
                }
                float la, lb, lc, ld;
                f2_unpack(l2[0], la, lb);
                f2_unpack(l2[1], lc, ld);
                l = fmaf((la + lb) + (lc + ld), iv[x], l);
                tmem_st16(tPb + 16u * x, pw);
            }
            // O is rescaled once P V of tile n - 1 has added to it
            if (__any_sync(0xffffffffu, rescale)) {
                if (!cs_wait(BAR(C_PV_DONE0 + (pair ^ 1u)), ((n - 1) >> 1) & 1u, lim)) break;
                tc_fence_after();
                const float alpha = rescale ? ex2_approx(before - now) : 1.0f;
#pragma unroll 1
                for (uint32_t ch = 0; ch < 2; ++ch) {
                    uint32_t ov[32];
                    tmem_ld32(tOb + ch * 32u, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                    tmem_st32(tOb + ch * 32u, ov);
                }
            }
            float2* const den = dens + (item & 1u) * 512u + (uint32_t)row;
            if (flags & (kCsPre | kCsLast)) den[grp * 128u] = make_float2(l, m);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(BAR(C_P_FULL0 + pair));
            if (!(flags & kCsLast)) continue;
            // Epilogue: the item's last P V. The other groups' shares were written before the P that it waited for.
            if (!cs_wait(BAR(C_PV_DONE0 + pair), par, lim)) break;
            tc_fence_after();
            l += den[(grp ^ 1u) * 128u].x;
            if (!(flags & kCsFirst)) {
                const float2 o0 = den[(2u * (pair ^ 1u)) * 128u], o1 = den[(2u * (pair ^ 1u) + 1u) * 128u];
                l += o0.y == -INFINITY ? 0.0f : (o0.x + o1.x) * ex2_approx(o0.y - m);
            }
            const float inv_l = l == 0.0f ? 0.0f : 1.0f / l;  // a row that saw no key gives zeros
            uint32_t ov[2][32];
            tmem_ld32(tOb, ov[0]);
            tmem_ld32(tOb + 32u, ov[1]);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(BAR(C_O_FREE));
            const uint32_t stage = base + kCsVf + pair * kTileBytes + half * kBoxBytes + (uint32_t)row * 128u;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const uint32_t j = (uint32_t)(x * 4 + q4);
                    uint32_t w[4];
#pragma unroll
                    for (int k2 = 0; k2 < 4; ++k2)
                        w[k2] = pack_bf16x2(__uint_as_float(ov[x][q4 * 8 + 2 * k2]) * inv_l,
                                            __uint_as_float(ov[x][q4 * 8 + 2 * k2 + 1]) * inv_l);
                    st_shared_v4(stage + ((j ^ ((uint32_t)row & 7u)) << 4), w[0], w[1], w[2], w[3]);
                }
            fence_proxy_async_smem();
            mbar_arrive(BAR(C_STAGED0 + pair));
            if (a.lse && half == 0)
                a.lse[(size_t)qrow + row] = l == 0.0f ? -INFINITY : (m - kCsBias + lg2_approx(l)) * 0.6931471805599453f;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace losa
