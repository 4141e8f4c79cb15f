// Host side of the streaming operators (rotary positions, the paged 8-bit cache and attention over it): argument checks
// and launches. Included once, by losa.cu, after its shared helpers.
#pragma once

namespace {

bool rope_ok(const losa_rope* r, int head_dim) {
    if (!r || r->head_dim != head_dim || head_dim > 2 * kRopeMaxPairs) return false;
    int64_t sum = 0;
    for (int a = 0; a < 3; ++a) {
        if (r->axis_dims[a] < 0 || (r->axis_dims[a] & 1)) return false;
        sum += r->axis_dims[a];
    }
    if (sum > head_dim || r->grid_y < 1 || r->grid_x < 1) return false;
    if (r->pairing != LOSA_ROPE_INTERLEAVED && r->pairing != LOSA_ROPE_HALVES) return false;
    return std::isfinite(r->theta) && r->theta > 0.0;
}

// Turns per unit of position of every pair, as fractions of 2^64. One power per axis, then i products for pair i, in 64-bit
// mantissas: f is off by i (2^-63 + 2^-64) of itself at most (the power's last place and a rounding each), which for 127
// products of at most 1 / (2 pi min(theta, 1)) is below 2^-58 / min(theta, 1); for theta = 10000 and 64 pairs, whose f shrinks
// meanwhile, below 3 units of 2^-64.
RopeArgs rope_args(const losa_rope* r) {
    RopeArgs a;
    a.gy = r->grid_y;
    a.gx = r->grid_x;
    int at = 0;
    const long double inv_two_pi = 0.15915494309189533576888376337251436L;
    for (int ax = 0; ax < 3; ++ax) {
        const int m = r->axis_dims[ax];
        a.half[ax] = m / 2;
        a.off[ax] = r->offset[ax];
        const long double ratio = m ? powl((long double)r->theta, -2.0L / m) : 1.0L;
        long double f = inv_two_pi;
        for (int i = 0; i < m / 2; ++i, f *= ratio) {
            const long double turns = f < 1.0L ? f : f - floorl(f);  // theta < 1 turns by more than one
            const long double fixed = turns * 18446744073709551616.0L + 0.5L;
            a.step[at / 2 + i] = fixed >= 18446744073709551616.0L ? 0ull : (uint64_t)fixed;
        }
        at += m;
        a.end[ax] = at;
    }
    return a;
}

// One side of a rotation: positive extents, strides that keep every 16-byte piece aligned.
bool view_ok(const losa_token_view* v, int head_dim, int size, bool written) {
    if (!v || v->parts < 1 || v->batch < 1 || v->heads < 1 || v->tokens < 0) return false;
    if (v->tokens == 0) return true;  // nothing is read or written through it
    const int64_t s[4] = {v->part_stride, v->batch_stride, v->token_stride, v->head_stride};
    const int32_t n[4] = {v->parts, v->batch, v->tokens, v->heads};
    for (int i = 0; i < 4; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < 0 || (s[i] * size) % 16 != 0) return false;
        if (written && s[i] < head_dim) return false;  // rows that overlap
    }
    return true;
}

bool cache_ok(const losa_cache* c) {
    return c && c->kv_heads > 0 && c->n_pages > 0 && c->seqs > 0 && c->table_stride > 0 && c->head_dim > 0 &&
           c->page_tokens > 0 && (int64_t)c->table_stride * c->page_tokens <= 2147483647ll - 128;
}

// Shapes the cache kernels exist for: TMA addresses the pool's rows with 32-bit coordinates.
bool cache_supported(const losa_cache* c) {
    return (c->head_dim == 64 || c->head_dim == 128) &&
           (c->page_tokens == 32 || c->page_tokens == 64 || c->page_tokens == 128) && c->seqs <= 65535 &&
           c->kv_heads <= 65535 && (int64_t)c->n_pages * c->kv_heads <= 2147483647ll / c->page_tokens;
}

bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

CacheGeom cache_geom(const losa_cache* c, const int32_t* table, const int32_t* lens) {
    CacheGeom g;
    g.kv_heads = c->kv_heads;
    g.page = c->page_tokens;
    g.n_pages = c->n_pages;
    g.table_stride = c->table_stride;
    g.table = table;
    g.lens = lens;
    return g;
}

// Tensor map over the pool's codes as a [pages * kv heads * page tokens][d] byte matrix, boxes of box_rows whole rows,
// swizzled over the row (64 or 128 bytes).
bool make_code_map(CUtensorMap* map, const losa_cache* c, const void* codes, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t gdim[2] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->n_pages * c->kv_heads * c->page_tokens};
    const cuuint64_t gstride[1] = {(cuuint64_t)c->head_dim};
    const cuuint32_t box[2] = {(cuuint32_t)c->head_dim, box_rows};
    const cuuint32_t estride[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), gdim, gstride, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              c->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The halves pairing's unit (see rope.cuh): 4, 2 or 1; 0 for the interleaved pairing.
int rope_unit_width(const losa_rope* r) {
    if (!r || r->pairing != LOSA_ROPE_HALVES) return 0;
    const int all = (r->axis_dims[0] | r->axis_dims[1] | r->axis_dims[2]) / 2;
    return all % 4 == 0 ? 4 : (all % 2 == 0 ? 2 : 1);
}

template <typename T, int W>
losa_status launch_rope(const RopeApplyArgs& a, const void* x, void* y, dim3 grid, cudaStream_t stream) {
    rope_apply_kernel<T, W>
        <<<grid, kRopeThreads, 0, stream>>>(a, static_cast<const T*>(x), static_cast<T*>(y));
    return launch_status();
}

template <typename T, int D, int W>
losa_status launch_append(const AppendArgs& a, const void* k, const void* v, dim3 grid, int threads,
                          cudaStream_t stream) {
    cache_append_kernel<T, D, W><<<grid, threads, 0, stream>>>(a, static_cast<const T*>(k), static_cast<const T*>(v));
    return launch_status();
}

template <typename T, int D>
losa_status launch_append_width(int width, const AppendArgs& a, const void* k, const void* v, dim3 grid, int threads,
                                cudaStream_t stream) {
    return width == 4   ? launch_append<T, D, 4>(a, k, v, grid, threads, stream)
           : width == 2 ? launch_append<T, D, 2>(a, k, v, grid, threads, stream)
           : width == 1 ? launch_append<T, D, 1>(a, k, v, grid, threads, stream)
                        : launch_append<T, D, 0>(a, k, v, grid, threads, stream);
}

// Where every sequence is short (max_len), a CTA takes a unit and there is nothing to join: up to 1024 keys (12 kv heads, 1000
// keys: 10.3 against 16.4 us), and up to 2048 where the units fill half the SMs by themselves (16 streams of 8 kv heads, 2000
// keys: 15.7 against 18.5 us; with 32 units it is 15.4 against 14.4). Otherwise two CTAs per SM share all units' keys in equal
// ranges; a unit, at most 1 / (kv heads x row tiles) of the work, lies in at most CTAs / (kv heads x row tiles) + 2 of
// them, and in at most kCaMaxSplits (see ca_work).
struct AttnPlan {
    int tile_rows, tiles, splits, ctas;
    int64_t rows;
    size_t ml_bytes, total;
};

AttnPlan attn_plan(const losa_cache* c, int heads, int tokens, int max_len, int sms) {
    AttnPlan p;
    const int64_t rows = (int64_t)tokens * (heads / c->kv_heads);
    p.tile_rows = rows <= kCaRows<1> ? kCaRows<1> : kCaRows<2>;
    p.tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
    p.rows = (int64_t)c->seqs * tokens * heads;
    const int64_t units = (int64_t)c->kv_heads * p.tiles;
    const int64_t cap = (int64_t)c->table_stride * c->page_tokens;
    const int64_t len = max_len <= 0 || max_len > cap ? cap : max_len;
    p.ml_bytes = p.total = 0;
    p.splits = 0;
    p.ctas = (int)(units * c->seqs);
    const int64_t all = units * c->seqs;
    if (len <= (2 * all >= sms ? 2048 : 1024) || all > (1 << 20)) return p;
    p.ctas = kCaCtas * sms;
    int64_t s = (p.ctas + units - 1) / units + 2;
    if (s > kCaMaxSplits) s = kCaMaxSplits;
    p.splits = (int)s;
    p.ml_bytes = align256((size_t)p.rows * p.splits * sizeof(float2));
    p.total = p.ml_bytes + (size_t)p.rows * p.splits * c->head_dim * sizeof(float);
    return p;
}

bool attn_shape_ok(const losa_cache* c, int heads, int tokens) {
    return heads > 0 && heads % c->kv_heads == 0 && tokens > 0 && (int64_t)tokens * heads <= (1 << 24);
}

template <int D, int NB, int NW>
losa_status launch_cache_attn_warps(const losa_cache* c, CacheAttnArgs& a, const AttnPlan& p, const void* k8, const void* v8,
                              cudaStream_t stream) {
    CUtensorMap tk, tv;
    if (!make_code_map(&tk, c, k8, kCaKeys) || !make_code_map(&tv, c, v8, kCaKeys)) return LOSA_ERR_CUDA;
    if (cudaFuncSetAttribute(cache_attn_kernel<D, NB, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kCaSmem<D, NB, NW>) != cudaSuccess)
        return LOSA_ERR_CUDA;
    cache_attn_kernel<D, NB, NW><<<p.ctas, NW * 32, kCaSmem<D, NB, NW>, stream>>>(tk, tv, a);
    const losa_status st = launch_status();
    if (st != LOSA_OK || p.splits == 0) return st;
    // the join may be scheduled while the splits drain; it waits for their results itself
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, cache_join_kernel<D>, a, p.ctas) != cudaSuccess) return LOSA_ERR_CUDA;
    return launch_status();
}

// A CTA with a unit to itself and an SM to itself shares its tiles among more warps: a warp takes about 0.85 us for one.
template <int D, int NB>
losa_status launch_cache_attn(const losa_cache* c, CacheAttnArgs& a, const AttnPlan& p, const void* k8, const void* v8,
                              int sms, cudaStream_t stream) {
    return p.splits == 0 && p.ctas <= sms ? launch_cache_attn_warps<D, NB, kCaUnitWarps>(c, a, p, k8, v8, stream)
                                          : launch_cache_attn_warps<D, NB, kCaWarps>(c, a, p, k8, v8, stream);
}

}  // namespace

extern "C" {

losa_status losa_rope_apply(const losa_rope* rope, int32_t dtype, const losa_token_view* x_view, const void* x,
                            const losa_token_view* y_view, void* y, uint32_t rotate, int32_t inverse,
                            const int32_t* positions, const int32_t* start, cudaStream_t stream) {
    if (dtype != LOSA_DTYPE_BF16 && dtype != LOSA_DTYPE_F32) return LOSA_ERR_INVALID_ARG;
    if (!rope || rope->head_dim <= 0 || !rope_ok(rope, rope->head_dim)) return LOSA_ERR_INVALID_ARG;
    const int size = dtype == LOSA_DTYPE_BF16 ? 2 : 4;
    if (!view_ok(x_view, rope->head_dim, size, false) || !view_ok(y_view, rope->head_dim, size, true))
        return LOSA_ERR_INVALID_ARG;
    if (x_view->parts != y_view->parts || x_view->batch != y_view->batch || x_view->heads != y_view->heads ||
        y_view->tokens < x_view->tokens)
        return LOSA_ERR_INVALID_ARG;
    if ((x_view->tokens > 0 && !aligned16(x)) || (y_view->tokens > 0 && (!aligned16(y) || x == y)))
        return LOSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(start)) & 3u)
        return LOSA_ERR_INVALID_ARG;
    if ((rope->head_dim * size) % 16 != 0 || x_view->parts > 32 || x_view->batch > 65535 ||
        (int64_t)x_view->parts * x_view->heads > (1 << 24))
        return LOSA_ERR_UNSUPPORTED;
    if (y_view->tokens == 0) return LOSA_OK;
    RopeApplyArgs a;
    a.r = rope_args(rope);
    a.xs = {x_view->part_stride, x_view->batch_stride, x_view->token_stride, x_view->head_stride};
    a.ys = {y_view->part_stride, y_view->batch_stride, y_view->token_stride, y_view->head_stride};
    a.positions = positions;
    a.start = start;
    a.parts = x_view->parts;
    a.batch = x_view->batch;
    a.heads = x_view->heads;
    a.n = x_view->tokens;
    a.n_out = y_view->tokens;
    a.d = rope->head_dim;
    const int width = rope_unit_width(rope);
    a.units = width ? (a.d + 2 * width - 1) / (2 * width) : a.d * size / 16;
    a.rotate = rotate;
    a.sign = inverse ? -1.0f : 1.0f;
    // One CTA walks all rows of its tokens when the tokens alone fill the GPU four times over; fewer tokens are shared by
    // several CTAs, each with its own angles.
    const int64_t tokens_ctas = ((int64_t)a.n_out * a.units + kRopeThreads - 1) / kRopeThreads;
    const int sms = sm_count();
    if (sms <= 0) return LOSA_ERR_CUDA;
    const int rows = a.parts * a.heads;
    int64_t groups = (4 * (int64_t)sms + tokens_ctas * a.batch - 1) / (tokens_ctas * a.batch);
    groups = groups < 1 ? 1 : (groups > rows ? rows : groups);
    a.per_cta = (int)((rows + groups - 1) / groups);
    const dim3 grid((unsigned)tokens_ctas, (unsigned)((rows + a.per_cta - 1) / a.per_cta), (unsigned)a.batch);
    if (grid.y > 65535u) return LOSA_ERR_UNSUPPORTED;
#define LOSA_ROPE(T)                                                       \
    (width == 4   ? launch_rope<T, 4>(a, x, y, grid, stream)               \
     : width == 2 ? launch_rope<T, 2>(a, x, y, grid, stream)               \
     : width == 1 ? launch_rope<T, 1>(a, x, y, grid, stream)               \
                  : launch_rope<T, 0>(a, x, y, grid, stream))
    return dtype == LOSA_DTYPE_BF16 ? LOSA_ROPE(__nv_bfloat16) : LOSA_ROPE(float);
#undef LOSA_ROPE
}

losa_status losa_cache_append(const losa_cache* cache, const losa_rope* rope, int32_t dtype, const void* k,
                              int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                              int64_t v_head_stride, int64_t total_tokens, int32_t new_tokens, const int32_t* indptr,
                              const int32_t* positions, const int32_t* page_table, const int32_t* lens,
                              int32_t* new_lens, void* k8, void* v8, float* k_scale, float* v_scale,
                              cudaStream_t stream) {
    if (!cache_ok(cache) || (rope && !rope_ok(rope, cache->head_dim))) return LOSA_ERR_INVALID_ARG;
    if (dtype != LOSA_DTYPE_BF16 && dtype != LOSA_DTYPE_F32) return LOSA_ERR_INVALID_ARG;
    if (new_tokens < 0 || total_tokens < 0 || (!indptr && (int64_t)new_tokens * cache->seqs > total_tokens))
        return LOSA_ERR_INVALID_ARG;
    const int size = dtype == LOSA_DTYPE_BF16 ? 2 : 4;
    const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    const int64_t counts[2] = {total_tokens, cache->kv_heads};
    for (int i = 0; i < 4; ++i)  // nothing steps by the stride of an extent of one
        if (counts[i % 2] > 1 && (strides[i] < 0 || (strides[i] * size) % 16 != 0)) return LOSA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!aligned16(k) || !aligned16(v))) return LOSA_ERR_INVALID_ARG;
    if (!aligned16(k8) || !aligned16(v8) || !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(page_table) ||
        !aligned4(lens) || lens == new_lens)
        return LOSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(indptr) | reinterpret_cast<uintptr_t>(positions) |
         reinterpret_cast<uintptr_t>(new_lens)) & 3u)
        return LOSA_ERR_INVALID_ARG;
    if (!cache_supported(cache)) return LOSA_ERR_UNSUPPORTED;
    AppendArgs a;
    if (rope) a.r = rope_args(rope);
    a.g = cache_geom(cache, page_table, lens);
    a.positions = positions;
    a.indptr = indptr;
    a.new_lens = new_lens;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.total = total_tokens;
    a.new_tokens = new_tokens;
    const int C = cache->page_tokens;
    int64_t spans = ((int64_t)new_tokens + 2 * C - 2) / C;
    if (spans > cache->table_stride) spans = cache->table_stride;
    if (spans < 1) spans = 1;
    a.spans = (int)spans;
    a.rotate = rope ? 1 : 0;
    a.code[0] = static_cast<uint8_t*>(k8);
    a.code[1] = static_cast<uint8_t*>(v8);
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    if (spans * cache->seqs > 2147483647ll) return LOSA_ERR_UNSUPPORTED;
    // A CTA computes its page's angles once for all its heads; heads are spread over CTAs only as far as the pages leave
    // SMs idle (keys and values have CTAs of their own).
    const int sms = sm_count();
    if (sms <= 0) return LOSA_ERR_CUDA;
    int64_t groups = ((int64_t)sms + spans * cache->seqs - 1) / (spans * cache->seqs);
    groups = groups < 1 ? 1 : (groups > cache->kv_heads ? cache->kv_heads : groups);
    a.heads_per_cta = (int)((cache->kv_heads + groups - 1) / groups);
    const dim3 grid((unsigned)(spans * cache->seqs),
                    (unsigned)((cache->kv_heads + a.heads_per_cta - 1) / a.heads_per_cta), 2);
    // 16 dimensions a thread: as many warps as the new rows of one page need
    const int rows = new_tokens < C ? (new_tokens > 0 ? new_tokens : 1) : C;
    const int threads = ((rows * cache->head_dim / kAppendDims + 127) / 128) * 128;
    const int width = rope_unit_width(rope);
    if (dtype == LOSA_DTYPE_BF16)
        return cache->head_dim == 128 ? launch_append_width<__nv_bfloat16, 128>(width, a, k, v, grid, threads, stream)
                                      : launch_append_width<__nv_bfloat16, 64>(width, a, k, v, grid, threads, stream);
    return cache->head_dim == 128 ? launch_append_width<float, 128>(width, a, k, v, grid, threads, stream)
                                  : launch_append_width<float, 64>(width, a, k, v, grid, threads, stream);
}

size_t losa_cache_attn_workspace_bytes(const losa_cache* cache, int32_t heads, int32_t tokens, int32_t max_len) {
    if (!cache_ok(cache) || !cache_supported(cache) || !attn_shape_ok(cache, heads, tokens)) return 0;
    const int sms = sm_count();
    return sms > 0 ? attn_plan(cache, heads, tokens, max_len, sms).total : 0;
}

losa_status losa_cache_attn(const losa_cache* cache, int32_t heads, int32_t tokens, int32_t causal, const void* q,
                            int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                            const int32_t* page_table, const int32_t* lens, const void* k8, const void* v8,
                            const float* k_scale, const float* v_scale, float scale, int32_t max_len, void* o,
                            int64_t o_seq_stride, int64_t o_token_stride, int64_t o_head_stride, float* lse,
                            void* workspace, size_t ws_bytes, cudaStream_t stream) {
    if (!cache_ok(cache) || !attn_shape_ok(cache, heads, tokens)) return LOSA_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return LOSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !aligned16(k8) || !aligned16(v8) || !aligned4(k_scale) || !aligned4(v_scale) ||
        !aligned4(page_table) || !aligned4(lens) || (lse && !aligned4(lse)) || q == o)
        return LOSA_ERR_INVALID_ARG;
    const int64_t strides[6] = {q_seq_stride, q_token_stride, q_head_stride, o_seq_stride, o_token_stride, o_head_stride};
    const int32_t counts[3] = {cache->seqs, tokens, heads};
    for (int i = 0; i < 6; ++i) {
        if (counts[i % 3] <= 1) continue;
        if (strides[i] < 0 || strides[i] % 8 != 0 || (i >= 3 && strides[i] < cache->head_dim))
            return LOSA_ERR_INVALID_ARG;
    }
    if (!cache_supported(cache)) return LOSA_ERR_UNSUPPORTED;
    const int sms = sm_count();
    if (sms <= 0) return LOSA_ERR_CUDA;
    const AttnPlan p = attn_plan(cache, heads, tokens, max_len, sms);
    if ((int64_t)cache->kv_heads * p.tiles * cache->seqs > 2147483647ll) return LOSA_ERR_UNSUPPORTED;
    if (p.total > 0) {
        if (!aligned16(workspace)) return LOSA_ERR_INVALID_ARG;
        if (ws_bytes < p.total) return LOSA_ERR_CAPACITY;
    }
    CacheAttnArgs a;
    a.g = cache_geom(cache, page_table, lens);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.v8 = static_cast<const uint8_t*>(v8);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.q_seq = q_seq_stride;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.o_seq = o_seq_stride;
    a.o_token = o_token_stride;
    a.o_head = o_head_stride;
    a.heads = heads;
    a.group = heads / cache->kv_heads;
    a.tokens = tokens;
    a.causal = causal ? 1 : 0;
    a.tiles = p.tiles;
    a.splits = p.splits;
    a.seqs = cache->seqs;
    a.tile_rows = p.tile_rows;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.part_ml = static_cast<float2*>(workspace);
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.ml_bytes);
    a.wait_limit_ns = g_wait_limit_ns;
    if (p.tile_rows == kCaRows<1>)
        return cache->head_dim == 128 ? launch_cache_attn<128, 1>(cache, a, p, k8, v8, sms, stream)
                                      : launch_cache_attn<64, 1>(cache, a, p, k8, v8, sms, stream);
    return cache->head_dim == 128 ? launch_cache_attn<128, 2>(cache, a, p, k8, v8, sms, stream)
                                  : launch_cache_attn<64, 2>(cache, a, p, k8, v8, sms, stream);
}

losa_status losa_cache_sparse_attn(const losa_shape* shape, const losa_cache* cache, const void* q,
                                   const int32_t* page_table, const int32_t* lens, const void* k8, const void* v8,
                                   const float* k_scale, const float* v_scale, float scale, const int32_t* indptr,
                                   const int32_t* kv_block_idx, const int32_t* order, void* o, float* lse,
                                   cudaStream_t stream) {
    const losa_status st = check_shape(shape);
    if (st != LOSA_OK) return st;
    if (!cache_ok(cache) || shape->head_dim != cache->head_dim || shape->block_k != cache->page_tokens ||
        shape->heads % cache->seqs != 0 || (shape->heads / cache->seqs) % cache->kv_heads != 0)
        return LOSA_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !std::isfinite(scale) || (indptr == nullptr) != (kv_block_idx == nullptr))
        return LOSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !aligned16(k8) || !aligned16(v8) || !aligned4(k_scale) || !aligned4(v_scale) ||
        !aligned4(page_table) || !aligned4(lens) || (lse && !aligned16(lse)) || q == o)
        return LOSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(indptr) | reinterpret_cast<uintptr_t>(kv_block_idx) |
         reinterpret_cast<uintptr_t>(order)) & 3u)
        return LOSA_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)shape->heads * shape->n_padded;
    if (shape->dtype != LOSA_DTYPE_BF16 || shape->head_dim != kTcDim || shape->block_q != kTcRows ||
        !cache_supported(cache) || rows > 2147483647ll)
        return LOSA_ERR_UNSUPPORTED;
    CUtensorMap tk, tv, to;
    if (!make_code_map(&tk, cache, k8, 32) || !make_code_map(&tv, cache, v8, 32) ||
        !make_tile_map(&to, o, (uint64_t)rows))
        return LOSA_ERR_CUDA;
    CacheSparseArgs a;
    a.g = cache_geom(cache, page_table, lens);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.lse = lse;
    a.heads = shape->heads / cache->seqs;
    a.group = a.heads / cache->kv_heads;
    a.Np = shape->n_padded;
    a.nq = shape->n_padded / kTcRows;
    a.n_items = shape->heads * a.nq;
    a.sub = kTcRows / cache->page_tokens;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.indptr = indptr;
    a.kv_idx = kv_block_idx;
    a.order = order;
    a.wait_limit_ns = g_wait_limit_ns;
    const int sms = sm_count();
    if (sms <= 0) return LOSA_ERR_CUDA;
    if (cudaFuncSetAttribute(cache_sparse_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kCsSmem) !=
        cudaSuccess)
        return LOSA_ERR_CUDA;
    cache_sparse_kernel<<<a.n_items < sms ? a.n_items : sms, kCsThreads, kCsSmem, stream>>>(tk, tv, to, a);
    return launch_status();
}

}  // extern "C"
