"""Rotary positions, the paged 8-bit cache and attention over it against plain 64-bit forms.

Tolerances. A value rounded once to type t is off by at most eps(t) / 2 of it: 2^-8 for bf16 (2^-9 of its binade's top),
2^-24 for fp32.
  * rotation: cosine and sine in fp32 (the angle to 2^-32 of a turn, sincospif to 2 ulp) and two products: at most
    6 * 2^-24 of |a| + |b|, then the rounding to the type;
  * codes: a value within 1e-5 of a rounding border (relative) may fall on either side; every other code is exact;
  * attention: weights rounded to fp16 (2^-11 each, either side of the quotient) and the output rounded to bf16:
    |dO| <= 2^-8 |O| + 2^-10 sum_j p_j |v_j|; lse: fp32 sums of products, 1e-4, and for large logits what a sum of 256
    fp32 products (two terms for each of 128 dimensions) can be off by, 256 * 2^-24 |lse|."""
import math

import pytest
import torch

import free_block_sparse_losa_b200 as L
from tests.gpu_util import require_gpu

TOP = 448.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def grid_positions(n, gy, gx, device="cuda"):
    n = torch.as_tensor(n, device=device).long()
    return torch.stack([n // (gy * gx), n // gx % gy, n % gx], -1)


def turn(x, pos, dims, halves, inverse=False, theta=10000.0):
    """x (..., d) float64; pos broadcastable to x's leading dimensions, last 3."""
    y = x.clone()
    at = 0
    for ax, m in enumerate(dims):
        i = torch.arange(m // 2, device=x.device)
        a, b = (at + i, at + m // 2 + i) if halves else (at + 2 * i, at + 2 * i + 1)
        ang = pos[..., ax:ax + 1].double() * theta ** (-2.0 * i.double() / max(m, 1))
        c, s = ang.cos(), ang.sin() * (-1 if inverse else 1)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        at += m
    return y


def rope_close(got, want, size, dtype):
    """size: |a| + |b| bound of what each element is formed from."""
    half = torch.finfo(dtype).eps / 2
    err = (got.double() - want).abs()
    bound = 6 * 2.0 ** -24 * size * (1 + half) + half * want.abs() + 1e-38
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("d,dims,grid,batch,parts,heads", [
    (128, (44, 42, 42), (3, 5, 7), 2, 3, 3),
    (64, (16, 18, 22), (1, 1, 1), 1, 1, 1),
    (128, (0, 64, 30), (2, 9, 1), 1, 2, 5),
    (40, (2, 0, 6), (5, 4, 9), 3, 1, 2),
    (256, (128, 64, 64), (1, 1, 33), 1, 2, 1),
])
def test_rope(dtype, halves, inverse, d, dims, grid, batch, parts, heads):
    require_gpu()
    dt = DT[dtype]
    n = grid[0] * grid[1] * grid[2]
    g = gen(d + n)
    x = torch.randn(batch, n, parts, heads, d, generator=g, device="cuda").to(dt)
    if sum(dims) < d:  # what is not rotated is carried as it is, next to anything
        x[0, 0, 0, 0, sum(dims)] = math.inf
    y = torch.full((parts, batch, heads, n + 5, d), 7.0, dtype=dt, device="cuda")
    rope = L.make_rope(d, dims, grid[1:], offset=(2, -3, 100000), halves=halves)
    mask = 0b101 if parts == 3 else 1
    L.losa_rope_apply(rope, x.permute(2, 0, 1, 3, 4), y.permute(0, 1, 3, 2, 4), rotate=mask, inverse=inverse)
    assert L.losa_get_device_error() == 0
    assert not y[:, :, :, n:].any()
    pos = grid_positions(torch.arange(n), *grid[1:]) + torch.tensor([2, -3, 100000], device="cuda")
    for p in range(parts):
        xs = x[:, :, p].permute(0, 2, 1, 3)
        if not (mask >> p) & 1:
            assert torch.equal(y[p, :, :, :n], xs)
            continue
        want = turn(xs.double(), pos, dims, halves, inverse)
        rest = slice(sum(dims), None)
        assert torch.equal(y[p, :, :, :n, rest], xs[..., rest])
        turned = slice(0, sum(dims))
        one = torch.ones_like(pos)  # |a| + |b| of every pair
        size = xs.double().abs().clone()
        at = 0
        for m in dims:
            i = torch.arange(m // 2, device="cuda")
            a, b = (at + i, at + m // 2 + i) if halves else (at + 2 * i, at + 2 * i + 1)
            tot = xs[..., a].double().abs() + xs[..., b].double().abs()
            size[..., a] = tot
            size[..., b] = tot
            at += m
        rope_close(y[p, :, :, :n, turned], want[..., turned], size[..., turned], dt)


@pytest.mark.gpu
def test_rope_far_positions_and_explicit_positions():
    """Angles at positions near 2^31, and the same tokens by start, by offset and by explicit triples."""
    require_gpu()
    d, dims = 128, (44, 42, 42)
    g = gen(3)
    x = torch.randn(1, 2, 6, 3, d, generator=g, device="cuda")
    pos = torch.tensor([[2 ** 31 - 1, 0, 5], [-(2 ** 31), 1, -7], [123456789, -2000000000, 77], [0, 0, 0],
                        [1, 2, 3], [10 ** 6, 10 ** 7, 10 ** 8]], device="cuda")
    pos = torch.stack([pos, pos.flip(0)])
    y = torch.empty_like(x)
    L.losa_rope_apply(L.make_rope(d, dims, (4, 4)), x, y, positions=pos.int().contiguous())
    want = turn(x[0].double(), pos[:, :, None], dims, False)
    # the 64-bit reference itself is off by 2^31 * 2^-53 radians at the far end
    bound = (6 * 2.0 ** -24 + 2.0 ** -21) * (x[0].double().view(2, 6, 3, 64, 2).abs().sum(-1, keepdim=True)
                                              .expand(-1, -1, -1, -1, 2).reshape(2, 6, 3, d)) + 1e-30
    assert bool(((y[0].double() - want).abs() <= bound).all())
    start = torch.tensor([17, 1000003], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    rope = L.make_rope(d, dims, (9, 13), offset=(1, 2, 3))
    L.losa_rope_apply(rope, x, a, start=start)
    n = start.long()[:, None] + torch.arange(6, device="cuda")
    plain = L.make_rope(d, dims, (9, 13))
    triples = (grid_positions(n, 9, 13) + torch.tensor([1, 2, 3], device="cuda")).int().contiguous()
    L.losa_rope_apply(plain, x, b, positions=triples)
    assert torch.equal(a, b)
    # the inverse call undoes it: it is the transposed (gradient) map of an orthogonal one
    back = torch.empty_like(x)
    L.losa_rope_apply(rope, a, back, start=start, inverse=True)
    assert float((back - x).abs().max()) < 1e-5


@pytest.mark.gpu
def test_rope_gradient_against_differences():
    """<g, f(x + h e) - f(x - h e)> / 2h equals <f^T(g), e> for the layout-changing call, in fp32."""
    require_gpu()
    d, dims, n = 64, (16, 18, 22), 35
    g = gen(9)
    rope = L.make_rope(d, dims, (5, 7), halves=True)
    x = torch.randn(1, n, 2, 3, d, generator=g, device="cuda")
    w = torch.randn(2, 1, 3, n, d, generator=g, device="cuda")
    e = torch.randn_like(x)
    run = lambda z: (lambda y: (L.losa_rope_apply(rope, z.permute(2, 0, 1, 3, 4), y.permute(0, 1, 3, 2, 4), rotate=3), y)[1])(
        torch.empty(2, 1, 3, n, d, device="cuda"))
    h = 0.5  # the map is linear
    diff = ((run(x + h * e) - run(x - h * e)).double() * w.double()).sum() / (2 * h)
    grad = torch.empty_like(x)
    L.losa_rope_apply(rope, w.permute(0, 1, 3, 2, 4), grad.permute(2, 0, 1, 3, 4), rotate=3, inverse=True)
    want = (grad.double() * e.double()).sum()
    assert abs(float(diff - want)) <= 1e-4 * float((grad.double().abs() * e.double().abs()).sum())


# ------------------------------------------------------------------------------------------------------------ append

def make_pool(g, pages, hk, page, d):
    """Codes without NaN and scales of mixed powers of two."""
    k8 = (torch.randn(pages, hk, page, d, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    v8 = (torch.randn(pages, hk, page, d, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    ks = torch.exp2(torch.randint(-8, -3, (pages, hk), generator=g, device="cuda").float())
    vs = torch.exp2(torch.randint(-8, -3, (pages, hk), generator=g, device="cuda").float())
    return k8, v8, ks, vs


def append_reference(x, codes, scale, table, held, new, page):
    """float64 new codes (unrounded) and scales of one tensor; x: list of (new_b, hk, d) float64 per sequence."""
    c, s = codes.double(), scale.double()
    for b, (h, m) in enumerate(zip(held, new)):
        for blk in range(h // page, -(-(h + m) // page)):
            lo, hi = max(h - blk * page, 0), min(page, h + m - blk * page)
            if hi <= lo:
                continue
            rows = x[b][blk * page + lo - h:blk * page + hi - h]
            pg = int(table[b, blk])
            fin = torch.where(rows.isfinite(), rows.abs(), torch.zeros_like(rows))
            e = torch.ceil(torch.log2(fin.amax((0, 2)) / TOP)).clamp(-40, 60)
            now = torch.exp2(e)
            if lo:
                now = torch.maximum(now, s[pg])
                c[pg, :, :lo] *= (s[pg] / now)[:, None, None]
            s[pg] = now
            c[pg, :, lo:hi] = (rows / now[None, :, None]).transpose(0, 1)
    return c, s


def codes_match(got, want):
    """Codes equal the reference rounded to e4m3, but for values within 1e-5 of a rounding border."""
    got, w = got.double(), want.clamp(-TOP, TOP)
    near = [(w * (1 + k)).clamp(-TOP, TOP).float().to(torch.float8_e4m3fn).double() for k in (0.0, 1e-5, -1e-5)]
    ok = (got == near[0]) | (got == near[1]) | (got == near[2]) | (got.isnan() & want.isnan())
    assert bool(ok.all()), int((~ok).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,page,hk,held,new,halves,indptr", [
    ("bf16", 128, 128, 3, [0], [1], False, False),
    ("bf16", 128, 128, 2, [127, 128, 5], [1, 1, 1], False, False),
    ("bf16", 128, 32, 5, [31, 0, 64, 70], [100, 0, 1, 33], True, True),
    ("f32", 64, 64, 4, [1, 63], [300, 2], True, True),
    ("bf16", 64, 128, 1, [200], [513], False, False),
    ("f32", 128, 128, 2, [3, 250, 0], [128, 6, 129], True, True),
])
@pytest.mark.parametrize("rotated", [True, False])
def test_append(dtype, d, page, hk, held, new, halves, indptr, rotated):
    require_gpu()
    g = gen(sum(held) + sum(new) + d)
    seqs = len(held)
    width = max(-(-(h + m) // page) for h, m in zip(held, new)) + 1
    pages = seqs * width + 2
    k8, v8, ks, vs = make_pool(g, pages, hk, page, d)
    before = [t.clone() for t in (k8, v8, ks, vs)]
    table = torch.randperm(pages, generator=g, device="cuda")[:seqs * width].view(seqs, width).int()
    kv = torch.randn(sum(new), 2, hk, d, generator=g, device="cuda").to(DT[dtype])
    kv *= torch.exp2(torch.arange(hk, device="cuda", dtype=torch.float32) - 2).to(kv.dtype)[:, None]
    lens = torch.tensor(held, dtype=torch.int32, device="cuda")
    out = torch.full((seqs,), -9, dtype=torch.int32, device="cuda")
    ptr = torch.tensor([sum(new[:i]) for i in range(seqs + 1)], dtype=torch.int32, device="cuda")
    dims = (16, 18, 22) if d == 64 else (44, 42, 36)
    rope = L.make_rope(d, dims, (6, 11), halves=halves) if rotated else None
    cache = L.make_cache(hk, d, page, pages, seqs, width)
    bound = max(new) + (3 if indptr else 0)
    L.losa_cache_append(cache, kv[:, 0], kv[:, 1], k8, v8, ks, vs, table, lens, bound, indptr=ptr if indptr else None,
                        new_lens=out, rope=rope)
    assert L.losa_get_device_error() == 0
    assert out.tolist() == [h + m for h, m in zip(held, new)]
    per = [kv[int(ptr[b]):int(ptr[b + 1])].double() for b in range(seqs)]
    keys = [turn(x[:, 0], grid_positions(torch.arange(held[b], held[b] + new[b]), 6, 11)[:, None], dims, halves)
            if rotated else x[:, 0] for b, x in enumerate(per)]
    for x, codes, scale, was8, was in ((keys, k8, ks, before[0], before[2]), ([x[:, 1] for x in per], v8, vs, before[1], before[3])):
        want, ws = append_reference(x, was8, was, table, held, new, page)
        assert torch.equal(scale.double(), ws)
        codes_match(codes, want)
        # what the call has no business with keeps its bits
        touched = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
        for b, (h, m) in enumerate(zip(held, new)):
            for n in range((h // page) * page, h + m if m else 0):
                touched[int(table[b, n // page]), n % page] = True
        rest = ~touched[:, None, :, None].expand_as(codes)
        assert torch.equal(codes.view(torch.uint8)[rest], was8.view(torch.uint8)[rest])


@pytest.mark.gpu
def test_append_values_out_of_the_ordinary():
    """Infinities saturate, NaN stays NaN and neither sets a scale; zeros and the smallest and largest finite values; a
    block of zeros takes the smallest scale."""
    require_gpu()
    hk, d, page = 1, 64, 32
    cache = L.make_cache(hk, d, page, 2, 1, 2)
    g = gen(1)
    k8, v8, ks, vs = make_pool(g, 2, hk, page, d)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.randn(33, 1, d, generator=g, device="cuda")
    k[0, 0, 0], k[0, 0, 1], k[0, 0, 2], k[5, 0, 3] = math.inf, -math.inf, math.nan, 1e-45
    v = torch.zeros_like(k)
    v[32, 0, 0] = 3.0e38
    L.losa_cache_append(cache, k, v, k8, v8, ks, vs, table, lens, 33)
    assert L.losa_get_device_error() == 0
    top = float(k[:32][k[:32].isfinite()].abs().max())
    assert float(ks[1, 0]) == 2.0 ** math.ceil(math.log2(top / TOP))
    assert k8[1, 0, 0, 0].item() == TOP and k8[1, 0, 0, 1].item() == -TOP and math.isnan(k8[1, 0, 0, 2].item())
    assert float(vs[1, 0]) == 2.0 ** -40 and float(vs[0, 0]) == 2.0 ** 60 and not v8[1].float().any()
    assert v8[0, 0, 0, 0].item() == TOP


@pytest.mark.gpu
def test_append_reports_and_skips_bad_input():
    require_gpu()
    hk, d, page = 2, 128, 32
    cache = L.make_cache(hk, d, page, 4, 2, 2)
    g = gen(2)
    k = torch.randn(8, hk, d, generator=g, device="cuda").bfloat16()
    for table, lens, indptr, want in (
            ([[0, 9], [2, 3]], [31, 0], [0, 4, 8], [35, 4]),      # a page out of range: its tokens are dropped
            ([[0, 1], [2, 3]], [62, 0], [0, 4, 8], [64, 4]),      # behind the table's capacity
            ([[0, 1], [2, 3]], [-1, 0], [0, 4, 8], None),         # a negative length
            ([[0, 1], [2, 3]], [0, 0], [4, 0, 8], None),          # decreasing offsets
            ([[0, 1], [2, 3]], [0, 0], [0, 4, 80], None)):        # more rows than k holds
        pool = make_pool(g, 4, hk, page, d)
        was = [t.clone() for t in pool]
        out = torch.zeros(2, dtype=torch.int32, device="cuda")
        L.losa_cache_append(cache, k, k, *pool, torch.tensor(table, dtype=torch.int32, device="cuda"),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), 4,
                            indptr=torch.tensor(indptr, dtype=torch.int32, device="cuda"), new_lens=out)
        assert L.losa_get_device_error() == -5
        if want:
            assert out.tolist() == want
        if lens[0] == -1:
            assert all(torch.equal(a[:2].view(torch.uint8), b[:2].view(torch.uint8)) for a, b in zip(pool, was))


# --------------------------------------------------------------------------------------------------------- attention

def attend(q, k, v, end, scale):
    """64-bit attention of rows q (r, d), row i over keys < end[i]; returns o, lse, sum p |v|."""
    x = scale * (q @ k.T)
    x.masked_fill_(torch.arange(len(k), device=q.device) >= end[:, None], -math.inf)
    lse = torch.logsumexp(x, 1) if len(k) else torch.full(q.shape[:1], -math.inf, dtype=q.dtype, device=q.device)
    p = torch.exp(x - lse[:, None]).nan_to_num(0.0)
    p[end <= 0] = 0
    return p @ v, lse, p @ v.abs()


def attn_close(o, lse, want, want_lse, size):
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * size + 1e-30
    err = (o.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    empty = want_lse == -math.inf
    assert torch.equal(empty, lse.double() == -math.inf)
    assert bool(((lse.double() - want_lse).abs() <= 1e-4 + 256 * 2.0 ** -24 * want_lse.abs())[~empty].all())


def poisoned_cache(g, lens, hk, page, d, width, spread=4):
    """A pool whose slots behind every sequence's length, and whose unused pages, hold NaN codes and huge scales."""
    seqs = len(lens)
    pages = seqs * width + 1
    k8, v8, ks, vs = make_pool(g, pages, hk, page, d)
    vs = torch.exp2(torch.randint(-spread, spread, (pages, hk), generator=g, device="cuda").float())
    table = torch.randperm(pages, generator=g, device="cuda")[:seqs * width].view(seqs, width).int()
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[int(table[b, j // page]), j % page] = True
    free = ~used.cuda()[:, None, :, None].expand(pages, hk, page, d)
    k8.view(torch.uint8)[free] = 0x7F
    v8.view(torch.uint8)[free] = 0x7F
    idle = ~used.any(1).cuda()
    ks[idle], vs[idle] = math.inf, math.nan
    return k8, v8, ks, vs, table


def dense(codes, scale, table, b, h, n):
    at = table[b].long()
    x = codes[at, h].double() * scale[at, h].double()[:, None, None]
    return x.flatten(0, 1)[:n]


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,lens,heads,hk,tokens,causal", [
    (128, 128, [1], 1, 1, 1, True),
    (128, 128, [33, 0, 128, 1000], 6, 2, 1, True),
    (128, 32, [31, 700], 8, 8, 3, True),
    (64, 64, [65, 4097, 2], 12, 3, 2, True),
    (64, 32, [5000], 4, 1, 5, False),
    (128, 64, [20000], 24, 2, 4, True),          # 48 rows: three 16-row tiles
    (128, 128, [40000, 7], 5, 5, 2, False),
    (128, 32, [3, 1], 2, 1, 6, True),            # more tokens than the cache holds: the first see nothing
])
def test_cache_attn(d, page, lens, heads, hk, tokens, causal):
    require_gpu()
    g = gen(sum(lens) + heads)
    seqs = len(lens)
    width = max(1, -(-max(lens) // page)) + 1
    k8, v8, ks, vs, table = poisoned_cache(g, lens, hk, page, d, width)
    q = torch.randn(seqs, tokens, heads, d, generator=g, device="cuda").bfloat16()
    q[0, 0, 0] *= 2.0 ** 40  # a loud row only shifts its own scale
    q[0, 0, 0] *= 2.0 ** -41
    scale = 0.3 / math.sqrt(d)
    cache = L.make_cache(hk, d, page, k8.shape[0], seqs, width)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for max_len in (0, max(lens), 64):
        ws = torch.empty(max(16, L.losa_cache_attn_workspace_bytes(cache, heads, tokens, max_len)), dtype=torch.uint8,
                         device="cuda")
        o = torch.full((seqs, tokens, heads + 1, d), 9.0, device="cuda").bfloat16()  # strided: a spare head behind
        lse = torch.full((seqs, tokens, heads), 9.0, device="cuda")
        L.losa_cache_attn(cache, q, k8, v8, ks, vs, table, lens_t, scale, o[:, :, :heads], lse=lse, causal=causal,
                          max_len=max_len, workspace=ws)
        assert L.losa_get_device_error() == 0
        assert bool((o[:, :, heads] == 9.0).all())
        for b in range(seqs):
            for h in range(hk):
                k, v = dense(k8, ks, table, b, h, lens[b]), dense(v8, vs, table, b, h, lens[b])
                G = heads // hk
                rows = q[b, :, h * G:(h + 1) * G].double().reshape(-1, d)
                end = torch.arange(tokens, device="cuda").repeat_interleave(G)
                end = lens[b] - (tokens - 1 - end) if causal else torch.full_like(end, lens[b])
                want, wl, size = attend(rows, k, v, end, scale)
                attn_close(o[b, :, h * G:(h + 1) * G].reshape(-1, d), lse[b, :, h * G:(h + 1) * G].reshape(-1), want, wl,
                           size)


@pytest.mark.gpu
def test_cache_attn_sinks_and_loud_blocks():
    """One key that takes nearly all the weight over 30000 that share the rest, values of very different loudness, and a
    block of zeros with the smallest scale that still counts in the denominator."""
    require_gpu()
    g = gen(5)
    d, page, n, hk = 128, 128, 30000, 1
    width = -(-n // page)
    k8, v8, ks, vs, table = poisoned_cache(g, [n], hk, page, d, width)
    k8.view(torch.uint8)[int(table[0, 0]), 0, 7] = torch.full((d,), 448.0, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    ks.fill_(2.0 ** -8)
    first = int(table[0, 3])
    v8.view(torch.uint8)[first] = 0
    vs[first] = 2.0 ** -40
    vs[int(table[0, 9])] = 2.0 ** 20
    q = torch.ones(1, 1, 1, d, device="cuda").bfloat16() * 0.07
    cache = L.make_cache(hk, d, page, k8.shape[0], 1, width)
    ws = torch.empty(max(16, L.losa_cache_attn_workspace_bytes(cache, 1, 1, n)), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 1, 1, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for scale in (1.0, 0.01):
        L.losa_cache_attn(cache, q, k8, v8, ks, vs, table, lens, scale, o, lse=lse, workspace=ws, max_len=n)
        want, wl, size = attend(q[0, 0].double(), dense(k8, ks, table, 0, 0, n), dense(v8, vs, table, 0, 0, n),
                                torch.tensor([n], device="cuda"), scale)
        attn_close(o[0, 0], lse[0, 0], want, wl, size)


@pytest.mark.gpu
def test_cache_attn_bad_pages_and_lengths_are_reported():
    require_gpu()
    g = gen(6)
    d, page, hk = 64, 32, 2
    k8, v8, ks, vs, table = poisoned_cache(g, [64, 64], hk, page, d, 2)
    cache = L.make_cache(hk, d, page, k8.shape[0], 2, 2)
    q = torch.randn(2, 1, 2, d, generator=g, device="cuda").bfloat16()
    o = torch.empty_like(q)
    bad = table.clone()
    bad[0, 1] = k8.shape[0]
    lens = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
    L.losa_cache_attn(cache, q, k8, v8, ks, vs, bad, lens, 0.1, o)
    assert L.losa_get_device_error() == -5
    for b, n in ((0, 32), (1, 64)):  # the bad page's keys are left out, the rest is computed
        for h in range(2):
            want, _, size = attend(q[b, :, h].double(), dense(k8, ks, table, b, h, n), dense(v8, vs, table, b, h, n),
                                   torch.tensor([n], device="cuda"), 0.1)
            assert bool(((o[b, :, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * size).all())
    L.losa_cache_attn(cache, q, k8, v8, ks, vs, table, torch.tensor([-3, 65], dtype=torch.int32, device="cuda"), 0.1, o)
    assert L.losa_get_device_error() == -5
    assert not o[0].any()


# ------------------------------------------------------------------------------------------------------ blocked queries

def random_lists(g, items, width, lo, hi, empty_every=0):
    counts = torch.randint(lo, hi + 1, (items,), generator=g, device="cuda")
    if empty_every:
        counts[::empty_every] = 0
    order_of = torch.rand(items, width, generator=g, device="cuda").argsort(1)  # distinct blocks, in any order
    keep = torch.arange(width, device="cuda")[None] < counts[:, None]
    indptr = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    return indptr, order_of[keep].int().contiguous()


def check_blocks(q, o, lse, pool, table, lens, page, heads, hk, n, scale, indptr, blocks, items=None):
    k8, v8, ks, vs = pool
    nq = q.shape[1] // 128
    H = q.shape[0]
    per = heads // hk
    ptr = None if indptr is None else indptr.tolist()
    cached = {}
    for item in (range(H * nq) if items is None else items):
        h, i = divmod(item, nq)
        b, kvh = h // heads, (h % heads) // per
        if (b, kvh) not in cached:
            cached = {(b, kvh): (dense(k8, ks, table, b, kvh, lens[b]), dense(v8, vs, table, b, kvh, lens[b]))}
        k, v = cached[(b, kvh)]
        if ptr is None:
            key = torch.arange(lens[b], device="cuda")
        else:
            at = blocks[ptr[item]:ptr[item + 1]].long()
            key = (at[:, None] * page + torch.arange(page, device="cuda")).flatten()
            key = key[key < lens[b]]
        rows = slice(i * 128, min(n, i * 128 + 128))
        want, wl, size = attend(q[h, rows].double(), k[key], v[key],
                                torch.full((q[h, rows].shape[0],), len(key), device="cuda"), scale)
        attn_close(o[h, rows], lse[h, rows], want, wl, size)


@pytest.mark.gpu
@pytest.mark.parametrize("page,lens,heads,hk,n,lo,hi,empty,ordered", [
    (128, [1000], 1, 1, 100, 1, 1, 0, False),
    (128, [129], 2, 1, 130, 1, 2, 0, True),
    (32, [777], 2, 2, 300, 1, 9, 4, True),
    (64, [640, 33], 4, 2, 257, 1, 5, 3, False),
    (128, [0, 4000], 6, 2, 900, 1, 20, 5, True),
    (32, [3000], 12, 12, 5000, 1, 3, 7, True),      # 480 items: several short items on every SM
    (64, [1999], 3, 3, 128 * 99, 1, 12, 0, True),
    (32, [20000], 2, 1, 4000, 100, 600, 0, True),   # long lists
    (128, [513, 5, 2048], 2, 2, 385, 0, 0, 0, False),  # no lists: every block
    (32, [100, 7000], 3, 1, 1, 0, 0, 0, False),
])
def test_cache_sparse_attn(page, lens, heads, hk, n, lo, hi, empty, ordered):
    require_gpu()
    g = gen(sum(lens) + n)
    seqs = len(lens)
    width = max(1, -(-max(lens) // page)) + 2  # lists may name blocks behind the sequence
    k8, v8, ks, vs, table = poisoned_cache(g, lens, hk, page, 128, width)
    H, nq = seqs * heads, -(-n // 128)
    q = torch.randn(H, nq * 128, 128, generator=g, device="cuda").bfloat16()
    q[0, 0] *= 2.0 ** 30  # a loud row, a quiet one and a zero one
    q[0, 0] *= 2.0 ** -30
    q[-1, 0] *= 2.0 ** -20
    q[0, min(n - 1, 1)] = 0
    q[:, n:] = math.nan  # padding rows hold anything
    items = H * nq
    indptr = blocks = order = None
    if hi:
        indptr, blocks = random_lists(g, items, width, lo, min(hi, width), empty)
    if ordered:
        order = torch.randperm(items, generator=g, device="cuda").int()
    scale = 0.3 / math.sqrt(128)
    o = torch.full_like(q, 9.0)
    lse = torch.full((H, nq * 128), 9.0, device="cuda")
    cache = L.make_cache(hk, 128, page, k8.shape[0], seqs, width)
    L.losa_cache_sparse_attn(L.make_shape(H, n, nq * 128, 128, 128, page, "bf16"), cache, q, k8, v8, ks, vs, table,
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, o, indptr=indptr,
                             kv_block_idx=blocks, order=order, lse=lse)
    assert L.losa_get_device_error() == 0
    check_blocks(q, o, lse, (k8, v8, ks, vs), table, lens, page, heads, hk, n, scale, indptr, blocks)


@pytest.mark.gpu
def test_cache_sparse_attn_sinks_and_growing_rows():
    """Rows whose maximum grows by far more than 2^8 from block to block, one key that outweighs 30000, loud and quiet
    values: the reference moves, nothing overflows, and the tail under the sink is kept."""
    require_gpu()
    g = gen(11)
    page, n = 128, 30000
    width = -(-n // page)
    k8, v8, ks, vs, table = poisoned_cache(g, [n], 1, page, 128, width, spread=6)
    ks[table[0].long(), 0] = torch.exp2(-9 + torch.arange(width, device="cuda").float() / 40)
    k8.view(torch.uint8)[int(table[0, 100]), 0, 7] = torch.full((128,), 448.0, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    v8.view(torch.uint8)[int(table[0, 3])] = 0
    vs[int(table[0, 3])] = 2.0 ** -40
    q = torch.randn(1, 128, 128, generator=g, device="cuda").bfloat16()
    q[0, :40] = 0.05
    o, lse = torch.empty_like(q), torch.empty(1, 128, device="cuda")
    cache = L.make_cache(1, 128, page, k8.shape[0], 1, width)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for scale in (1.0, 0.05):
        L.losa_cache_sparse_attn(L.make_shape(1, 128, 128, 128, 128, page, "bf16"), cache, q, k8, v8, ks, vs, table, lens,
                                 scale, o, lse=lse)
        assert L.losa_get_device_error() == 0
        want, wl, size = attend(q[0].double(), dense(k8, ks, table, 0, 0, n), dense(v8, vs, table, 0, 0, n),
                                torch.full((128,), n, device="cuda"), scale)
        attn_close(o[0], lse[0], want, wl, size)


@pytest.mark.gpu
def test_cache_sparse_attn_reports_bad_input():
    require_gpu()
    g = gen(12)
    page, n = 64, 256
    k8, v8, ks, vs, table = poisoned_cache(g, [n], 1, page, 128, 4)
    q = torch.randn(1, 256, 128, generator=g, device="cuda").bfloat16()
    shape, cache = L.make_shape(1, 256, 256, 128, 128, page, "bf16"), L.make_cache(1, 128, page, k8.shape[0], 1, 4)
    good = dict(table=table, lens=[n], indptr=[0, 2, 4], blocks=[0, 1, 2, 3], order=[0, 1])
    i32 = lambda v: v if torch.is_tensor(v) else torch.tensor(v, dtype=torch.int32, device="cuda")
    low = table.clone()
    low[0, 1] = -1
    for bad, left in ((dict(blocks=[0, 4, 2, 3]), [0]), (dict(blocks=[0, -1, 2, 3]), [0]), (dict(table=low), [0]),
                      (dict(indptr=[0, 2, 1]), None), (dict(lens=[n + 1]), [0, 1]), (dict(order=[0, 2]), [0, 1])):
        c = {**good, **bad}
        o = torch.full_like(q, 9.0)
        lse = torch.full((1, 256), 9.0, device="cuda")
        L.losa_cache_sparse_attn(shape, cache, q, k8, v8, ks, vs, i32(c["table"]), i32(c["lens"]), 0.02, o,
                                 indptr=i32(c["indptr"]), kv_block_idx=i32(c["blocks"]), order=i32(c["order"]), lse=lse)
        assert L.losa_get_device_error() == -5, bad
        if left is not None:  # item 0 over the blocks that are left
            k, v = dense(k8, ks, table, 0, 0, n), dense(v8, vs, table, 0, 0, n)
            key = torch.cat([torch.arange(j * page, j * page + page, device="cuda") for j in left])
            want, wl, size = attend(q[0, :128].double(), k[key], v[key], torch.full((128,), len(key), device="cuda"), 0.02)
            attn_close(o[0, :128], lse[0, :128], want, wl, size)


# ------------------------------------------------------------------------------------------- together, streams, graphs

@pytest.mark.gpu
@pytest.mark.parametrize("page", [128, 32])
def test_a_stream_of_chunks_end_to_end(page):
    """A clip generated in two chunks and then token by token, through the harness: projection -> rotated layer ->
    pattern from the exact masses -> 8-bit cache -> sparse attention over the frozen lists -> token-major output; then
    three drafted tokens decoded over everything. Every step against 64 bits on what the step before stored."""
    require_gpu()
    from free_block_sparse_losa_b200.harness import KvCache, LayerBuffers
    g = gen(21)
    H, d, n, gy, gx = 3, 128, 2 * 13 * 21, 13, 21
    scale = 1 / math.sqrt(d)
    rope = L.make_rope(d, (44, 42, 42), (gy, gx))
    cache = KvCache(1, H, d, 2 * n + 64, page_tokens=page, rope=rope)
    qkv = torch.randn(1, 2 * n, 3, H, d, generator=g, device="cuda").bfloat16()
    qkv[:, :, :2] *= 1.5
    np_ = -(-n // 128) * 128
    layer = LayerBuffers(H, n, np_, d, 128, "bf16", block_k=page if page == 32 else 0)
    for chunk in range(2):
        part = qkv[:, chunk * n:(chunk + 1) * n]
        start = torch.tensor([chunk * n], dtype=torch.int32, device="cuda")
        q, k, v = layer.pack_qkv(part, rope, start=start)
        pos = grid_positions(chunk * n + torch.arange(n), gy, gx)
        want = turn(part[0, :, 0].double(), pos[:, None], (44, 42, 42), False).transpose(0, 1)
        assert bool(((q[:, :n].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())
        assert not k[:, n:].any() and torch.equal(v[:, :n], part[0, :, 2].transpose(0, 1))
        if chunk == 0:
            layer.profile(q, k, v, scale)
            layer.select(0.95)
        cache.append(part[0, :, 1], part[0, :, 2], n)
        assert cache.lens.tolist() == [(chunk + 1) * n]
        o, lse = torch.empty_like(q), torch.empty(H, np_, device="cuda")
        cache.sparse(layer, q, scale, o, lse=lse)  # the second chunk reuses the frozen lists
        assert L.losa_get_device_error() == 0
        check_blocks(q, o, lse, (cache.k8, cache.v8, cache.k_scale, cache.v_scale), cache.page_table, cache.lens.tolist(),
                     page, H, H, n, scale, layer.indptr, layer.kv_idx)
        back = layer.unpack_o(rope, torch.empty(1, n, H, d, dtype=torch.bfloat16, device="cuda"), o=o)
        assert torch.equal(back[0].transpose(0, 1), o[:, :n])
        if chunk == 0:  # the 8-bit step stays near the 16-bit one: e4m3 values are off by at most 2^-4, on average far less
            ref = torch.empty_like(q)
            layer.sparse(q, k, v, scale, out=ref)
            rel = (o[:, :n].float() - ref[:, :n].float()).norm() / ref[:, :n].float().norm()
            assert float(rel) <= 2.0 ** -4
    for step in range(2):
        new = torch.randn(3, 3, H, d, generator=g, device="cuda").bfloat16()
        base = 2 * n + 3 * step
        q = torch.empty(1, 3, H, d, dtype=torch.bfloat16, device="cuda")
        L.losa_rope_apply(rope, new[:, 0][None, None], q[None], start=cache.lens)
        cache.append(new[:, 1], new[:, 2], 3)
        o, lse = torch.empty_like(q), torch.empty(1, 3, H, device="cuda")
        cache.attend(q, scale, o, lse=lse)
        assert cache.lens.tolist() == [base + 3] and L.losa_get_device_error() == 0
        for h in range(H):
            k = dense(cache.k8, cache.k_scale, cache.page_table, 0, h, base + 3)
            v = dense(cache.v8, cache.v_scale, cache.page_table, 0, h, base + 3)
            end = torch.tensor([base + 1, base + 2, base + 3], device="cuda")
            want, wl, size = attend(q[0, :, h].double(), k, v, end, scale)
            attn_close(o[0, :, h], lse[0, :, h], want, wl, size)
        # what the cache holds is the rotated keys, to within the rounding of their block's scale
        pos = grid_positions(base + torch.arange(3), gy, gx)
        keys = turn(new[:, 1].double(), pos[:, None], (44, 42, 42), False)
        got = torch.stack([dense(cache.k8, cache.k_scale, cache.page_table, 0, h, base + 3)[-3:] for h in range(H)], 1)
        top = keys.abs().amax() * 2  # a block's scale is below twice what its loudest key needs
        assert bool(((got - keys).abs() <= 2.0 ** -4 * keys.abs() + 2.0 ** -9 * 4 * top / 448 + 2.0 ** -4 * top / 64).all())


@pytest.mark.gpu
def test_calls_on_other_streams_with_their_own_workspaces():
    """The same decode from four streams at once, each with its own inputs, outputs and workspace, gives what one stream
    gives, bit for bit; the blocked form and the append run beside them."""
    require_gpu()
    g = gen(31)
    lens, hk, page, d = [5000, 9000], 2, 64, 128
    width = -(-max(lens) // page)
    pool = poisoned_cache(g, lens, hk, page, d, width)
    k8, v8, ks, vs, table = pool
    cache = L.make_cache(hk, d, page, k8.shape[0], 2, width)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    need = L.losa_cache_attn_workspace_bytes(cache, 4, 2, max(lens))
    assert need > 0
    runs = []
    for _ in range(4):
        q = torch.randn(2, 2, 4, d, generator=g, device="cuda").bfloat16()
        runs.append([q, torch.empty_like(q), torch.empty(need, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()])
    qb = torch.randn(8, 256, 128, generator=g, device="cuda").bfloat16()
    shape = L.make_shape(8, 256, 256, 128, 128, page, "bf16")
    ob = torch.empty_like(qb)

    def decode(q, o, ws, stream=None):
        L.losa_cache_attn(cache, q, k8, v8, ks, vs, table, lens_t, 0.02, o, max_len=max(lens), workspace=ws, stream=stream)

    want = []
    for q, o, ws, _ in runs:
        decode(q, o, ws)
        want.append(o.clone())
    L.losa_cache_sparse_attn(shape, cache, qb, k8, v8, ks, vs, table, lens_t, 0.02, ob)
    want_b = ob.clone()
    torch.cuda.synchronize()
    for _ in range(10):
        for q, o, ws, st in runs:
            o.zero_()
        ob.zero_()
        torch.cuda.synchronize()
        for q, o, ws, st in runs:
            decode(q, o, ws, stream=st)
        with torch.cuda.stream(runs[0][3]):
            L.losa_cache_sparse_attn(shape, cache, qb, k8, v8, ks, vs, table, lens_t, 0.02, ob)
        torch.cuda.synchronize()
        assert all(torch.equal(r[1], w) for r, w in zip(runs, want)) and torch.equal(ob, want_b)
    assert L.losa_get_device_error() == 0


@pytest.mark.gpu
def test_captured_steps_replayed_on_new_inputs():
    """A captured step (rotation, append, decode over the grown cache, blocked attention) replayed with new tokens and new
    lengths in place gives what eager calls give."""
    require_gpu()
    g = gen(41)
    hk, page, d, H = 2, 32, 128, 4
    width = 40
    pages = 2 * width
    cache = L.make_cache(hk, d, page, pages, 2, width)
    rope = L.make_rope(d, (16, 56, 56), (3, 7), halves=True)
    table = torch.randperm(pages, generator=g, device="cuda").view(2, width).int()
    shape = L.make_shape(2 * H, 100, 128, 128, 128, page, "bf16")

    def state(seed):
        z = gen(seed)
        return dict(pool=make_pool(gen(99), pages, hk, page, d), lens=torch.tensor([40 + seed, 1100], dtype=torch.int32, device="cuda"),
                    new=torch.zeros(2, dtype=torch.int32, device="cuda"),
                    x=torch.randn(2, 2, H + 2 * hk, d, generator=z, device="cuda").bfloat16(),
                    q=torch.zeros(2, 2, H, d, device="cuda").bfloat16(), o=torch.zeros(2, 2, H, d, device="cuda").bfloat16(),
                    qb=torch.randn(2 * H, 128, d, generator=z, device="cuda").bfloat16(),
                    ob=torch.zeros(2 * H, 128, d, device="cuda").bfloat16(),
                    ws=torch.empty(max(16, L.losa_cache_attn_workspace_bytes(cache, H, 2)), dtype=torch.uint8, device="cuda"))

    def step(s):
        L.losa_rope_apply(rope, s["x"][None, :, :, :H], s["q"][None], start=s["lens"])
        kv = s["x"].view(4, H + 2 * hk, d)
        L.losa_cache_append(cache, kv[:, H:H + hk], kv[:, H + hk:], *s["pool"], table, s["lens"], 2, new_lens=s["new"], rope=rope)
        L.losa_cache_attn(cache, s["q"], *s["pool"], table, s["new"], 0.05, s["o"], workspace=s["ws"])
        L.losa_cache_sparse_attn(shape, cache, s["qb"], *s["pool"], table, s["new"], 0.05, s["ob"])

    a = state(1)
    step(a)  # loads the kernels
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    a = state(1)
    with torch.cuda.graph(graph, stream=side):
        step(a)
    for seed in (2, 3):
        b = state(seed)
        step(b)
        fresh = state(seed)
        for key in ("lens", "x", "qb"):
            a[key].copy_(fresh[key])
        for dst, src in zip(a["pool"], fresh["pool"]):
            dst.view(torch.uint8).copy_(src.view(torch.uint8)) if dst.dtype == torch.float8_e4m3fn else dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for key in ("new", "q", "o", "ob"):
            assert torch.equal(a[key], b[key]), key
        assert all(torch.equal(u.view(torch.uint8), w.view(torch.uint8)) for u, w in zip(a["pool"], b["pool"]))
    assert L.losa_get_device_error() == 0


@pytest.mark.gpu
def test_a_captured_decode_keeps_its_workspace():
    """A decode captured through the harness shares no memory with later calls: calls with other row counts, and tensors made
    since, are as they were after a replay; and calls on two streams at once give what one gives."""
    require_gpu()
    from free_block_sparse_losa_b200.harness import KvCache
    g = gen(57)
    hk, d, n = 2, 128, 6000
    cache = KvCache(2, hk, d, n, page_tokens=64)
    cache.append(*torch.randn(2, 2 * n, hk, d, generator=g, device="cuda").bfloat16(), n)
    q = [torch.randn(2, t, 8, d, generator=g, device="cuda").bfloat16() for t in (1, 1, 3)]
    o = [torch.zeros_like(x) for x in q]
    for x, y in zip(q, o):
        cache.attend(x, 0.05, y)
    want = [y.clone() for y in o]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(q[0], 0.05, o[0])
    cache.attend(q[2], 0.05, o[2])
    need = L.losa_cache_attn_workspace_bytes(cache.cache, 8, 1, n)
    assert need > 0
    marks = [torch.full((need + 7 * i,), 90 + i, dtype=torch.uint8, device="cuda") for i in range(8)]
    for y in o:
        y.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        cache.attend(q[1], 0.05, o[1], stream=streams[1])
        cache.attend(q[2], 0.05, o[2], stream=torch.cuda.default_stream().cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(o, want))
    assert all(bool((m == 90 + i).all()) for i, m in enumerate(marks))
    assert L.losa_get_device_error() == 0


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 codes and a rotation of more than 2^31 elements: the far ends are read and written."""
    require_gpu()
    g = gen(51)
    hk, page, d = 8, 128, 128
    pages = (2 ** 31) // (hk * page * d) + 64
    assert pages * hk * page * d > 2 ** 31
    k8 = torch.zeros(pages, hk, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v8 = torch.zeros(pages, hk, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks, vs = torch.ones(pages, hk, device="cuda"), torch.ones(pages, hk, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    cache = L.make_cache(hk, d, page, pages, 1, 3)
    n = 300
    kv = torch.randn(n, 2, hk, d, generator=g, device="cuda").bfloat16()
    lens, new = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.losa_cache_append(cache, kv[:, 0], kv[:, 1], k8, v8, ks, vs, table, lens, n, new_lens=new)
    q = torch.randn(1, 2, hk, d, generator=g, device="cuda").bfloat16()
    o = torch.empty_like(q)
    ws = torch.empty(max(16, L.losa_cache_attn_workspace_bytes(cache, hk, 2)), dtype=torch.uint8, device="cuda")
    L.losa_cache_attn(cache, q, k8, v8, ks, vs, table, new, 0.05, o, workspace=ws)
    qb = torch.randn(hk, 128, d, generator=g, device="cuda").bfloat16()
    ob, lb = torch.empty_like(qb), torch.empty(hk, 128, device="cuda")
    L.losa_cache_sparse_attn(L.make_shape(hk, 128, 128, d, 128, page, "bf16"), cache, qb, k8, v8, ks, vs, table, new, 0.05, ob,
                             lse=lb)
    assert L.losa_get_device_error() == 0
    for h in (0, hk - 1):
        k, v = dense(k8, ks, table, 0, h, n), dense(v8, vs, table, 0, h, n)
        assert float((k - kv[:, 0, h].double()).abs().max()) <= 2.0 ** -4 * float(kv.abs().max())
        want, _, size = attend(q[0, :, h].double(), k, v, torch.tensor([n - 1, n], device="cuda"), 0.05)
        assert bool(((o[0, :, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * size).all())
        want, wl, size = attend(qb[h].double(), k, v, torch.full((128,), n, device="cuda"), 0.05)
        attn_close(ob[h], lb[h], want, wl, size)
    del k8, v8
    heads, n = 128, 131100
    x = torch.zeros(1, 1, n, heads, d, dtype=torch.bfloat16, device="cuda")
    x[0, 0, -3:] = torch.randn(3, heads, d, generator=g, device="cuda").bfloat16()
    y = torch.empty(1, 1, heads, n, d, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    L.losa_rope_apply(L.make_rope(d, (44, 42, 42), (45, 80)), x, y.transpose(2, 3))
    want = turn(x[0, 0, -3:].double(), grid_positions(n - 3 + torch.arange(3), 45, 80)[:, None], (44, 42, 42), False)
    assert bool(((y[0, 0, :, -3:].transpose(0, 1).double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())
    assert not y[0, 0, :, :-3].any()
