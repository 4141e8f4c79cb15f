"""The streaming calls at the ends of what their documentation allows, against 64-bit forms; the tolerances are those of
tests/test_gpu_stream.py unless a test derives its own."""
import math

import pytest
import torch

import free_block_sparse_losa_b200 as L
from tests.gpu_util import require_gpu
from tests.test_gpu_stream import (append_reference, attend, attn_close, check_blocks, dense, gen, grid_positions, make_pool,
                                   poisoned_cache, random_lists, turn)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def blocks_call(q, pool, table, lens, page, heads, hk, n, scale, **lists):
    """The blocked call over the cache of poisoned_cache; returns o and lse."""
    H, rows, d = q.shape
    o, lse = torch.full_like(q, 9.0), torch.full((H, rows), 9.0, device="cuda")
    cache = L.make_cache(hk, d, page, pool[0].shape[0], table.shape[0], table.shape[1])
    L.losa_cache_sparse_attn(L.make_shape(H, n, rows, d, 128, page, "bf16"), cache, q, *pool, table, ints(lens), scale, o,
                             lse=lse, **lists)
    return o, lse


def decode_call(q, pool, table, lens, scale, causal=True, max_len=0):
    """The few-token call over the cache of poisoned_cache; returns o and lse."""
    seqs, tokens, heads, d = q.shape
    hk, page = pool[0].shape[1:3]
    cache = L.make_cache(hk, d, page, pool[0].shape[0], seqs, table.shape[1])
    ws = torch.empty(max(16, L.losa_cache_attn_workspace_bytes(cache, heads, tokens, max_len)), dtype=torch.uint8,
                     device="cuda")
    o, lse = torch.full_like(q, 9.0), torch.full((seqs, tokens, heads), 9.0, device="cuda")
    L.losa_cache_attn(cache, q, *pool, table, ints(lens), scale, o, lse=lse, causal=causal, max_len=max_len, workspace=ws)
    return o, lse


def check_decode(q, o, lse, pool, table, lens, scale, causal=True):
    seqs, tokens, heads, d = q.shape
    k8, v8, ks, vs = pool
    hk = k8.shape[1]
    G = heads // hk
    for b in range(seqs):
        end = torch.arange(tokens, device="cuda").repeat_interleave(G)
        end = lens[b] - (tokens - 1 - end) if causal else torch.full_like(end, lens[b])
        for h in range(hk):
            at = slice(h * G, (h + 1) * G)
            want, wl, size = attend(q[b, :, at].double().reshape(-1, d), dense(k8, ks, table, b, h, lens[b]),
                                    dense(v8, vs, table, b, h, lens[b]), end, scale)
            attn_close(o[b, :, at].reshape(-1, d), lse[b, :, at].reshape(-1), want, wl, size)


@pytest.mark.gpu
@pytest.mark.parametrize("page,n", [(32, 70), (128, 200), (64, 1000)])
def test_blocks_of_zero_keys_and_quiet_rows(page, n):
    """Blocks of zero keys carry the smallest scale, 2^-40; times the factor of a row whose largest element is near 2^-110
    that is zero in fp32. A part-full last block of them must still hide the slots that hold no token."""
    require_gpu()
    g = gen(61)
    width = -(-n // page)
    k8, v8, ks, vs, table = poisoned_cache(g, [n], 1, page, 128, width)
    used = table[0].long()
    slot = torch.arange(width * page, device="cuda").view(width, 1, page) < n
    codes = k8.view(torch.uint8)
    codes[used] = torch.where(slot[..., None], 0, codes[used])
    ks[used] = 2.0 ** -40
    q = torch.randn(1, 128, 128, generator=g, device="cuda").bfloat16()
    q[0, ::3] *= 2.0 ** -110
    q[0, 1::3] *= 2.0 ** -120
    for scale in (0.09, 1e-6):
        o, lse = blocks_call(q, (k8, v8, ks, vs), table, [n], page, 1, 1, 128, scale)
        assert L.losa_get_device_error() == 0
        check_blocks(q, o, lse, (k8, v8, ks, vs), table, [n], page, 1, 1, 128, scale, None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("lists", [None, "empty", "some"])
@pytest.mark.parametrize("lens,clamped", [([-1, 200], [0, 200]), ([200, 257], [200, 256]), ([200, -2 ** 31], [200, 0])])
def test_blocks_report_every_bad_length(lists, lens, clamped):
    """A length out of [0, capacity] is reported whether or not a list entry looks at it, and read as the nearest end."""
    require_gpu()
    g = gen(62)
    page, heads, n = 64, 2, 200
    k8, v8, ks, vs, table = poisoned_cache(g, [256, 256], 1, page, 128, 4)
    q = torch.randn(2 * heads, 256, 128, generator=g, device="cuda").bfloat16()
    items = 2 * heads * 2
    counts = {None: None, "empty": [0] * items, "some": [0, 2] * (items // 2)}[lists]
    kw = {}
    if counts:
        kw = dict(indptr=ints([sum(counts[:i]) for i in range(items + 1)]), kv_block_idx=ints([0, 3] * max(1, sum(counts) // 2)))
    o, lse = blocks_call(q, (k8, v8, ks, vs), table, lens, page, heads, 1, n, 0.02, **kw)
    assert L.losa_get_device_error() == -5
    check_blocks(q, o, lse, (k8, v8, ks, vs), table, clamped, page, heads, 1, n, 0.02, kw.get("indptr"),
                 kw.get("kv_block_idx"))
    good = blocks_call(q, (k8, v8, ks, vs), table, clamped, page, heads, 1, n, 0.02, **kw)
    assert L.losa_get_device_error() == 0
    assert torch.equal(good[0], o) and torch.equal(good[1], lse)


BAD = (math.inf, -math.inf, math.nan)


@pytest.mark.gpu
@pytest.mark.parametrize("d,lens,tokens,max_len", [(128, [1, 40, 0], 1, 64), (64, [700, 3], 2, 64), (128, [5000, 1, 0], 1, 0),
                                                   (64, [3000, 2500], 5, 0)])
def test_decode_rows_with_infinities_are_nan(d, lens, tokens, max_len):
    """A query row that holds an infinity or NaN has no softmax: o and lse are NaN wherever it sees a key, however the keys'
    signs fall, and zero and -inf where it sees none. Other rows keep their bits."""
    require_gpu()
    g = gen(64)
    seqs, hk, heads, page = len(lens), 2, 6, 32
    width = -(-max(lens) // page)
    *pool, table = poisoned_cache(g, lens, hk, page, d, width)
    q = torch.randn(seqs, tokens, heads, d, generator=g, device="cuda").bfloat16()
    clean = decode_call(q, pool, table, lens, 0.1, max_len=max_len)
    bad = torch.zeros(seqs, tokens, heads, dtype=torch.bool, device="cuda")
    for i, (h, value) in enumerate(zip((0, 3, 4), BAD)):
        q[:, :, h, (7 * i + 5) % d] = value
        bad[:, :, h] = True
    o, lse = decode_call(q, pool, table, lens, 0.1, max_len=max_len)
    assert L.losa_get_device_error() == 0
    end = ints(lens)[:, None] - (tokens - 1 - torch.arange(tokens, device="cuda"))
    nan = bad & (end > 0)[:, :, None]
    assert bool(o[nan].isnan().all()) and bool(lse[nan].isnan().all())
    assert torch.equal(o[~nan], clean[0][~nan]) and torch.equal(lse[~nan], clean[1][~nan])


@pytest.mark.gpu
@pytest.mark.parametrize("page,lens,listed", [(128, [300, 0], False), (32, [1, 999], False), (64, [500, 130], True)])
def test_block_rows_with_infinities_are_nan(page, lens, listed):
    """The same of the blocked call."""
    require_gpu()
    g = gen(65)
    heads, n, seqs = 2, 200, len(lens)
    width = -(-max(lens) // page)
    *pool, table = poisoned_cache(g, lens, 1, page, 128, width)
    q = torch.randn(seqs * heads, 256, 128, generator=g, device="cuda").bfloat16()
    kw, sees = {}, ints(lens).repeat_interleave(2 * heads) > 0
    if listed:
        counts = [0, 3, 1, 2] * seqs
        kw = dict(indptr=ints([sum(counts[:i]) for i in range(len(counts) + 1)]), kv_block_idx=ints([0, 1, 2, 1, 0, 2] * seqs))
        sees = ints(counts) > 0
    clean = blocks_call(q, pool, table, lens, page, heads, 1, n, 0.1, **kw)
    bad = torch.zeros(seqs * heads, 256, dtype=torch.bool, device="cuda")
    for i, value in enumerate(BAD):
        q[:, 17 * i + 1::64, 31 * i] = value
        bad[:, 17 * i + 1::64] = True
    o, lse = blocks_call(q, pool, table, lens, page, heads, 1, n, 0.1, **kw)
    assert L.losa_get_device_error() == 0
    nan = bad & sees.view(seqs * heads, 2).repeat_interleave(128, 1)
    assert bool(o[nan].isnan().all()) and bool(lse[nan].isnan().all())
    assert torch.equal(o[~nan], clean[0][~nan]) and torch.equal(lse[~nan], clean[1][~nan])


def subnormal_rows(q):
    """q's values as bf16 numbers below 2^-126, of the same signs."""
    bits = (q.float().abs() * 40).clamp(max=127).to(torch.int16)
    return torch.where(q < 0, bits | -2 ** 15, bits).view(torch.bfloat16)


# (scale, sizes of rows): logits of the loudest rows are near one, the others' near zero
ROWS = [(0.03 * 2.0 ** -40, (40, 0, -50, None, 38)), (0.03 * 2.0 ** -100, (100, 96, 0, None)), (0.03 * 2.0 ** 60, (-60, -64, -110, None)),
        (0.03 * 2.0 ** 100, (-100, -103, None)), (2.0 ** 124, ("sub", None, "sub"))]


def sized(q, sizes):
    """Rows of q (leading dimensions flattened) brought to the sizes in turn: a power of two, None for zeros."""
    rows = q.view(-1, q.shape[-1])
    for i, s in enumerate(sizes):
        part = rows[i::len(sizes)]
        rows[i::len(sizes)] = subnormal_rows(part) if s == "sub" else torch.zeros_like(part) if s is None else part * 2.0 ** s
    return q


@pytest.mark.gpu
@pytest.mark.parametrize("scale,sizes", ROWS)
@pytest.mark.parametrize("d,tokens,max_len", [(128, 1, 64), (64, 4, 0)])
def test_decode_rows_of_any_size(scale, sizes, d, tokens, max_len):
    require_gpu()
    g = gen(68)
    lens, hk, heads, page = [1300, 77], 1, 5, 64
    *pool, table = poisoned_cache(g, lens, hk, page, d, -(-max(lens) // page))
    q = sized(torch.randn(2, tokens, heads, d, generator=g, device="cuda").bfloat16(), sizes)
    o, lse = decode_call(q, pool, table, lens, scale, max_len=max_len)
    assert L.losa_get_device_error() == 0
    check_decode(q, o, lse, pool, table, lens, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("scale,sizes", ROWS)
def test_block_rows_of_any_size(scale, sizes):
    require_gpu()
    g = gen(69)
    lens, page, heads, n = [900], 64, 2, 256
    *pool, table = poisoned_cache(g, lens, 1, page, 128, -(-max(lens) // page))
    q = sized(torch.randn(heads, n, 128, generator=g, device="cuda").bfloat16(), sizes)
    o, lse = blocks_call(q, pool, table, lens, page, heads, 1, n, scale)
    assert L.losa_get_device_error() == 0
    check_blocks(q, o, lse, pool, table, lens, page, heads, 1, n, scale, None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("d,lens,tokens,heads,max_len", [
    (128, [33, 3, 64], 3, 2, 64), (64, [96, 2, 1], 5, 4, 64), (128, [4000, 1025], 4, 4, 0), (64, [2049, 4000], 8, 4, 0),
    (128, [1500, 1499], 40, 2, 0)])
def test_decode_hides_later_tokens_whatever_they_hold(d, lens, tokens, heads, max_len):
    """NaN codes in the values or keys of a drafted token reach the rows that see it and no earlier one: a value's NaN in its
    own dimension, a key's in the whole row."""
    require_gpu()
    g = gen(66)
    page, hk, seqs = 32, 2, len(lens)
    width = -(-max(lens) // page)
    k8, v8, ks, vs, table = poisoned_cache(g, lens, hk, page, d, width)
    q = torch.randn(seqs, tokens, heads, d, generator=g, device="cuda").bfloat16()
    clean = decode_call(q, (k8, v8, ks, vs), table, lens, 0.1, max_len=max_len)
    for keys in (False, True):
        codes = [k8.clone(), v8.clone()]
        want = torch.zeros_like(q, dtype=torch.bool)
        for b, n in enumerate(lens):
            for back, dim in ((0, 3), (0, d - 1), (1, 0), (tokens // 2, 37), (tokens - 1, 5)):
                at = n - 1 - back  # a key that rows tokens - 1 - back and later see
                if at < 0:
                    continue
                codes[0 if keys else 1].view(torch.uint8)[int(table[b, at // page]), :, at % page, dim] = 0x7F | (0x80 * (back & 1))
                first = max(0, tokens - 1 - back)
                want[b, first:, :, slice(None) if keys else dim] = True
        o, lse = decode_call(q, (codes[0], codes[1], ks, vs), table, lens, 0.1, max_len=max_len)
        assert L.losa_get_device_error() == 0
        assert torch.equal(o.isnan(), want)
        assert torch.equal(o[~want], clean[0][~want])
        rows = want.all(-1)
        assert torch.equal(lse.isnan(), rows) and torch.equal(lse[~rows], clean[1][~rows])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_tokens_before_the_grid(dtype):
    """A negative start is a token before the grid's first: the one before (0, 0, 0) is (-1, gy - 1, gx - 1), as explicit
    positions say it."""
    require_gpu()
    g = gen(67)
    gy, gx, n, d = 5, 7, 90, 64
    x = torch.randn(1, 3, n, 2, d, generator=g, device="cuda").to(dtype)
    starts = [-1, -36, -1000003]
    a, b = torch.empty_like(x), torch.empty_like(x)
    rope = L.make_rope(d, (16, 22, 18), (gy, gx))
    L.losa_rope_apply(rope, x, a, start=ints(starts))
    tok = ints(starts).long()[:, None] + torch.arange(n, device="cuda")
    row = tok.div(gx, rounding_mode="floor")
    pos = torch.stack([row.div(gy, rounding_mode="floor"), row.remainder(gy), tok.remainder(gx)], -1)
    L.losa_rope_apply(rope, x, b, positions=pos.int().contiguous())
    assert L.losa_get_device_error() == 0
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_append_strides_of_single_extents():
    """One kv head, and one token: the stride that nothing steps by may be anything."""
    require_gpu()
    g = gen(74)
    d, page = 64, 32
    for tokens, hk, strides in ((7, 1, (2 * d, 5)), (1, 3, (13, 2 * d)), (1, 1, (3, 1))):
        base = torch.randn(2, 1000, generator=g, device="cuda").bfloat16()
        kv = [b.as_strided((tokens, hk, d), (*strides, 1)) for b in base]
        out = []
        for k, v in (kv, [t.contiguous() for t in kv]):
            pool = make_pool(gen(75), 2, hk, page, d)
            L.losa_cache_append(L.make_cache(hk, d, page, 2, 1, 2), k, v, *pool, ints([[1, 0]]), ints([30]), tokens)
            out.append(pool)
        assert L.losa_get_device_error() == 0
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*out))


@pytest.mark.gpu
def test_a_captured_harness_step_advances_with_every_replay():
    """KvCache.append and attend captured once and replayed token by token, with eager calls before, between and behind: the
    cache, its lengths and the outputs are what eager calls alone give."""
    require_gpu()
    from free_block_sparse_losa_b200.harness import KvCache
    g = gen(63)
    hk, d, heads, seqs = 2, 64, 4, 2
    rope = L.make_rope(d, (20, 22, 20), (3, 5))
    start = torch.randn(2, seqs * 50, hk, d, generator=g, device="cuda").bfloat16()
    steps = torch.randn(9, 2, seqs, hk, d, generator=g, device="cuda").bfloat16()
    qs = torch.randn(9, seqs, 1, heads, d, generator=g, device="cuda").bfloat16()

    def fresh():
        c = KvCache(seqs, hk, d, 96, page_tokens=32, rope=rope)
        c.append(start[0], start[1], 50)
        return c

    eager, want = fresh(), []
    for kv, q in zip(steps, qs):
        eager.append(kv[0], kv[1], 1)
        want.append(torch.empty_like(q))
        eager.attend(q, 0.2, want[-1])
    assert eager.lens.tolist() == [59, 59]

    cache = fresh()
    lens = cache.lens  # what a caller holds stays the cache's lengths
    kv, q, o = torch.empty_like(steps[0]), torch.empty_like(qs[0]), torch.empty_like(qs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(kv[0], kv[1], 1)
        cache.attend(q, 0.2, o)
    assert cache.lens.tolist() == [50, 50]  # nothing ran yet
    for i in range(9):
        if i in (0, 4):  # an eager step, before the first replay too
            got = torch.empty_like(qs[i])
            cache.append(steps[i, 0], steps[i, 1], 1)
            cache.attend(qs[i], 0.2, got)
        else:
            kv.copy_(steps[i])
            q.copy_(qs[i])
            graph.replay()
            got = o
        torch.cuda.synchronize()
        assert lens.tolist() == cache.lens.tolist() == [51 + i, 51 + i]
        assert cache.max_len >= 51 + i
        # the captured call's work may be split elsewhere: two bf16 roundings and the sums' order
        assert float((got.float() - want[i].float()).abs().max()) <= 2.0 ** -7 * float(want[i].float().abs().max())
    for a, b in zip(cache.buffers, eager.buffers):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert L.losa_get_device_error() == 0


@pytest.mark.gpu
def test_decode_with_a_raw_workspace():
    """The workspace as a device pointer and its size gives what the tensor gives; too small a size is refused."""
    require_gpu()
    g = gen(76)
    lens, hk, page, d, heads = [5000, 77], 1, 64, 64, 2
    *pool, table = poisoned_cache(g, lens, hk, page, d, -(-max(lens) // page))
    q = torch.randn(2, 1, heads, d, generator=g, device="cuda").bfloat16()
    want = decode_call(q, pool, table, lens, 0.1)
    cache = L.make_cache(hk, d, page, pool[0].shape[0], 2, table.shape[1])
    need = L.losa_cache_attn_workspace_bytes(cache, heads, 1)
    ws = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    for space in (ws.data_ptr(), ws):
        o, lse = torch.full_like(q, 9.0), torch.full((2, 1, heads), 9.0, device="cuda")
        assert L.losa_cache_attn(cache, q, *pool, table, ints(lens), 0.1, o, lse=lse, workspace=space, ws_bytes=need) == 0
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert L.losa_cache_attn(cache, q, *pool, table, ints(lens), 0.1, o, workspace=space, ws_bytes=need - 1,
                                 raise_on_error=False) == -3
    bare = lambda max_len: L.losa_cache_attn(cache, q, *pool, table, ints([900, 77]), 0.1, o, max_len=max_len,  # noqa: E731
                                             workspace=ws.data_ptr(), raise_on_error=False)
    assert bare(900) == 0 and bare(0) == -3  # without a size it counts as empty
    assert L.losa_get_device_error() == 0


@pytest.mark.gpu
def test_packing_on_a_side_stream():
    """pack_qkv on another stream while the current one still writes memory that it has given back to the allocator."""
    require_gpu()
    from free_block_sparse_losa_b200.harness import LayerBuffers
    g = gen(77)
    heads, n, d = 8, 1000, 128
    rope = L.make_rope(d, (44, 42, 42), (25, 20))
    layer = LayerBuffers(heads, n, 1024, d, 128, "bf16")
    qkv = torch.randn(1, n, 3, heads, d, generator=g, device="cuda").bfloat16()
    want = [t.clone() for t in layer.pack_qkv(qkv, rope)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        late = torch.empty(3, heads, 1024, d, dtype=torch.bfloat16, device="cuda")
        torch.cuda._sleep(20_000_000)  # about 10 ms
        late.fill_(5.0)
        del late  # its memory is free for the current stream's next tensor of this size, behind the fill
        got = layer.pack_qkv(qkv, rope, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got
    assert L.losa_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("theta", [1e-4, 0.3, 1.0, 1.0001, 37.5, 10000.0, 1e6, 1e30])
@pytest.mark.parametrize("halves", [False, True])
def test_rope_angles_at_far_positions(theta, halves):
    """Any theta, at positions over all of 32 bits, against angles in 60 decimal digits. The documented bound of an angle,
    |pos| 2^-58 / min(theta, 1) + 2^-33 turns, on top of what cosine, sine and the products are rounded by."""
    require_gpu()
    from decimal import Decimal, localcontext
    g = gen(73)
    d, dims = 64, (20, 22, 20)
    pos = [[2 ** 31 - 1, -2 ** 31, 1999999999], [1, -1, 0], [123456, -98765, 1 << 20], [-7, 1 << 30, 33]]
    x = torch.randn(1, 1, len(pos), 2, d, generator=g, device="cuda")
    y = torch.empty_like(x)
    L.losa_rope_apply(L.make_rope(d, dims, (4, 4), theta=theta, halves=halves), x, y, positions=ints([pos]))
    assert L.losa_get_device_error() == 0
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    xs, ys = x[0, 0].double().cpu(), y[0, 0].double().cpu()
    for i, triple in enumerate(pos):
        at = 0
        for p, m in zip(triple, dims):
            for j in range(m // 2):
                with localcontext() as ctx:
                    ctx.prec = 60
                    turns = Decimal(p) * (Decimal(theta) ** (Decimal(-2 * j) / m)) / (2 * pi)
                    angle = float((turns % 1) * 2 * pi)
                a, b = (at + j, at + m // 2 + j) if halves else (at + 2 * j, at + 2 * j + 1)
                c, s = math.cos(angle), math.sin(angle)
                off = 2 * math.pi * (abs(p) * 2.0 ** -58 / min(theta, 1.0) + 2.0 ** -33) + 6 * 2.0 ** -24
                size = xs[i, :, a].abs() + xs[i, :, b].abs()
                assert bool(((ys[i, :, a] - (xs[i, :, a] * c - xs[i, :, b] * s)).abs() <= off * size + 1e-38).all()), (p, j)
                assert bool(((ys[i, :, b] - (xs[i, :, a] * s + xs[i, :, b] * c)).abs() <= off * size + 1e-38).all()), (p, j)
            at += m


def codes_near(got, want, off):
    """Codes equal the reference rounded to e4m3, or that of a value at most `off` away."""
    near = [(want + s * off).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() for s in (0, 1, -1)]
    ok = (got.double() == near[0]) | (got.double() == near[1]) | (got.double() == near[2])
    assert bool(ok.all()), int((~ok).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,hk,halves", [(128, 128, 3, True), (64, 32, 5, False), (128, 64, 2, False)])
def test_append_of_many_fp32_pages(d, page, hk, halves):
    """Thousands of fp32 tokens in ragged sequences, against the 64-bit form. A rotated value is a c - b s in fp32: off by at
    most 6 * 2^-24 (|a| + |b|), which among millions of them is more than 1e-5 of a value that cancels to a few per cent, so
    the band around a rounding border is this bound (over the block's scale) and not a share of the value; a value that is not
    rotated is exact."""
    require_gpu()
    g = gen(72)
    held, new = [0, 77, page - 1, 500], [5000, 1, 3001, 0]
    seqs, width = 4, -(-5100 // page)
    pool = make_pool(g, seqs * width, hk, page, d)
    before = [t.clone() for t in pool]
    table = torch.randperm(seqs * width, generator=g, device="cuda").view(seqs, width).int()
    kv = torch.randn(sum(new), 2, hk, d, generator=g, device="cuda")
    ptr = [sum(new[:i]) for i in range(seqs + 1)]
    dims = (20, 22, 20) if d == 64 else (44, 42, 42)
    out = ints([0] * seqs)
    L.losa_cache_append(L.make_cache(hk, d, page, seqs * width, seqs, width), kv[:, 0], kv[:, 1], *pool, table, ints(held), 5000,
                        indptr=ints(ptr), new_lens=out, rope=L.make_rope(d, dims, (30, 52), halves=halves))
    assert L.losa_get_device_error() == 0
    assert out.tolist() == [h + m for h, m in zip(held, new)]
    per = [kv[ptr[b]:ptr[b + 1]].double() for b in range(seqs)]
    keys = [turn(x[:, 0], grid_positions(torch.arange(held[b], held[b] + new[b]), 30, 52)[:, None], dims, halves)
            for b, x in enumerate(per)]
    size = []  # |a| + |b| of every element of k
    for x in per:
        z, at = x[:, 0].abs().clone(), 0
        for m in dims:
            i = torch.arange(m // 2, device="cuda")
            a, b = (at + i, at + m // 2 + i) if halves else (at + 2 * i, at + 2 * i + 1)
            z[..., a] = z[..., b] = x[:, 0, :, a].abs() + x[:, 0, :, b].abs()
            at += m
        z[..., at:] = 0
        size.append(z)
    for x, codes, scale, was8, was, of in ((keys, pool[0], pool[2], before[0], before[2], size),
                                           ([x[:, 1] for x in per], pool[1], pool[3], before[1], before[3], None)):
        want, ws = append_reference(x, was8, was, table, held, new, page)
        assert torch.equal(scale.double(), ws)
        off = torch.zeros_like(want)
        for b in range(seqs if of else 0):
            for blk in range(held[b] // page, -(-(held[b] + new[b]) // page)):
                lo, hi = max(held[b] - blk * page, 0), min(page, held[b] + new[b] - blk * page)
                pg = int(table[b, blk])
                if hi > lo:
                    rows = of[b][blk * page + lo - held[b]:blk * page + hi - held[b]]
                    off[pg, :, lo:hi] = (6 * 2.0 ** -24 * rows / ws[pg][None, :, None]).transpose(0, 1)
        codes_near(codes, want, off)


@pytest.mark.gpu
def test_blocks_of_more_items_than_one_window():
    """More than 32 rounds of items a CTA (the reader's window): short lists, some empty, in a shuffled order."""
    require_gpu()
    g = gen(70)
    page, heads, n = 32, 24, 300 * 128 - 5
    items = heads * 300
    assert items > 33 * torch.cuda.get_device_properties(0).multi_processor_count
    lens = [1000]
    width = -(-lens[0] // page) + 1
    *pool, table = poisoned_cache(g, lens, 3, page, 128, width)
    q = torch.randn(heads, 300 * 128, 128, generator=g, device="cuda").bfloat16()
    indptr, blocks = random_lists(g, items, width, 1, 2, empty_every=11)
    order = torch.randperm(items, generator=g, device="cuda").int()
    o, lse = blocks_call(q, pool, table, lens, page, heads, 3, n, 0.03, indptr=indptr, kv_block_idx=blocks, order=order)
    assert L.losa_get_device_error() == 0
    check_blocks(q, o, lse, pool, table, lens, page, heads, 3, n, 0.03, indptr, blocks, items=sorted(order[::29].tolist()))
    again = blocks_call(q, pool, table, lens, page, heads, 3, n, 0.03, indptr=indptr, kv_block_idx=blocks)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d,hk,heads,tokens,seqs,top", [(128, 2, 4, 1, 70, 3000), (64, 1, 8, 4, 37, 5000), (128, 1, 40, 1, 33, 2000),
                                                        (128, 1, 24, 1, 3, 9000)])
def test_decode_of_many_ragged_sequences(d, hk, heads, tokens, seqs, top):
    """More sequences than a warp has lanes, and 17 to 40 rows to a kv head, in ranges that cross the sequences' borders."""
    require_gpu()
    g = gen(71)
    page = 64
    lens = [0 if b % 5 == 2 else max(1, (top * (b * 7919 % 101)) // 100) for b in range(seqs)]
    lens[-1] = top
    *pool, table = poisoned_cache(g, lens, hk, page, d, -(-top // page))
    q = torch.randn(seqs, tokens, heads, d, generator=g, device="cuda").bfloat16()
    o, lse = decode_call(q, pool, table, lens, 0.05)
    assert L.losa_get_device_error() == 0
    check_decode(q, o, lse, pool, table, lens, 0.05)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,max_len", [(1, 64), (3, 0)])
def test_scales_at_the_ends_of_their_range(tokens, max_len):
    """Value blocks at 2^-40, 1 and 2^60 next to each other: the quiet ones count in the denominator as the loud ones do. Key
    blocks at 2^-40 and 2^-6."""
    require_gpu()
    g = gen(78)
    lens, hk, page, heads, n = [1500, 200], 2, 64, 4, 256
    k8, v8, ks, vs, table = poisoned_cache(g, lens, hk, page, 128, -(-max(lens) // page))
    pick = lambda of: of[torch.randint(len(of), ks.shape, generator=g, device="cuda")]  # noqa: E731
    for b, count in enumerate(lens):
        used = table[b, :-(-count // page)].long()
        ks[used] = pick(torch.tensor([2.0 ** -40, 2.0 ** -6], device="cuda"))[used]
        vs[used] = pick(torch.tensor([2.0 ** -40, 1.0, 2.0 ** 60], device="cuda"))[used]
    pool = (k8, v8, ks, vs)
    q = torch.randn(2, tokens, heads, 128, generator=g, device="cuda").bfloat16()
    o, lse = decode_call(q, pool, table, lens, 0.1, max_len=max_len)
    check_decode(q, o, lse, pool, table, lens, 0.1)
    qb = torch.randn(2 * heads, n, 128, generator=g, device="cuda").bfloat16()
    indptr, blocks = random_lists(g, 2 * heads * 2, table.shape[1], 1, 9)
    for kw in ({}, dict(indptr=indptr, kv_block_idx=blocks)):
        o, lse = blocks_call(qb, pool, table, lens, page, heads, hk, n, 0.1, **kw)
        assert L.losa_get_device_error() == 0
        check_blocks(qb, o, lse, pool, table, lens, page, heads, hk, n, 0.1, kw.get("indptr"), kw.get("kv_block_idx"))


@pytest.mark.gpu
def test_captured_reads_follow_eager_appends():
    """A captured rotation that starts at the cache's lengths, a captured decode and a captured blocked call, replayed behind
    eager appends, give what eager calls give."""
    require_gpu()
    from free_block_sparse_losa_b200.harness import KvCache, LayerBuffers
    g = gen(79)
    hk, d, page = 2, 128, 32
    rope = L.make_rope(d, (44, 42, 42), (3, 5))
    cache = KvCache(1, hk, d, 400, page_tokens=page, rope=rope)
    layer = LayerBuffers(hk, 100, 128, d, 128, "bf16", block_k=page)
    kv = torch.randn(8, 2, 50, hk, d, generator=g, device="cuda").bfloat16()
    x, qb = torch.randn(1, 2, hk, d, generator=g, device="cuda").bfloat16(), torch.randn(hk, 128, d, generator=g, device="cuda").bfloat16()

    def step(r, o, ob, stream=None):
        L.losa_rope_apply(rope, x[None], r[None], start=cache.lens, stream=stream)
        cache.attend(r, 0.05, o, stream=stream)
        cache.sparse(layer, qb, 0.05, ob, lists=False, stream=stream)

    bufs = lambda: (torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(qb))  # noqa: E731
    cache.append(kv[0, 0], kv[0, 1], 50)
    step(*bufs())  # loads the kernels
    got, graph = bufs(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*got)
    for i in range(1, 8):
        cache.append(kv[i, 0], kv[i, 1], 50)
        graph.replay()
        want = bufs()
        step(*want)
        torch.cuda.synchronize()
        assert cache.lens.tolist() == [50 * (i + 1)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert L.losa_get_device_error() == 0
