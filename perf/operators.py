"""Measured cases of the streaming operators: rotary positions over (t, y, x), appending keys and values to a paged
8-bit cache, and attention over that cache for a few tokens and for listed blocks of 128 queries.

`run` with own = False is the plain form of each operator in elementary torch operations; with own = True it makes the
library calls. Sizes come from the layers of losa_synth (the 21x30x52 grid with 12 heads, the 21x45x80 grid with 40,
the 33x45x80 grid with 24) and from single steps of a stream."""
import functools
import math

import torch

own = False

FMT = torch.float8_e4m3fn
TOP = 448.0          # largest e4m3 value
E_MIN, E_MAX = -40, 60   # range of a block scale's exponent
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One new token in each of four streams: query and key rows of a step, in place of a whole clip.
        dict(name="rope-step", op="rope", parts=2, batch=4, heads=12, t=1, y=1, x=1, gy=30, gx=52, d=128, d0=44, d1=42,
             d2=42, dtype="bf16", halves=False, inverse=False, started=True),
        # The fused query/key/value projection of a 480p layer, to the head-major padded layout attention reads.
        dict(name="rope-480p-qkv", op="rope", parts=3, batch=1, heads=12, t=21, y=30, x=52, gy=30, gx=52, d=128, d0=44,
             d1=42, d2=42, dtype="bf16", halves=False, inverse=False, started=False),
        # The gradient of query and key on the largest layer, back to the projection's layout; halves pairing.
        dict(name="rope-720p-grad", op="rope", parts=2, batch=1, heads=24, t=33, y=45, x=80, gy=45, gx=80, d=128, d0=16,
             d1=56, d2=56, dtype="bf16", halves=True, inverse=True, started=False),
        # A small exact layer in 32 bits, two samples, an odd grid and a tail of unrotated dimensions.
        dict(name="rope-odd-f32", op="rope", parts=2, batch=2, heads=5, t=7, y=13, x=11, gy=13, gx=11, d=64, d0=16, d1=18,
             d2=22, dtype="f32", halves=True, inverse=False, started=False),
        # One token appended to each of 16 streams whose last page is part full.
        dict(name="append-token", op="append", seqs=16, kv_heads=8, d=128, page=128, held=1111, new=1, dtype="bf16", gy=30,
             gx=52, halves=False),
        # A whole 720p clip's keys and values entering an empty cache.
        dict(name="append-clip", op="append", seqs=1, kv_heads=24, d=128, page=128, held=0, new=118800, dtype="bf16",
             gy=45, gx=80, halves=False),
        # One token against a short cache: the latency of the smallest call.
        dict(name="decode-short", op="decode", seqs=1, heads=12, kv_heads=12, d=128, page=128, length=333, tokens=1,
             causal=True),
        # One token in each of eight streams of 480p length, ragged, four query heads to a key head.
        dict(name="decode-batch", op="decode", seqs=8, heads=40, kv_heads=10, d=128, page=128, length=32760, tokens=1,
             causal=True),
        # Four drafted tokens on two long streams, small pages.
        dict(name="decode-long", op="decode", seqs=2, heads=24, kv_heads=8, d=128, page=32, length=118800, tokens=4,
             causal=True),
        # The smallest blocked call: two heads, a few listed blocks each.
        dict(name="blocks-small", op="blocks", seqs=1, heads=2, kv_heads=2, page=128, queries=960, length=960, listed=3),
        # A 480p layer attending to its frozen lists at the density the mass threshold keeps, at 32-key blocks.
        dict(name="blocks-480p-lists", op="blocks", seqs=1, heads=12, kv_heads=12, page=32, queries=32760, length=32760,
             listed=16),
        # A chunk of three frames attending to everything held for the clip.
        dict(name="blocks-chunk-all", op="blocks", seqs=1, heads=12, kv_heads=12, page=128, queries=4680, length=32760,
             listed=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "blocks"])
    if op == "rope":
        d = rng.choice([64, 128])
        d0 = 2 * rng.randint(2, d // 8)
        d1 = 2 * rng.randint(2, d // 8)
        d2 = rng.choice([d - d0 - d1, 2 * rng.randint(2, d // 8)])
        t, y, x = _log(rng, 1, 33), _log(rng, 1, 45), _log(rng, 1, 80)
        return dict(op=op, parts=rng.randint(1, 3), batch=rng.randint(1, 3), heads=rng.randint(1, 8), t=t, y=y, x=x, gy=y,
                    gx=x, d=d, d0=d0, d1=d1, d2=d2, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    halves=rng.random() < 0.5, inverse=rng.random() < 0.4, started=rng.random() < 0.3)
    if op == "append":
        seqs = _log(rng, 1, 16)
        return dict(op=op, seqs=seqs, kv_heads=rng.randint(1, 16), d=rng.choice([64, 128, 128]),
                    page=rng.choice([32, 64, 128]), held=rng.randint(0, 3000), new=_log(rng, 1, 60000 // seqs),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), gy=rng.randint(1, 45), gx=rng.randint(1, 80),
                    halves=rng.random() < 0.5)
    if op == "decode":
        kv, g = rng.choice([1, 2, 5, 8, 12]), rng.choice([1, 2, 3, 4, 8])
        seqs = _log(rng, 1, 8)
        return dict(op=op, seqs=seqs, heads=kv * g, kv_heads=kv, d=rng.choice([64, 128, 128]),
                    page=rng.choice([32, 64, 128]), length=_log(rng, 1, 118800 // seqs), tokens=rng.randint(1, 5),
                    causal=rng.random() < 0.7)
    kv, g = rng.choice([1, 2, 4]), rng.choice([1, 1, 2, 3])
    page = rng.choice([32, 64, 128])
    return dict(op=op, seqs=rng.randint(1, 2), heads=kv * g, kv_heads=kv, page=page, queries=_log(rng, 1, 4680),
                length=_log(rng, 1, 32760), listed=rng.choice([0, 2, 5, 9]) * (128 // page))


# ------------------------------------------------------------------------------------------------------------- sizes

def _dims(case):
    """Rotated dimensions per axis of the append cases: the 44/42/42 split of 128, in proportion for 64."""
    return (44, 42, 42) if case["d"] == 128 else (20, 22, 20)


def _lengths(case, top):
    """Each sequence's length: from `top` down to about half of it, uneven; one of three or more is empty."""
    n = [max(1, top - b * max(1, top // (2 * case["seqs"])) - (b % 3)) if top else 0 for b in range(case["seqs"])]
    if case["seqs"] >= 3 and case["op"] == "decode":
        n[1] = 0
    return n


def _counts(case):
    """New tokens of each sequence of an append: ragged, the last of several adds none."""
    n = [max(1, case["new"] - b * (case["new"] // (2 * case["seqs"]))) for b in range(case["seqs"])]
    if case["seqs"] >= 3:
        n[-1] = 0
    return n


def _list_lengths(case):
    """Listed blocks of each (head, query block): 1 .. 2 * listed - 1, at most all; every ninth list of small layers
    is empty."""
    nq, nk = -(-case["queries"] // 128), -(-case["length"] // case["page"])
    items = case["seqs"] * case["heads"] * nq
    i = torch.arange(items, dtype=torch.int64)
    n = (1 + (i * 7919) % (2 * case["listed"] - 1)).clamp(max=nk)
    if items < 256:
        n[8::9] = 0
    return n


# ----------------------------------------------------------------------------------------------------------- prepare

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(g, pages, heads, page, d, keys):
    """A pool of pages holding quantised keys or values with per-page, per-head loudness; a few loud rows (sinks)."""
    x = _rand(g, pages, heads, page, d, dtype=torch.bfloat16)
    x *= torch.exp2(torch.randint(-2, 2, (pages, heads, 1, 1), generator=g, device="cuda").to(x.dtype)) if not keys else 1.5
    x[:, :, 0] *= 2.0
    amax = x.abs().amax((2, 3)).float()
    m, e = torch.frexp(amax / TOP)
    e = torch.where(m == 0.5, e - 1, e).clamp(E_MIN, E_MAX)
    s = torch.exp2(e.float())
    return (x / s[:, :, None, None].to(x.dtype)).to(FMT), s


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "rope":
        n, d, dt = case["t"] * case["y"] * case["x"], case["d"], DT[case["dtype"]]
        p, b, h = case["parts"], case["batch"], case["heads"]
        np_ = -(-n // 128) * 128
        token_major = (b, n, p, h, d)
        head_major = (p, b, h, np_, d)
        a, z = (head_major, token_major) if case["inverse"] else (token_major, head_major)
        s["x"] = _rand(g, *a, dtype=dt)
        s["y"] = torch.empty(*z, dtype=dt, device="cuda")
        s["start"] = _ints([1000 + 997 * i for i in range(b)]) if case["started"] else None
    elif case["op"] == "append":
        held, new = _lengths(case, case["held"]), _counts(case)
        page, hk, d = case["page"], case["kv_heads"], case["d"]
        width = max(-(-(a + b) // page) for a, b in zip(held, new))
        pages = width * case["seqs"] + 1
        s["k8"], s["ks"] = _cache(g, pages, hk, page, d, True)
        s["v8"], s["vs"] = _cache(g, pages, hk, page, d, False)
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[:width * case["seqs"]].view(case["seqs"], width).int()
        s["lens"], s["new_lens"] = _ints(held), _ints([0] * case["seqs"])
        s["indptr"] = _ints([sum(new[:i]) for i in range(case["seqs"] + 1)])
        # keys louder than what the part-full pages hold in some heads, so that some scales grow
        kv = _rand(g, sum(new), 2, hk, d, dtype=DT[case["dtype"]])
        kv *= 1.0 + 2.0 * (torch.arange(hk, device="cuda") % 3 == 1).to(kv.dtype)[:, None]
        s["kv"] = kv
        s["bound"] = max(new)
    else:
        tokens = case["tokens"] if case["op"] == "decode" else 1
        lens = _lengths(case, max(case["length"], tokens))
        lens = [max(v, tokens) if v else 0 for v in lens]
        page, hk = case["page"], case["kv_heads"]
        d = case["d"] if case["op"] == "decode" else 128
        width = -(-max(lens) // page)
        pages = width * case["seqs"] + 1
        s["k8"], s["ks"] = _cache(g, pages, hk, page, d, True)
        s["v8"], s["vs"] = _cache(g, pages, hk, page, d, False)
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[:width * case["seqs"]].view(case["seqs"], width).int()
        s["lens"], s["max_len"] = _ints(lens), max(lens)
        s["scale"] = 1.0 / math.sqrt(d)
        if case["op"] == "decode":
            s["q"] = _rand(g, case["seqs"], tokens, case["heads"], d, dtype=torch.bfloat16) * 1.5
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(case["seqs"], tokens, case["heads"], device="cuda")
            # scratch of a decoding loop, kept for all its steps: partial results of at most 128 splits of a sequence
            rows = case["seqs"] * tokens * case["heads"]
            s["ws"] = torch.empty(rows * 128 * (d + 4) * 4 + 4096, dtype=torch.uint8, device="cuda")
        else:
            nq = -(-case["queries"] // 128)
            h = case["seqs"] * case["heads"]
            s["q"] = _rand(g, h, nq * 128, 128, dtype=torch.bfloat16) * 1.5
            s["q"][:, case["queries"]:] = 0
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(h, nq * 128, device="cuda")
            s["indptr"] = s["blocks"] = s["order"] = None
            s["longest"] = 0
            if case["listed"]:
                counts = _list_lengths(case).cuda()
                near = (torch.arange(nq, device="cuda")[:, None] * width / nq
                        - torch.arange(width, device="cuda")[None]).abs() / max(1, width / 8)
                noise = torch.rand(h, nq, width, generator=g, device="cuda") + near
                s["longest"] = int(counts.max())
                best = noise.view(h * nq, width).argsort(1)[:, :s["longest"]]
                keep = torch.arange(s["longest"], device="cuda")[None] < counts[:, None]
                best = torch.where(keep, best, width).sort(1).values
                s["blocks"] = best[keep].int().contiguous()
                s["indptr"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
                s["order"] = torch.argsort(counts, descending=True, stable=True).int()
    return s


# --------------------------------------------------------------------------------------------------- the library's calls

@functools.lru_cache(maxsize=None)
def _rope(d, dims, gy, gx, halves):
    import free_block_sparse_losa_b200 as L
    return L.make_rope(d, dims, grid=(gy, gx), theta=10000.0, halves=halves)


@functools.lru_cache(maxsize=None)
def _pool(kv_heads, d, page, pages, seqs, width):
    import free_block_sparse_losa_b200 as L
    return L.make_cache(kv_heads, d, page, pages, seqs, width)


@functools.lru_cache(maxsize=None)
def _shape(heads, n, padded, page):
    import free_block_sparse_losa_b200 as L
    return L.make_shape(heads, n, padded, 128, 128, page, "bf16")


def _rope_views(s):
    """x and y as (parts, batch, tokens, heads, d) views of their layouts."""
    token, head = (2, 0, 1, 3, 4), (0, 1, 3, 2, 4)
    a, b = (head, token) if s["case"]["inverse"] else (token, head)
    return s["x"].permute(a), s["y"].permute(b)


def _run_own(s):
    import free_block_sparse_losa_b200 as L
    c = s["case"]
    if c["op"] == "rope":
        x, y = _rope_views(s)
        n = c["t"] * c["y"] * c["x"]
        L.losa_rope_apply(_rope(c["d"], (c["d0"], c["d1"], c["d2"]), c["gy"], c["gx"], c["halves"]), x[:, :, :n], y,
                          rotate=3 if c["parts"] > 1 else 1, inverse=c["inverse"], start=s["start"])
        return s["y"]
    pages, hk, page, d = s["k8"].shape
    pool = _pool(hk, d, page, pages, s["table"].shape[0], s["table"].shape[1])
    if c["op"] == "append":
        L.losa_cache_append(pool, s["kv"][:, 0], s["kv"][:, 1], s["k8"], s["v8"], s["ks"], s["vs"], s["table"], s["lens"],
                            new_tokens=s["bound"], indptr=s["indptr"], new_lens=s["new_lens"],
                            rope=_rope(d, _dims(c), c["gy"], c["gx"], c["halves"]))
        return s["k8"], s["v8"], s["ks"], s["vs"], s["new_lens"]
    if c["op"] == "decode":
        L.losa_cache_attn(pool, s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"], s["o"],
                          lse=s["lse"], causal=c["causal"], max_len=s["max_len"], workspace=s["ws"])
        return s["o"], s["lse"]
    shape = _shape(s["q"].shape[0], c["queries"], s["q"].shape[1], page)
    L.losa_cache_sparse_attn(shape, pool, s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"],
                             s["o"], indptr=s["indptr"], kv_block_idx=s["blocks"], order=s["order"], lse=s["lse"])
    return s["o"][:, :c["queries"]], s["lse"][:, :c["queries"]]


# ------------------------------------------------------------------------------------------------------- the plain form

def _angles(pos, dims, theta=10000.0):
    """cos and sin of every rotated pair, (..., pairs): pair i of an axis of m dimensions turns by pos * theta^(-2i/m).
    Angles in 64 bits (far positions), their cosines rounded to 32."""
    a = torch.cat([pos[..., k:k + 1].double() * theta ** (-torch.arange(0, m, 2, device=pos.device, dtype=torch.float64) / m)
                   for k, m in enumerate(dims)], -1)
    return a.cos().float(), a.sin().float()


def _pairs(dims, halves, device):
    """Indices of the first and second member of every rotated pair."""
    base = [sum(dims[:k]) for k in range(3)]
    one = [torch.arange(m // 2, device=device) * (1 if halves else 2) + b for m, b in zip(dims, base)]
    two = [i + (m // 2 if halves else 1) for i, m in zip(one, dims)]
    return torch.cat(one), torch.cat(two)


def _grid_position(n, gy, gx):
    return torch.stack([n // (gy * gx), n // gx % gy, n % gx], -1)


def _turn(x, cos, sin, dims, halves, inverse=False):
    """x (..., d) in 32 bits, rotated by the angles (broadcast over what lies between)."""
    i, j = _pairs(dims, halves, x.device)
    a, b = x[..., i], x[..., j]
    if inverse:
        sin = -sin
    y = x.clone()
    y[..., i] = a * cos - b * sin
    y[..., j] = a * sin + b * cos
    return y


def _plain_rope(s):
    c = s["case"]
    n = c["t"] * c["y"] * c["x"]
    x, y = _rope_views(s)
    x = x[:, :, :n]
    dims = (c["d0"], c["d1"], c["d2"])
    at = torch.arange(n, device=x.device)[None] + (s["start"].long()[:, None] if c["started"] else 0)
    cos, sin = _angles(_grid_position(at.expand(c["batch"], n), c["gy"], c["gx"]), dims)
    turned = _turn(x[:2].float(), cos[None, :, :, None], sin[None, :, :, None], dims, c["halves"], c["inverse"])
    y[:2, :, :n] = turned.to(y.dtype)
    y[2:, :, :n] = x[2:]
    y[:, :, n:] = 0
    return s["y"]


def _plain_append(s):
    c = s["case"]
    page, hk, d = c["page"], c["kv_heads"], c["d"]
    lens, ptr = s["lens"].long(), s["indptr"].long()
    tok = torch.arange(s["kv"].shape[0], device="cuda")
    seq = torch.searchsorted(ptr[1:], tok, right=True)
    at = lens[seq] + tok - ptr[seq]
    pg, slot = s["table"][seq, at // page].long(), at % page
    cos, sin = _angles(_grid_position(at, c["gy"], c["gx"]), _dims(c))
    k = _turn(s["kv"][:, 0].float(), cos[:, None], sin[:, None], _dims(c), c["halves"])
    v = s["kv"][:, 1].float()
    # what the part-full pages hold keeps its scale or takes a larger one
    last = s["table"].gather(1, (lens // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    grows = (lens % page > 0) & (ptr[1:] > ptr[:-1])
    for x, codes, scale in ((k, s["k8"], s["ks"]), (v, s["v8"], s["vs"])):
        amax = torch.zeros(codes.shape[0], hk, device="cuda").index_reduce_(0, pg, x.abs().amax(-1), "amax")
        m, e = torch.frexp(amax / TOP)
        e = torch.where(m == 0.5, e - 1, e).clamp(E_MIN, E_MAX)
        new = torch.where(amax > 0, torch.exp2(e.float()), 2.0 ** E_MIN)
        old = torch.zeros_like(new)
        old[last[grows]] = scale[last[grows]]
        new = torch.maximum(new, old)
        touched = torch.zeros(codes.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, pg, True)
        held = codes[last[grows]].float() * (old[last[grows]] / new[last[grows]])[:, :, None, None]
        stays = (torch.arange(page, device="cuda") >= (lens[grows] % page)[:, None])[:, None, :, None]
        codes[last[grows]] = torch.where(stays, codes[last[grows]].float(), held).to(FMT)
        codes.view(torch.uint8)[pg, :, slot] = (x / new[pg][:, :, None]).clamp(-TOP, TOP).to(FMT).view(torch.uint8)
        scale[touched] = new[touched]
    s["new_lens"].copy_(lens + ptr[1:] - ptr[:-1])
    return s["k8"], s["v8"], s["ks"], s["vs"], s["new_lens"]


def _attend(q, k, v, seen):
    """softmax over the seen keys and its log-sum-exp; rows that see nothing give 0 and -inf. q already scaled."""
    x = (q @ k.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l.clamp(min=1e-38)
    return o, (m + l.log())[..., 0]


def _plain_decode(s):
    c = s["case"]
    b, m, h, d = s["q"].shape
    hk = c["kv_heads"]
    at = s["table"].long()
    k = (s["k8"][at].float() * s["ks"][at][..., None, None]).transpose(1, 2).reshape(b, hk, -1, d)
    v = (s["v8"][at].float() * s["vs"][at][..., None, None]).transpose(1, 2).reshape(b, hk, -1, d)
    q = (s["q"].float() * s["scale"]).view(b, m, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    end = s["lens"].long()[:, None]
    if c["causal"]:
        end = end - m + 1 + torch.arange(m, device="cuda")[None]
    seen = torch.arange(k.shape[2], device="cuda") < end.expand(b, m)[..., None]
    o, lse = _attend(q, k, v, seen[:, None, :, None].expand(b, 1, m, h // hk, -1).reshape(b, 1, m * (h // hk), -1))
    o = o.view(b, hk, m, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, m, h, d)
    return o.to(torch.bfloat16), lse.view(b, hk, m, h // hk).permute(0, 2, 1, 3).reshape(b, m, h)


def _plain_blocks(s):
    c = s["case"]
    b, h, hk, page, n = c["seqs"], c["heads"], c["kv_heads"], c["page"], c["queries"]
    q = s["q"].float() * s["scale"]
    if s["blocks"] is None:
        at = s["table"].long()
        k = (s["k8"][at].float() * s["ks"][at][..., None, None]).transpose(1, 2).reshape(b, hk, 1, -1, 128)
        v = (s["v8"][at].float() * s["vs"][at][..., None, None]).transpose(1, 2).reshape(b, hk, 1, -1, 128)
        seen = torch.arange(k.shape[3], device="cuda") < s["lens"].long()[:, None]
        o, lse = _attend(q.view(b, hk, h // hk, -1, 128), k, v, seen[:, None, None, None])
    else:
        nq = s["q"].shape[1] // 128
        item = torch.arange(b * h * nq, device="cuda")
        seq, kvh = item // (h * nq), item // nq % h // (h // hk)
        slot = torch.arange(s["longest"], device="cuda")[None]
        ptr = s["indptr"].long()
        real = slot < (ptr[1:] - ptr[:-1])[:, None]
        blk = s["blocks"].long()[(ptr[:-1, None] + slot).clamp(max=s["blocks"].numel() - 1)]
        pg = s["table"].long()[seq[:, None], blk]
        k = (s["k8"][pg, kvh[:, None]].float() * s["ks"][pg, kvh[:, None]][..., None, None]).view(len(item), -1, 128)
        v = (s["v8"][pg, kvh[:, None]].float() * s["vs"][pg, kvh[:, None]][..., None, None]).view(len(item), -1, 128)
        key = blk[..., None] * page + torch.arange(page, device="cuda")
        seen = (real[..., None] & (key < s["lens"].long()[seq][:, None, None])).view(len(item), 1, -1)
        o, lse = _attend(q.view(len(item), 128, 128), k, v, seen)
    return o.reshape(b * h, -1, 128)[:, :n].to(torch.bfloat16), lse.reshape(b * h, -1)[:, :n]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "append":
        return _plain_append(state)
    if op == "decode":
        return _plain_decode(state)
    return _plain_blocks(state)


# --------------------------------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["t"] * case["y"] * case["x"]
        lanes = case["parts"] * case["batch"] * case["heads"] * case["d"]
        written = n if case["inverse"] else -(-n // 128) * 128
        return {"bytes": lanes * (n + written) * size, "flops": 3.0 * n * lanes}
    if case["op"] == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        lanes = 2 * sum(_counts(case)) * case["kv_heads"] * case["d"]
        return {"bytes": lanes * (size + 1), "flops": 4.0 * lanes}
    tokens = case["tokens"] if case["op"] == "decode" else 1
    lens = [max(v, tokens) if v else 0 for v in _lengths(case, max(case["length"], tokens))]
    if case["op"] == "decode":
        rows = case["heads"] * tokens
        return {"bytes": 2 * sum(lens) * case["kv_heads"] * case["d"] + case["seqs"] * rows * (4 * case["d"] + 4),
                "flops": 4.0 * rows * sum(lens) * case["d"]}
    nq, page = -(-case["queries"] // 128), case["page"]
    if case["listed"]:
        keys = int(_list_lengths(case).sum()) * page
        held = min(keys * case["kv_heads"] // case["heads"], sum(lens) * case["kv_heads"])
    else:
        keys = sum(lens) * case["heads"] * nq
        held = sum(lens) * case["kv_heads"]
    rows = case["seqs"] * case["heads"] * nq * 128
    return {"bytes": 2 * held * 128 + rows * (4 * 128 + 4), "flops": 4.0 * 128 * keys * 128}


# -------------------------------------------------------------------------------------------------------------- exact

def _spin(x, pos, dims, halves, sign):
    """x (N, heads, d) in 64 bits, each pair taken as a complex number and turned."""
    out, at = x.clone(), 0
    for axis, m in enumerate(dims):
        part = x[..., at:at + m]
        z = torch.complex(part[..., :m // 2], part[..., m // 2:]) if halves else torch.view_as_complex(
            part.reshape(*part.shape[:-1], m // 2, 2).contiguous())
        f = torch.tensor([10000.0 ** (-2.0 * i / m) for i in range(m // 2)], dtype=torch.float64, device=x.device)
        w = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), sign * pos[:, axis].double()[:, None] * f)
        z = z * w[:, None]
        out[..., at:at + m] = torch.cat([z.real, z.imag], -1) if halves else torch.view_as_real(z).reshape(part.shape)
        at += m
    return out


def _exact_rows(q, k, v, scale):
    """Attention of rows q (r, d) over the keys k (n, d), in 64 bits."""
    if not len(k):
        return torch.zeros_like(q), torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=q.device)
    x = scale * torch.einsum("rd,nd->rn", q, k)
    lse = torch.logsumexp(x, 1)
    return torch.einsum("rn,nd->rd", torch.exp(x - lse[:, None]), v), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        n, gy, gx = case["t"] * case["y"] * case["x"], case["gy"], case["gx"]
        x, y = _rope_views(s)
        out = torch.zeros_like(s["y"], dtype=torch.float64)
        view = out.permute((2, 0, 1, 3, 4) if case["inverse"] else (0, 1, 3, 2, 4))
        for p in range(case["parts"]):
            for b in range(case["batch"]):
                at = torch.arange(n, device="cuda") + (int(s["start"][b]) if case["started"] else 0)
                row = x[p, b, :n].double()
                if p < 2:
                    pos = torch.stack([at.div(gy * gx, rounding_mode="floor"), at.remainder(gy * gx).div(gx, rounding_mode="floor"),
                                       at.remainder(gx)], 1)
                    row = _spin(row, pos, (case["d0"], case["d1"], case["d2"]), case["halves"], -1.0 if case["inverse"] else 1.0)
                view[p, b, :n] = row
        return out
    page = case["page"]
    if case["op"] == "append":
        held, new, d = _lengths(case, case["held"]), _counts(case), case["d"]
        k8, v8, ks, vs = s["k8"].double(), s["v8"].double(), s["ks"].double(), s["vs"].double()
        first = 0
        for b in range(case["seqs"]):
            if not new[b]:
                continue
            at = torch.arange(held[b], held[b] + new[b], device="cuda")
            gy, gx = case["gy"], case["gx"]
            pos = torch.stack([at.div(gy * gx, rounding_mode="floor"), at.remainder(gy * gx).div(gx, rounding_mode="floor"), at.remainder(gx)], 1)
            rows = s["kv"][first:first + new[b]].double()
            first += new[b]
            for codes, scale, x in ((k8, ks, _spin(rows[:, 0], pos, _dims(case), case["halves"], 1.0)), (v8, vs, rows[:, 1])):
                lo, hi = held[b] // page, -(-(held[b] + new[b]) // page)
                skip = held[b] - lo * page
                span = torch.zeros((hi - lo) * page, *x.shape[1:], dtype=torch.float64, device="cuda")
                span[skip:skip + new[b]] = x
                pg = s["table"][b, lo:hi].long()
                loud = span.view(hi - lo, page, -1, d).abs().amax((1, 3))
                e = torch.ceil(torch.log2(loud / TOP)).clamp(E_MIN, E_MAX)
                grown = torch.exp2(e)
                before = scale[pg]
                if skip:
                    grown[0] = torch.maximum(grown[0], before[0])
                was = codes[pg].clone()
                codes[pg] = torch.where(
                    ((torch.arange((hi - lo) * page, device="cuda") >= skip) & (torch.arange((hi - lo) * page, device="cuda") < skip + new[b])).view(hi - lo, 1, page, 1),
                    (span.view(hi - lo, page, -1, d).transpose(1, 2) / grown[:, :, None, None]).clamp(-TOP, TOP), was)
                if skip:
                    codes[pg[0], :, :skip] = was[0][:, :skip] * (before[0] / grown[0])[:, None, None]
                scale[pg] = grown
        return k8, v8, ks, vs, None
    b, hk, g = case["seqs"], case["kv_heads"], case["heads"] // case["kv_heads"]
    lens = [int(v) for v in s["lens"]]
    if case["op"] == "decode":
        tokens = case["tokens"]
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
        for i in range(b):
            pg = s["table"][i].long()
            for j in range(hk):
                k = (s["k8"][pg, j].double() * s["ks"][pg, j].double()[:, None, None]).flatten(0, 1)
                v = (s["v8"][pg, j].double() * s["vs"][pg, j].double()[:, None, None]).flatten(0, 1)
                for t in range(tokens):
                    end = max(0, lens[i] - (tokens - 1 - t if case["causal"] else 0))
                    at = slice(j * g, (j + 1) * g)
                    o[i, t, at], lse[i, t, at] = _exact_rows(s["q"][i, t, at].double(), k[:end], v[:end], s["scale"])
        return o, lse
    n = case["queries"]
    nq = -(-n // 128)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    ptr = s["indptr"].tolist() if s["blocks"] is not None else None
    for h in range(b * case["heads"]):
        i, j = h // case["heads"], h % case["heads"] // g
        pg = s["table"][i].long()
        k = (s["k8"][pg, j].double() * s["ks"][pg, j].double()[:, None, None]).flatten(0, 1)
        v = (s["v8"][pg, j].double() * s["vs"][pg, j].double()[:, None, None]).flatten(0, 1)
        if ptr is None:
            o[h], lse[h] = _exact_rows(s["q"][h].double(), k[:lens[i]], v[:lens[i]], s["scale"])
            continue
        for t in range(nq):
            at = s["blocks"][ptr[h * nq + t]:ptr[h * nq + t + 1]].long()
            key = (at[:, None] * page + torch.arange(page, device="cuda")).flatten()
            key = key[key < lens[i]]
            rows = slice(t * 128, t * 128 + 128)
            o[h, rows], lse[h, rows] = _exact_rows(s["q"][h, rows].double(), k[key], v[key], s["scale"])
    return o[:, :n], lse[:, :n]
