"""CPU checks of the streaming entry points: host-side refusals before anything is launched, and the binding's checks of
tensors. No call here reaches the CUDA runtime."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

import free_block_sparse_losa_b200 as L
from free_block_sparse_losa_b200 import build as B

FAKE = 0x10000  # aligned, never dereferenced
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def view(parts=2, batch=1, tokens=5, heads=3, d=128, **over):
    f = dict(parts=parts, batch=batch, tokens=tokens, heads=heads, part_stride=heads * tokens * d,
             batch_stride=parts * heads * tokens * d, token_stride=d, head_stride=tokens * d)
    f.update(over)
    return L.LosaTokenView(*[f[k] for k, _ in L.LosaTokenView._fields_])


def rope_call(lib, rope=None, x=None, y=None, px=FAKE, py=2 * FAKE, dtype=1, pos=None, start=None):
    rope = L.make_rope(128, (44, 42, 42), (4, 4)) if rope is None else rope
    return lib.losa_rope_apply(ctypes.byref(rope), dtype, ctypes.byref(x or view()), px, ctypes.byref(y or view()), py, 1, 0,
                               pos, start, 0)


def test_rope_refusals(lib):
    bad_ropes = [L.make_rope(128, (43, 42, 42), (4, 4)),          # odd axis
                 L.make_rope(128, (64, 64, 2), (4, 4)),           # more than the row
                 L.make_rope(128, (-2, 64, 64), (4, 4)),
                 L.make_rope(128, (44, 42, 42), (0, 4)),          # empty grid
                 L.make_rope(128, (44, 42, 42), (4, 4), theta=0.0),
                 L.make_rope(128, (44, 42, 42), (4, 4), theta=float("inf")),
                 L.make_rope(0, (0, 0, 0), (4, 4)),
                 L.make_rope(264, (44, 42, 42), (4, 4))]          # head_dim above 256
    weird = L.make_rope(128, (44, 42, 42), (4, 4))
    weird.pairing = 2
    for r in bad_ropes + [weird]:
        assert rope_call(lib, rope=r) == INVALID
    for over in (dict(heads=0), dict(tokens=-1), dict(token_stride=4), dict(head_stride=-128), dict(parts=0)):
        assert rope_call(lib, x=view(**over)) == INVALID
    assert rope_call(lib, y=view(tokens=4)) == INVALID                      # fewer rows than x
    assert rope_call(lib, y=view(heads=2)) == INVALID
    assert rope_call(lib, y=view(token_stride=0)) == INVALID                # rows written over each other
    assert rope_call(lib, px=FAKE + 8) == INVALID
    assert rope_call(lib, px=FAKE, py=FAKE) == INVALID
    assert rope_call(lib, px=None) == INVALID
    assert rope_call(lib, pos=FAKE + 2) == INVALID
    assert rope_call(lib, start=FAKE + 1) == INVALID
    assert rope_call(lib, dtype=5) == INVALID
    assert lib.losa_rope_apply(None, 1, None, None, None, None, 1, 0, None, None, 0) == INVALID
    # a row that is not a multiple of 16 bytes
    assert rope_call(lib, rope=L.make_rope(20, (4, 4, 4), (4, 4)), x=view(d=24), y=view(d=24)) == UNSUPPORTED
    assert rope_call(lib, x=view(parts=33), y=view(parts=33)) == UNSUPPORTED
    assert rope_call(lib, x=view(tokens=0), y=view(tokens=0)) == 0          # nothing to do


def append_call(lib, cache=None, rope=None, dtype=1, k=FAKE, strides=(1024, 128, 1024, 128), total=8, new=4, indptr=FAKE,
                table=FAKE, lens=FAKE, new_lens=2 * FAKE, k8=FAKE, ks=FAKE, pos=None):
    cache = cache or L.make_cache(8, 128, 128, 10, 2, 5)
    return lib.losa_cache_append(ctypes.byref(cache), None if rope is None else ctypes.byref(rope), dtype, k, strides[0],
                                 strides[1], FAKE, strides[2], strides[3], total, new, indptr, pos, table, lens, new_lens, k8,
                                 FAKE, ks, FAKE, 0)


BAD_CACHES = [L.make_cache(0, 128, 128, 10, 2, 5), L.make_cache(8, 128, 0, 10, 2, 5), L.make_cache(8, 128, 128, 0, 2, 5),
              L.make_cache(8, 128, 128, 10, 0, 5), L.make_cache(8, 128, 128, 10, 2, 0),
              L.make_cache(8, 128, 128, 10, 2, 1 << 25)]
ODD_CACHES = [L.make_cache(8, 96, 128, 10, 2, 5), L.make_cache(8, 128, 48, 10, 2, 5), L.make_cache(8, 128, 256, 10, 2, 5),
              L.make_cache(8, 128, 128, 10, 70000, 5), L.make_cache(8, 128, 128, 1 << 22, 2, 5)]


def test_append_refusals(lib):
    for c in BAD_CACHES:
        assert append_call(lib, cache=c) == INVALID
    for c in ODD_CACHES:
        assert append_call(lib, cache=c) == UNSUPPORTED
    assert append_call(lib, rope=L.make_rope(64, (16, 16, 16), (4, 4))) == INVALID  # another head_dim
    for over in (dict(dtype=2), dict(strides=(1023, 128, 1024, 128)), dict(strides=(1024, 128, -8, 128)), dict(new=-1),
                 dict(total=-1), dict(k=FAKE + 2), dict(k=None), dict(table=None), dict(lens=None), dict(lens=2 * FAKE),
                 dict(k8=FAKE + 4), dict(ks=FAKE + 2), dict(indptr=FAKE + 2), dict(pos=FAKE + 2), dict(new_lens=FAKE + 2),
                 dict(indptr=None, new=5)):  # 2 sequences x 5 tokens of 8
        assert append_call(lib, **over) == INVALID, over
    assert lib.losa_cache_append(None, None, 1, FAKE, 0, 0, FAKE, 0, 0, 0, 0, *[None] * 10) == INVALID


def attn_call(lib, cache=None, heads=16, tokens=2, q=FAKE, o=2 * FAKE, strides=(4096, 2048, 128, 4096, 2048, 128), scale=0.1,
              table=FAKE, lens=FAKE, k8=FAKE, ks=FAKE, lse=None, max_len=64):
    cache = cache or L.make_cache(8, 128, 128, 10, 2, 5)
    return lib.losa_cache_attn(ctypes.byref(cache), heads, tokens, 1, q, *strides[:3], table, lens, k8, FAKE, ks, FAKE, scale,
                               max_len, o, *strides[3:], lse, None, 0, 0)


def test_attn_refusals(lib):
    for c in BAD_CACHES:
        assert attn_call(lib, cache=c) == INVALID
        assert L.losa_cache_attn_workspace_bytes(c, 16, 1) == 0
    for c in ODD_CACHES:
        assert attn_call(lib, cache=c) == UNSUPPORTED
        assert L.losa_cache_attn_workspace_bytes(c, 16, 1) == 0
    for over in (dict(heads=12), dict(heads=0), dict(tokens=0), dict(q=FAKE + 4), dict(q=None), dict(o=FAKE), dict(o=None),
                 dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(table=FAKE + 1),
                 dict(lens=None), dict(k8=FAKE + 8), dict(ks=None), dict(lse=FAKE + 2),
                 dict(strides=(4096, 2048, 100, 4096, 2048, 128)), dict(strides=(4096, 2048, 128, 4096, 2048, 64)),
                 dict(strides=(4096, -2048, 128, 4096, 2048, 128))):
        assert attn_call(lib, **over) == INVALID, over


def sparse_call(lib, shape=None, cache=None, q=FAKE, o=2 * FAKE, scale=0.1, indptr=FAKE, idx=FAKE, order=None, lse=None,
                table=FAKE):
    shape = shape or L.make_shape(16, 200, 256, 128, 128, 32, "bf16")
    cache = cache or L.make_cache(8, 128, 32, 10, 2, 5)
    return lib.losa_cache_sparse_attn(ctypes.byref(shape), ctypes.byref(cache), q, table, FAKE, FAKE, FAKE, FAKE, FAKE, scale,
                                      indptr, idx, order, o, lse, 0)


def test_sparse_refusals(lib):
    for s in (L.make_shape(16, 300, 256, 128, 128, 32, "bf16"),   # more tokens than rows
              L.make_shape(16, 200, 256, 128, 128, 64, "bf16"),   # another block than the cache's pages
              L.make_shape(16, 200, 256, 64, 128, 32, "bf16"),    # another head_dim
              L.make_shape(15, 200, 256, 128, 128, 32, "bf16"),   # heads do not fall into sequences
              L.make_shape(24, 200, 256, 128, 128, 32, "bf16")):  # nor into kv heads
        assert sparse_call(lib, shape=s) == INVALID
    for c in BAD_CACHES:
        assert sparse_call(lib, cache=c) == INVALID
    for over in (dict(q=FAKE + 2), dict(o=FAKE), dict(scale=0.0), dict(scale=float("nan")), dict(indptr=None), dict(idx=None),
                 dict(indptr=FAKE + 2), dict(order=FAKE + 1), dict(lse=FAKE + 4), dict(table=None)):
        assert sparse_call(lib, **over) == INVALID, over
    for s in (L.make_shape(16, 200, 256, 128, 64, 32, "bf16"), L.make_shape(16, 200, 256, 128, 128, 32, "f32")):
        assert sparse_call(lib, shape=s) == UNSUPPORTED


def test_binding_refuses_wrong_tensors(lib):
    rope = L.make_rope(128, (44, 42, 42), (4, 4))
    t = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="expected torch.bfloat16 or torch.float32"):
        L.losa_rope_apply(rope, t(1, 1, 4, 2, 128, dt=torch.float16), t(1, 1, 4, 2, 128))
    with pytest.raises(ValueError, match="y: expected torch.bfloat16"):
        L.losa_rope_apply(rope, t(1, 1, 4, 2, 128), t(1, 1, 4, 2, 128, dt=torch.float32))
    with pytest.raises(ValueError, match="expected .parts, batch, tokens, heads, 128."):
        L.losa_rope_apply(rope, t(1, 4, 2, 128), t(1, 1, 4, 2, 128))
    with pytest.raises(ValueError, match="x: the last dimension"):
        L.losa_rope_apply(rope, t(1, 1, 4, 2, 256)[..., ::2], t(1, 1, 4, 2, 128))
    with pytest.raises(ValueError, match="start: holds"):
        L.losa_rope_apply(rope, t(1, 2, 4, 2, 128), t(1, 2, 4, 2, 128), start=t(1, dt=torch.int32))
    with pytest.raises(ValueError, match="positions: holds"):
        L.losa_rope_apply(rope, t(1, 2, 4, 2, 128), t(1, 2, 4, 2, 128), positions=t(23, dt=torch.int32))
    with pytest.raises(ValueError, match="x: expected a CUDA tensor"):
        L.losa_rope_apply(rope, t(1, 1, 4, 2, 128), t(1, 1, 4, 2, 128))
    c = L.make_cache(2, 128, 32, 6, 2, 3)
    pool = lambda: (t(6, 2, 32, 128, dt=torch.float8_e4m3fn), t(6, 2, 32, 128, dt=torch.float8_e4m3fn),  # noqa: E731
                    t(6, 2, dt=torch.float32), t(6, 2, dt=torch.float32), t(2, 3, dt=torch.int32), t(2, dt=torch.int32))
    kv = t(4, 2, 128)
    with pytest.raises(ValueError, match="k, v: shapes"):
        L.losa_cache_append(c, kv, t(5, 2, 128), *pool(), 2)
    with pytest.raises(ValueError, match="indptr: holds"):
        L.losa_cache_append(c, kv, kv, *pool(), 2, indptr=t(2, dt=torch.int32))
    with pytest.raises(ValueError, match="v: expected torch.bfloat16"):
        L.losa_cache_append(c, kv, t(4, 2, 128, dt=torch.float32), *pool(), 2)
    for i, name in enumerate(("k8", "v8", "k_scale", "v_scale", "page_table", "lens")):
        p = list(pool())
        p[i] = p[i].flatten()[:-1]
        with pytest.raises(ValueError, match=f"{name}: holds"):
            L.losa_cache_append(c, kv, kv, *p, 2)
    p = list(pool())
    p[0] = t(6, 2, 32, 128, dt=torch.uint8)
    with pytest.raises(ValueError, match="k8: expected torch.float8_e4m3fn"):
        L.losa_cache_append(c, kv, kv, *p, 2)
    with pytest.raises(ValueError, match="q, o: shapes"):
        L.losa_cache_attn(c, t(3, 1, 4, 128), *pool(), 0.1, t(3, 1, 4, 128))
    with pytest.raises(ValueError, match="lse: holds"):
        L.losa_cache_attn(c, t(2, 1, 4, 128), *pool(), 0.1, t(2, 1, 4, 128), lse=t(7, dt=torch.float32))
    with pytest.raises(ValueError, match="o: holds"):
        L.losa_cache_sparse_attn(L.make_shape(4, 100, 128, 128, 128, 32, "bf16"), c, t(4, 128, 128), *pool(), 0.1,
                                 t(4, 127, 128))


def test_calls_leave_the_interpreter_to_other_threads(lib, tmp_path):
    """A launch may wait for room in its queue: other Python threads go on meanwhile, as during a ctypes call. A C function
    that takes its time stands in for the entry points; with raw pointers no argument needs a device."""
    src = tmp_path / "slow.c"
    src.write_text("#include <unistd.h>\nint slow(void) { usleep(400000); return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(tmp_path / "slow.so")], check=True)
    slow = ctypes.cast(ctypes.CDLL(str(tmp_path / "slow.so")).slow, ctypes.c_void_p).value
    mod = L._fast()
    mod.bind(slow, slow, slow, slow)
    try:
        shape, c = L.make_shape(16, 200, 256, 128, 128, 32, "bf16"), L.make_cache(2, 128, 32, 6, 2, 3)
        laps, done = [], threading.Event()

        def other():
            while not done.is_set():
                laps.append(time.perf_counter())
                time.sleep(0.001)

        t = threading.Thread(target=other)
        t.start()
        begin = time.perf_counter()
        assert L.losa_cache_sparse_attn(shape, c, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, 2 * FAKE, stream=0) == 0
        end = time.perf_counter()
        done.set()
        t.join()
        assert sum(begin + 0.05 < x < end - 0.05 for x in laps) >= 5
    finally:
        L._binding = None
        L._fast()
