"""CPU checks of the streaming calls at the ends of what their documentation allows. No call here reaches the CUDA runtime."""
import ctypes
import os
import subprocess
import sys

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


def test_append_strides_of_single_extents(lib):
    """Nothing steps by the stride of an extent of one: such a call is refused for its head_dim only, which comes later."""
    def call(hk, total, strides):
        cache = L.make_cache(hk, 96, 128, 10, 1, 5)
        return lib.losa_cache_append(ctypes.byref(cache), None, 1, FAKE, strides[0], strides[1], FAKE, strides[2], strides[3],
                                     total, 1, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 0)

    assert call(1, 8, (96, 5, 96, -3)) == UNSUPPORTED
    assert call(4, 1, (7, 96, 1, 96)) == UNSUPPORTED
    for hk, total, strides in ((1, 8, (95, 8, 96, 8)), (4, 1, (8, 96, 8, 95)), (4, 1, (8, -96, 8, 96))):
        assert call(hk, total, strides) == INVALID


def test_lengths_of_captured_and_eager_appends(monkeypatch):
    """KvCache's lengths without a GPU: a fake append that runs at once stands in for the call, a flag for the capture. A step
    kept and run again goes on from the lengths the last append left, whichever kind it was."""
    from free_block_sparse_losa_b200 import harness
    capturing, kept = [False], []

    def fake(cache, k, v, k8, v8, ks, vs, table, lens, new, indptr=None, new_lens=None, **kw):
        def step():
            new_lens.copy_(lens + new)
        kept.append(step)
        if not capturing[0]:
            step()

    monkeypatch.setattr(harness, "losa_cache_append", fake)
    monkeypatch.setattr(harness, "_capturing", lambda t: capturing[0], raising=False)
    cache = harness.KvCache(2, 1, 64, 96, page_tokens=32, device="cpu")
    cache.append(None, None, 5)
    before = cache.lens
    cache.append(None, None, 2)
    assert before.tolist() == [5, 5] and cache.lens.tolist() == [7, 7] and cache.max_len == 7
    held = cache.lens
    capturing[0] = True
    real_copy, copies = torch.Tensor.copy_, []
    monkeypatch.setattr(torch.Tensor, "copy_", lambda a, b: copies.append((a, b)))
    cache.append(None, None, 1)
    monkeypatch.setattr(torch.Tensor, "copy_", real_copy)
    capturing[0] = False
    graph = [kept[-1]] + [lambda a=a, b=b: a.copy_(b) for a, b in copies]
    assert cache.lens.tolist() == [7, 7] and cache.max_len == 96
    n = 7
    for kind in "rrerer":
        if kind == "e":
            cache.append(None, None, 3)
            n += 3
        else:
            for step in graph:
                step()
            n += 1
        assert cache.lens.tolist() == held.tolist() == [n, n]
    assert cache.max_len == 96


def test_raw_pointers_need_no_torch(lib):
    """Device pointers as ints and a stream handle: the calls that go through ctypes work where torch cannot be imported."""
    code = """
import sys
sys.modules["torch"] = None
import free_block_sparse_losa_b200 as L
p = 0x10000
s = L.make_shape(2, 300, 256, 128, 128, 128, "bf16")  # more tokens than rows: refused before anything is launched
kw = dict(stream=0, raise_on_error=False)
assert L.losa_sparse_attn(s, p, p, p, 0.1, p, p, p, 2 * p, **kw) == -1
assert L.losa_dense_profile(s, p, p, p, 0.1, 2 * p, **kw) == -1
assert L.losa_dense_profile_ws(s, p, p, p, 0.1, 2 * p, p, p, p, ws_bytes=16, **kw) == -1
assert L.losa_select(s, p, 0.9, p, p, p, p, idx_capacity=8, ws_bytes=16, **kw) == -1
assert L.losa_select_topk(s, p, 1, p, p, p, p, idx_capacity=8, ws_bytes=16, **kw) == -1
assert L.losa_select_noalloc(s, p, 0.9, p, p, p, idx_capacity=8, **kw) == -1
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_workspace_bytes(lib):
    """A raw workspace comes with its size, as for the other calls; a tensor's size is its own unless less is said."""
    c = L.make_cache(2, 128, 32, 6, 2, 3)
    t = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt)  # noqa: E731
    q, o = t(2, 1, 4, 128), t(2, 1, 4, 128)

    def call(**kw):
        return L.losa_cache_attn(c, q, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, o, stream=0, raise_on_error=False, **kw)

    with pytest.raises(ValueError, match="workspace: holds 64 bytes, ws_bytes says 65"):
        call(workspace=t(64, dt=torch.uint8), ws_bytes=65)
    with pytest.raises(ValueError, match="ws_bytes: out of range"):
        call(workspace=FAKE, ws_bytes=-1)
    for kw in (dict(workspace=FAKE), dict(workspace=FAKE, ws_bytes=64), dict(workspace=t(64, dt=torch.uint8), ws_bytes=64), dict(ws_bytes=0), {}):
        with pytest.raises(ValueError, match="q: expected a CUDA tensor"):  # the last check: these got past the sizes
            call(**kw)


def test_packed_projection_is_allocated_on_the_calls_stream(lib, monkeypatch):
    """pack_qkv's own buffer belongs to the stream that fills it: memory that the current stream still uses must not be
    handed to a call on another one."""
    from free_block_sparse_losa_b200 import harness
    inside, seen = [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *a):
            inside.pop()

    real = torch.empty
    layer = harness.LayerBuffers(4, 100, 128, 64, 128, "f32", device="cpu")
    monkeypatch.setattr(harness, "_on_stream", On)
    monkeypatch.setattr(harness, "losa_rope_apply", lambda *a, **kw: seen.append(("call", kw["stream"])))
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: seen.append(("alloc", list(inside))) or real(*a, **kw))
    for stream in (None, 77, "side"):
        layer.pack_qkv(torch.zeros(2, 100, 3, 2, 64), None, stream=stream)
        assert seen == [("alloc", [stream]), ("call", stream)]
        seen.clear()


def test_lengths_read_by_a_captured_call(monkeypatch):
    """A graph that only reads the lengths (an attention, a rotation that starts at them) reads them in one place: eager
    appends behind the capture advance that tensor."""
    from free_block_sparse_losa_b200 import harness
    capturing, read = [False], []
    monkeypatch.setattr(harness, "_capturing", lambda t: capturing[0], raising=False)
    monkeypatch.setattr(harness, "losa_cache_append",
                        lambda c, k, v, k8, v8, ks, vs, table, lens, new, new_lens=None, **kw: new_lens.copy_(lens + new))
    monkeypatch.setattr(harness, "losa_cache_attn", lambda c, q, k8, v8, ks, vs, table, lens, *a, **kw: read.append(lens))
    monkeypatch.setattr(harness, "losa_cache_sparse_attn", lambda s, c, q, k8, v8, ks, vs, table, lens, *a, **kw: read.append(lens))
    q = torch.zeros(2, 1, 1, 64)
    layer = type("Layer", (), dict(shape=None, indptr=None, kv_idx=None, order=None))
    for use in (lambda c: c.attend(q, 0.1, q), lambda c: c.sparse(layer, q, 0.1, q), lambda c: read.append(c.lens)):
        cache = harness.KvCache(2, 1, 64, 96, page_tokens=32, device="cpu")
        cache.append(None, None, 5)
        capturing[0] = True
        use(cache)
        capturing[0] = False
        for n in (8, 11, 14):
            cache.append(None, None, 3)
            assert read[-1].tolist() == cache.lens.tolist() == [n, n] and cache.max_len == n
