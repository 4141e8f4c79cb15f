"""Python binding of the LoSA C ABI (include/losa.h): argument marshalling only.

Every function has the name of its C entry point, takes torch CUDA tensors (or raw device pointers as ints)
and passes their pointers, sizes and the current CUDA stream to the library. All computation happens in the
library's CUDA kernels; there is no fallback. Importing this module does not load the library; the first call
does, and raises if liblosa.so is missing (build it with `python -m free_block_sparse_losa_b200.build`). The streaming
calls go through a compiled binding (_binding.so, same build): their checks and marshalling are the same, in C++.
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["LosaShape", "LosaError", "make_shape", "losa_dense_profile", "losa_select", "losa_select_noalloc",
           "losa_select_topk", "losa_sparse_attn",
           "losa_select_workspace_bytes", "losa_get_device_error", "losa_selftest_wait_timeout",
           "losa_set_wait_limit_ns", "losa_status_string", "losa_version", "library_path", "load",
           "LosaRope", "LosaCache", "LosaTokenView", "make_rope", "make_cache", "losa_rope_apply", "losa_cache_append",
           "losa_cache_attn", "losa_cache_attn_workspace_bytes", "losa_cache_sparse_attn",
           "DTYPE_F32", "DTYPE_BF16", "STATUS"]

DTYPE_F32 = 0
DTYPE_BF16 = 1
STATUS = {0: "LOSA_OK", -1: "LOSA_ERR_INVALID_ARG", -2: "LOSA_ERR_UNSUPPORTED", -3: "LOSA_ERR_CAPACITY",
          -4: "LOSA_ERR_CUDA", -5: "LOSA_ERR_DEVICE_FAULT", -6: "LOSA_ERR_TIMEOUT"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


class LosaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


class LosaShape(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("n_padded", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_q", ctypes.c_int32), ("block_k", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class LosaRope(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("axis_dims", ctypes.c_int32 * 3), ("grid_y", ctypes.c_int32),
                ("grid_x", ctypes.c_int32), ("offset", ctypes.c_int32 * 3), ("pairing", ctypes.c_int32),
                ("theta", ctypes.c_double)]


class LosaCache(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("seqs", ctypes.c_int32), ("table_stride", ctypes.c_int32)]


class LosaTokenView(ctypes.Structure):
    _fields_ = [("parts", ctypes.c_int32), ("batch", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("part_stride", ctypes.c_int64), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def make_rope(head_dim, axis_dims, grid, offset=(0, 0, 0), theta=10000.0, halves=False) -> LosaRope:
    """Rotary positions with three axes: rotated dimensions per axis (t, y, x) and the token grid's (y, x) extents."""
    return LosaRope(head_dim, (ctypes.c_int32 * 3)(*axis_dims), grid[0], grid[1], (ctypes.c_int32 * 3)(*offset),
                    1 if halves else 0, theta)


def make_cache(kv_heads, head_dim, page_tokens, n_pages, seqs, table_stride) -> LosaCache:
    return LosaCache(kv_heads, head_dim, page_tokens, n_pages, seqs, table_stride)


def make_shape(heads, n_tokens, n_padded, head_dim, block_q, block_k, dtype) -> LosaShape:
    if isinstance(dtype, str):
        dtype = {"f32": DTYPE_F32, "bf16": DTYPE_BF16}[dtype]
    return LosaShape(heads, n_tokens, n_padded, head_dim, block_q, block_k, dtype)


def library_path() -> str:
    return os.environ.get("LOSA_LIBRARY", os.path.join(_HERE, "liblosa.so"))


def load():
    """Load liblosa.so (once). Raises if it is missing: there is no other implementation."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing")
    L = ctypes.CDLL(path)
    vp, i32, f32, f64, i64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_double,
                                  ctypes.c_int64, ctypes.c_size_t)
    sp = ctypes.POINTER(LosaShape)
    L.losa_dense_profile.argtypes = [sp, vp, vp, vp, f32, vp, vp, vp, vp]
    L.losa_dense_profile_ws.argtypes = [sp, vp, vp, vp, f32, vp, vp, vp, vp, sz, vp]
    L.losa_dense_profile_workspace_bytes.argtypes = [sp]
    L.losa_dense_profile_workspace_bytes.restype = sz
    L.losa_select.argtypes = [sp, vp, f64, vp, vp, i64, vp, vp, sz, vp]
    L.losa_select_noalloc.argtypes = [sp, vp, f64, vp, vp, i64, vp, vp]
    L.losa_select_topk.argtypes = [sp, vp, i32, vp, vp, i64, vp, vp, sz, vp]
    L.losa_select_workspace_bytes.argtypes = [sp]
    L.losa_select_workspace_bytes.restype = sz
    L.losa_sparse_attn.argtypes = [sp, vp, vp, vp, f32, vp, vp, vp, vp, vp, vp]
    rp, cp = ctypes.POINTER(LosaRope), ctypes.POINTER(LosaCache)
    tp = ctypes.POINTER(LosaTokenView)
    L.losa_rope_apply.argtypes = [rp, i32, tp, vp, tp, vp, ctypes.c_uint32, i32, vp, vp, vp]
    L.losa_cache_append.argtypes = [cp, rp, i32, vp, i64, i64, vp, i64, i64, i64, i32] + [vp] * 10
    L.losa_cache_attn.argtypes = ([cp, i32, i32, i32, vp, i64, i64, i64] + [vp] * 6 + [f32, i32, vp, i64, i64, i64] +
                                  [vp, vp, sz, vp])
    L.losa_cache_attn_workspace_bytes.argtypes = [cp, i32, i32, i32]
    L.losa_cache_attn_workspace_bytes.restype = sz
    L.losa_cache_sparse_attn.argtypes = [sp, cp] + [vp] * 7 + [f32] + [vp] * 6
    L.losa_get_device_error.argtypes = [vp]
    L.losa_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
    L.losa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.losa_set_wait_limit_ns.restype = None
    L.losa_status_string.argtypes = [i32]
    L.losa_status_string.restype = ctypes.c_char_p
    L.losa_version.restype = ctypes.c_int
    for name in ("losa_dense_profile", "losa_dense_profile_ws", "losa_select", "losa_select_noalloc", "losa_select_topk",
                 "losa_sparse_attn", "losa_rope_apply", "losa_cache_append", "losa_cache_attn",
                 "losa_cache_sparse_attn",
                 "losa_get_device_error",
                 "losa_selftest_wait_timeout"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def _dims(shape):
    """(H, Np, d, nq, nk) of a shape; 0 for a block count whose block size is not positive."""
    nq = shape.n_padded // shape.block_q if shape.block_q > 0 else 0
    nk = shape.n_padded // shape.block_k if shape.block_k > 0 else 0
    return max(shape.heads, 0), max(shape.n_padded, 0), max(shape.head_dim, 0), max(nq, 0), max(nk, 0)


def _token_dtype(shape):
    return {DTYPE_F32: "float32", DTYPE_BF16: "bfloat16"}.get(shape.dtype)


_torch_module = None
_dtypes = {}


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _dtypes.update({n: getattr(torch, n) for n in ("float32", "bfloat16", "int32")})
        _torch_module = torch
    return _torch_module


def _ptrs(*specs):
    """Device pointers of arguments given as (value, name, dtype, numel). None stays NULL and an int is taken as a raw
    device pointer (the caller vouches for its size). A tensor must have the expected dtype (if given), hold at least
    `numel` elements (if given), be contiguous and live on the current CUDA device, so that a wrong buffer is refused
    here instead of being read or written out of bounds on the GPU. The dtype, size and layout of every argument are
    checked before any argument's device. Raw pointers alone need no torch."""
    out, where = [], []
    torch = None
    for t, name, dtype, numel in specs:
        if t is None or isinstance(t, int):
            out.append(t)
            continue
        torch = torch or _torch()
        if dtype is not None and t.dtype is not _dtypes[dtype]:
            raise ValueError(f"{name}: expected torch.{dtype}, got {t.dtype}")
        if numel is not None and t.numel() < numel:
            raise ValueError(f"{name}: holds {t.numel()} elements, the shape needs {numel}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
        where.append(t.get_device())  # -1 on the host
        out.append(t.data_ptr())
    if where and min(where) < 0:
        name = next(s[1] for s in specs if s[0] is not None and not isinstance(s[0], int) and s[0].get_device() < 0)
        raise ValueError(f"{name}: expected a CUDA tensor")
    if where:
        here = torch._C._cuda_getDevice()
        if where.count(here) != len(where):
            t, name = next(s[:2] for s in specs
                           if s[0] is not None and not isinstance(s[0], int) and s[0].get_device() != here)
            raise ValueError(f"{name}: lives on {t.device}, the current device is cuda:{here}")
    return out


def _stream(stream):
    if stream is None:
        c = _torch()._C
        return c._cuda_getCurrentRawStream(c._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str, raise_on_error: bool):
    if status != 0 and raise_on_error:
        raise LosaError(status, where)
    return status


def losa_dense_profile(shape, q, k, v, scale, o, lse=None, mass=None, stream=None, raise_on_error=True):
    H, Np, d, nq, nk = _dims(shape)
    tdt = _token_dtype(shape)
    pq, pk, pv, po, pl, pm = _ptrs((q, "q", tdt, H * Np * d), (k, "k", tdt, H * Np * d), (v, "v", tdt, H * Np * d),
                                   (o, "o", tdt, H * Np * d), (lse, "lse", "float32", H * Np),
                                   (mass, "mass", "float32", H * nq * nk))
    st = load().losa_dense_profile(ctypes.byref(shape), pq, pk, pv, float(scale), po, pl, pm, _stream(stream))
    return _check(st, "losa_dense_profile", raise_on_error)


def losa_dense_profile_workspace_bytes(shape) -> int:
    return int(load().losa_dense_profile_workspace_bytes(ctypes.byref(shape)))


def losa_dense_profile_ws(shape, q, k, v, scale, o, lse, mass, workspace, ws_bytes=None, stream=None,
                          raise_on_error=True):
    """losa_dense_profile with the masses taken in the forward pass (needs a workspace of
    losa_dense_profile_workspace_bytes(shape) bytes)."""
    H, Np, d, nq, nk = _dims(shape)
    tdt = _token_dtype(shape)
    if isinstance(workspace, int):
        if ws_bytes is None:
            raise ValueError("workspace: a raw pointer needs ws_bytes")
        wsb = int(ws_bytes)
    else:
        have = workspace.numel() * workspace.element_size()
        wsb = have if ws_bytes is None else int(ws_bytes)
        if have < wsb:
            raise ValueError(f"workspace: holds {have} bytes, ws_bytes says {wsb}")
    pq, pk, pv, po, pl, pm, pw = _ptrs((q, "q", tdt, H * Np * d), (k, "k", tdt, H * Np * d),
                                       (v, "v", tdt, H * Np * d), (o, "o", tdt, H * Np * d),
                                       (lse, "lse", "float32", H * Np), (mass, "mass", "float32", H * nq * nk),
                                       (workspace, "workspace", None, None))
    st = load().losa_dense_profile_ws(ctypes.byref(shape), pq, pk, pv, float(scale), po, pl, pm, pw, wsb,
                                      _stream(stream))
    return _check(st, "losa_dense_profile_ws", raise_on_error)


def losa_select_workspace_bytes(shape) -> int:
    return int(load().losa_select_workspace_bytes(ctypes.byref(shape)))


def _select_args(shape, mass, indptr, kv_block_idx, order, idx_capacity, workspace=None, ws_bytes=None):
    """Pointers of the selection calls' arguments, the index capacity and the workspace size."""
    H, _, _, nq, nk = _dims(shape)
    if idx_capacity is None:
        if isinstance(kv_block_idx, int):
            raise ValueError("kv_block_idx: a raw pointer needs idx_capacity")
        cap, idx_numel = kv_block_idx.numel(), None
    else:
        cap = idx_numel = int(idx_capacity)
    wsb = None
    if workspace is not None:
        if isinstance(workspace, int):
            if ws_bytes is None:
                raise ValueError("workspace: a raw pointer needs ws_bytes")
            wsb = int(ws_bytes)
        else:
            have = workspace.numel() * workspace.element_size()
            wsb = have if ws_bytes is None else int(ws_bytes)
            if have < wsb:
                raise ValueError(f"workspace: holds {have} bytes, ws_bytes says {wsb}")
    ptrs = _ptrs((mass, "mass", "float32", H * nq * nk), (indptr, "indptr", "int32", H * nq + 1),
                 (kv_block_idx, "kv_block_idx", "int32", idx_numel), (order, "order", "int32", H * nq),
                 (workspace, "workspace", None, None))
    return ptrs, cap, wsb


def losa_select(shape, mass, tau, indptr, kv_block_idx, order, workspace, idx_capacity=None, ws_bytes=None,
                stream=None, raise_on_error=True):
    (pm, pi, pk, po, pw), cap, wsb = _select_args(shape, mass, indptr, kv_block_idx, order, idx_capacity, workspace,
                                                  ws_bytes)
    st = load().losa_select(ctypes.byref(shape), pm, float(tau), pi, pk, cap, po, pw, wsb, _stream(stream))
    return _check(st, "losa_select", raise_on_error)


def losa_select_topk(shape, mass, k_blocks, indptr, kv_block_idx, order, workspace, idx_capacity=None, ws_bytes=None,
                     stream=None, raise_on_error=True):
    (pm, pi, pk, po, pw), cap, wsb = _select_args(shape, mass, indptr, kv_block_idx, order, idx_capacity, workspace,
                                                  ws_bytes)
    st = load().losa_select_topk(ctypes.byref(shape), pm, int(k_blocks), pi, pk, cap, po, pw, wsb, _stream(stream))
    return _check(st, "losa_select_topk", raise_on_error)


def losa_select_noalloc(shape, mass, tau, indptr, kv_block_idx, order, idx_capacity=None, stream=None,
                        raise_on_error=True):
    """losa_select with the library's fixed device scratch instead of a caller workspace (see include/losa.h)."""
    (pm, pi, pk, po, _), cap, _ = _select_args(shape, mass, indptr, kv_block_idx, order, idx_capacity)
    st = load().losa_select_noalloc(ctypes.byref(shape), pm, float(tau), pi, pk, cap, po, _stream(stream))
    return _check(st, "losa_select_noalloc", raise_on_error)


def losa_sparse_attn(shape, q, k, v, scale, indptr, kv_block_idx, order, o, lse=None, stream=None,
                     raise_on_error=True):
    H, Np, d, nq, _ = _dims(shape)
    tdt = _token_dtype(shape)
    pq, pk, pv, pi, px, po, pout, pl = _ptrs(
        (q, "q", tdt, H * Np * d), (k, "k", tdt, H * Np * d), (v, "v", tdt, H * Np * d),
        (indptr, "indptr", "int32", H * nq + 1), (kv_block_idx, "kv_block_idx", "int32", None),
        (order, "order", "int32", H * nq), (o, "o", tdt, H * Np * d), (lse, "lse", "float32", H * Np))
    st = load().losa_sparse_attn(ctypes.byref(shape), pq, pk, pv, float(scale), pi, px, po, pout, pl,
                                 _stream(stream))
    return _check(st, "losa_sparse_attn", raise_on_error)


_binding = None


def _fast():
    """The streaming calls' argument marshalling (csrc/binding.cpp), bound to the loaded library."""
    global _binding
    if _binding is None:
        import importlib
        lib = load()
        _torch()
        try:
            mod = importlib.import_module("._binding", __name__)
        except ImportError as e:
            raise RuntimeError(f"binding not built: {e} (python -m free_block_sparse_losa_b200.build)") from e
        mod.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                   for f in ("losa_rope_apply", "losa_cache_append", "losa_cache_attn", "losa_cache_sparse_attn")))
        _binding = mod
    return _binding


def losa_rope_apply(rope, x, y, rotate=1, inverse=False, positions=None, start=None, stream=None, raise_on_error=True):
    """x, y: (parts, batch, tokens, heads, head_dim) views of any layouts (last dimension contiguous); y may hold more
    tokens, which become zero rows. `rotate` is a bit mask of the parts that are rotated."""
    st = (_binding or _fast()).rope_apply(rope, x, y, rotate, inverse, positions, start, stream)
    return st if st == 0 else _check(st, "losa_rope_apply", raise_on_error)


def losa_cache_append(cache, k, v, k8, v8, k_scale, v_scale, page_table, lens, new_tokens, indptr=None, new_lens=None,
                      rope=None, positions=None, stream=None, raise_on_error=True):
    """k, v: (tokens, kv_heads, head_dim) of all sequences' new tokens, strided alike or not."""
    st = (_binding or _fast()).cache_append(cache, k, v, k8, v8, k_scale, v_scale, page_table, lens, new_tokens, indptr,
                                            new_lens, rope, positions, stream)
    return st if st == 0 else _check(st, "losa_cache_append", raise_on_error)


def losa_cache_attn_workspace_bytes(cache, heads, tokens, max_len=0) -> int:
    return int(load().losa_cache_attn_workspace_bytes(ctypes.byref(cache), int(heads), int(tokens), int(max_len)))


def losa_cache_attn(cache, q, k8, v8, k_scale, v_scale, page_table, lens, scale, o, lse=None, causal=True, max_len=0,
                    workspace=None, stream=None, raise_on_error=True, ws_bytes=None):
    """q, o: (seqs, tokens, heads, head_dim) bf16, any strides but a contiguous last dimension; lse: (seqs, tokens,
    heads). max_len bounds the lengths (0: the page table's capacity). ws_bytes: the workspace's size, where it is a raw pointer
    (0 otherwise: enough for a call that needs none) or less than the tensor."""
    st = (_binding or _fast()).cache_attn(cache, q, k8, v8, k_scale, v_scale, page_table, lens, scale, o, lse, causal,
                                          max_len, workspace, ws_bytes, stream)
    return st if st == 0 else _check(st, "losa_cache_attn", raise_on_error)


def losa_cache_sparse_attn(shape, cache, q, k8, v8, k_scale, v_scale, page_table, lens, scale, o, indptr=None,
                           kv_block_idx=None, order=None, lse=None, stream=None, raise_on_error=True):
    """losa_sparse_attn over the paged 8-bit cache; without lists every block of the sequence is attended to."""
    st = (_binding or _fast()).cache_sparse_attn(shape, cache, q, k8, v8, k_scale, v_scale, page_table, lens, scale, o,
                                                 indptr, kv_block_idx, order, lse, stream)
    return st if st == 0 else _check(st, "losa_cache_sparse_attn", raise_on_error)


def losa_get_device_error(stream=None) -> int:
    return int(load().losa_get_device_error(_stream(stream)))


def losa_selftest_wait_timeout(limit_ns: int, stream=None, raise_on_error=True):
    st = load().losa_selftest_wait_timeout(int(limit_ns), _stream(stream))
    return _check(st, "losa_selftest_wait_timeout", raise_on_error)


def losa_set_wait_limit_ns(limit_ns: int):
    load().losa_set_wait_limit_ns(int(limit_ns))


def losa_status_string(status: int) -> str:
    return load().losa_status_string(int(status)).decode()


def losa_version() -> int:
    return int(load().losa_version())
