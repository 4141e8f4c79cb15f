"""Device-buffer harness around the C ABI: allocates the caller-owned buffers of one attention layer (LayerBuffers) and of
a layer's paged 8-bit key/value cache (KvCache) with PyTorch (device memory and streams only) and calls the entry points
in order. No computation happens here; every step runs in the library's kernels."""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import numpy as np
import torch

from . import (DTYPE_BF16, DTYPE_F32, losa_cache_append, losa_cache_attn, losa_cache_attn_workspace_bytes,
               losa_cache_sparse_attn, losa_dense_profile, losa_dense_profile_workspace_bytes, losa_dense_profile_ws,
               losa_rope_apply, losa_select, losa_select_topk, losa_select_workspace_bytes, losa_sparse_attn, make_cache,
               make_shape)


def host_tokens_to_device(a: np.ndarray, dtype: str, device="cuda") -> torch.Tensor:
    """[H][Np][d] host tokens (fp32 values, or uint16 bf16 bit patterns) -> contiguous device tensor."""
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t.to(device)


def device_tokens_to_f32(t: torch.Tensor) -> np.ndarray:
    return t.float().cpu().numpy()


def _on_stream(stream):
    """Allocations and copies inside belong to a call on `stream` (None: the current one; an int: a raw handle)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _capturing(t):
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


@dataclass
class LayerBuffers:
    heads: int
    n_tokens: int
    n_padded: int
    head_dim: int
    block: int
    dtype: str
    device: str = "cuda"
    block_k: int = 0  # key block size when it differs from the query block size

    def __post_init__(self):
        bk = self.block_k or self.block
        self.shape = make_shape(self.heads, self.n_tokens, self.n_padded, self.head_dim, self.block, bk, self.dtype)
        self.nq = self.n_padded // self.block
        self.nk = self.n_padded // bk
        self.rows = self.heads * self.nq
        tdt = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        dev = self.device
        self.o = torch.empty((self.heads, self.n_padded, self.head_dim), dtype=tdt, device=dev)
        self.lse = torch.empty((self.heads, self.n_padded), dtype=torch.float32, device=dev)
        self.mass = torch.empty((self.heads, self.nq, self.nk), dtype=torch.float32, device=dev)
        self.indptr = torch.empty(self.rows + 1, dtype=torch.int32, device=dev)
        self.kv_idx = torch.empty(self.rows * self.nk, dtype=torch.int32, device=dev)
        self.order = torch.empty(self.rows, dtype=torch.int32, device=dev)
        ws = losa_select_workspace_bytes(self.shape)
        self.workspace = torch.empty((ws + 15) // 16 * 16, dtype=torch.uint8, device=dev)
        pws = losa_dense_profile_workspace_bytes(self.shape)  # 0 on the fp32 path
        self.profile_workspace = torch.empty(max(16, (pws + 15) // 16 * 16), dtype=torch.uint8, device=dev)

    @classmethod
    def for_config(cls, cfg, device="cuda"):
        return cls(cfg.heads, cfg.n_tokens, cfg.n_padded, cfg.head_dim, cfg.block, cfg.dtype, device,
                   getattr(cfg, "block_k", 0))

    def profile(self, q, k, v, scale, with_mass=True, stream=None, one_pass=True):
        """The dense step; with_mass adds the block masses, in the forward pass (one_pass, the default) or in a
        second pass that needs no workspace."""
        if with_mass and one_pass:
            losa_dense_profile_ws(self.shape, q, k, v, scale, self.o, self.lse, self.mass, self.profile_workspace,
                                  stream=stream)
        else:
            losa_dense_profile(self.shape, q, k, v, scale, self.o, self.lse, self.mass if with_mass else None,
                               stream=stream)

    def select(self, tau, mass=None, stream=None):
        losa_select(self.shape, self.mass if mass is None else mass, tau, self.indptr, self.kv_idx, self.order,
                    self.workspace, stream=stream)

    def select_topk(self, k_blocks, mass=None, stream=None):
        losa_select_topk(self.shape, self.mass if mass is None else mass, k_blocks, self.indptr, self.kv_idx,
                         self.order, self.workspace, stream=stream)

    def sparse(self, q, k, v, scale, out=None, lse=None, stream=None, order=True):
        losa_sparse_attn(self.shape, q, k, v, scale, self.indptr, self.kv_idx, self.order if order else None,
                         self.o if out is None else out, lse, stream=stream)

    def pack_qkv(self, qkv, rope, out=None, positions=None, start=None, stream=None):
        """A fused projection's output (batch, N, 3, heads / batch, d), any strides but a contiguous last dimension, as the
        calls' q, k, v: query and key rotated, head-major, padding rows zero. Returns views of one (3, H, Np, d) buffer,
        which belongs to the call's stream if it is made here."""
        batch, n, _, heads, d = qkv.shape
        if out is None:
            with _on_stream(stream):
                out = torch.empty((3, self.heads, self.n_padded, self.head_dim), dtype=qkv.dtype, device=qkv.device)
        y = out.view(3, batch, heads, self.n_padded, d).permute(0, 1, 3, 2, 4)
        losa_rope_apply(rope, qkv.permute(2, 0, 1, 3, 4), y, rotate=0b011, positions=positions, start=start, stream=stream)
        return out[0], out[1], out[2]

    def unpack_o(self, rope, out, o=None, stream=None):
        """The head-major output's real rows into out (batch, N, heads / batch, d), for the output projection."""
        batch, n, heads, d = out.shape
        o = (self.o if o is None else o).view(1, batch, heads, self.n_padded, d).permute(0, 1, 3, 2, 4)[:, :, :n]
        losa_rope_apply(rope, o, out[None], rotate=0, stream=stream)
        return out

    def csr_host(self):
        indptr = self.indptr.cpu().numpy()
        nnz = int(indptr[-1])
        return indptr, self.kv_idx[:nnz].cpu().numpy(), self.order.cpu().numpy()


class KvCache:
    """A layer's paged 8-bit cache for `seqs` sequences of up to `capacity` tokens: its pool, page table (each sequence's
    pages in order) and lengths, which live on the device. An eager append leaves the lengths before it where they were and
    flips to another buffer; once a call or a reading of `lens` is captured into a graph, `lens` stays one tensor that every
    append advances, eager or replayed, so that both go on from each other. max_len bounds the lengths on the host; as replays
    are not seen there, it is the capacity from the first captured append on."""

    def __init__(self, seqs, kv_heads, head_dim, capacity, page_tokens=128, rope=None, device="cuda"):
        self.seqs, self.page_tokens, self.rope = seqs, page_tokens, rope
        width = -(-capacity // page_tokens)
        self.cache = make_cache(kv_heads, head_dim, page_tokens, seqs * width, seqs, width)
        pool = (seqs * width, kv_heads, page_tokens, head_dim)
        self.k8 = torch.zeros(pool, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.v8 = torch.zeros(pool, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.k_scale = torch.ones(pool[:2], dtype=torch.float32, device=device)
        self.v_scale = torch.ones(pool[:2], dtype=torch.float32, device=device)
        self.page_table = torch.arange(seqs * width, dtype=torch.int32, device=device).view(seqs, width)
        self._lens = torch.zeros((2, seqs), dtype=torch.int32, device=device)
        self._now = 0
        self._fixed = self._replayed = False  # a graph holds the lengths' address; a graph may append
        self.max_len = 0

    @property
    def lens(self):
        self._fixed |= _capturing(self._lens)
        return self._lens[self._now]

    @property
    def buffers(self):
        return self.k8, self.v8, self.k_scale, self.v_scale, self.page_table

    def append(self, k, v, new_tokens, indptr=None, positions=None, stream=None):
        """k, v: (tokens, kv_heads, d) of all sequences; new_tokens of each, or at most that many with indptr."""
        nxt = 1 - self._now
        with _on_stream(stream):
            lens = self.lens
            losa_cache_append(self.cache, k, v, *self.buffers, lens, new_tokens, indptr=indptr, new_lens=self._lens[nxt],
                              rope=self.rope, positions=positions, stream=stream)
            self._replayed |= _capturing(self._lens)
            if self._fixed:
                lens.copy_(self._lens[nxt])
            else:
                self._now = nxt
        capacity = self.cache.table_stride * self.page_tokens
        self.max_len = capacity if self._replayed else min(self.max_len + int(new_tokens), capacity)

    def attend(self, q, scale, o, lse=None, causal=True, stream=None):
        """The last tokens q (seqs, tokens, heads, d), appended before, over the whole cache. The workspace comes from the
        allocator on the call's stream every time: calls on several streams, and captured ones, each have their own."""
        need = losa_cache_attn_workspace_bytes(self.cache, q.shape[2], q.shape[1], self.max_len)
        with _on_stream(stream):
            lens = self.lens
            workspace = torch.empty(need, dtype=torch.uint8, device=self.k8.device) if need else None
        losa_cache_attn(self.cache, q, *self.buffers, lens, scale, o, lse=lse, causal=causal, max_len=self.max_len,
                        workspace=workspace, stream=stream)

    def sparse(self, layer, q, scale, out, lse=None, lists=True, order=True, stream=None):
        """Query blocks of a layer (LayerBuffers with block_k = page_tokens) over its frozen lists, or over every block."""
        with _on_stream(stream):
            lens = self.lens
        losa_cache_sparse_attn(layer.shape, self.cache, q, *self.buffers, lens, scale, out,
                               indptr=layer.indptr if lists else None, kv_block_idx=layer.kv_idx if lists else None,
                               order=layer.order if lists and order else None, lse=lse, stream=stream)
