"""The attention operators between the qkv projection and o_proj -- Python
binding of ``include/mxattn.h``: checks of dtypes and shapes, outputs allocated
with torch, one call of the C entry point of the same name.  The marshalling is
in C++ (``csrc/bind.cpp``), since these calls are short.

Tensors of heads are (tokens, heads, D) bf16 with a unit inner stride; the
other strides are free (multiples of 8 elements), so a slice of the packed qkv
projection is passed as it is.  A paged cache is a `KVCache`.  A call runs on
`stream` (None = the current one); what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import MxgError, lib

MAX_SEQS, MAX_NODES = 4096, 64


class Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("tok_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("layers", ctypes.c_int), ("pages", ctypes.c_int), ("page_size", ctypes.c_int)]


class AttnOpts(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("dev_status", ctypes.c_void_p),
                ("timeout_ms", ctypes.c_uint32), ("debug_stall", ctypes.c_int)]


def bind(L: ctypes.CDLL):
    """Argument types of the entry points of include/mxattn.h."""
    vp, i, f, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64
    H, C, O = ctypes.POINTER(Heads), ctypes.POINTER(CacheDesc), ctypes.POINTER(AttnOpts)
    L.qk_norm_rope.argtypes = [H, H, i, i, i, i, vp, vp, f, vp, vp, i, i, i, H, H, H, C, vp, vp, vp]
    L.qk_norm_rope.restype = i
    L.attn_prompt.argtypes = [H, H, H, vp, i, i, i, i, i, f, H, O, vp]
    L.attn_prompt.restype = i
    L.mxg_attn_tree_workspace_bytes.argtypes = [i]
    L.mxg_attn_tree_workspace_bytes.restype = ctypes.c_size_t
    L.attn_tree.argtypes = [H, H, H, vp, vp, i, i, C, vp, i, i, vp, i, i, i, f, H, O, vp]
    L.attn_tree.restype = i
    L.kv_append.argtypes = [H, i64, H, i64, vp, i, i, vp, i, i, C, vp, i, i, vp, i, i, vp, vp, vp]
    L.kv_append.restype = i


_mod = None


def _load():
    """The CPython module of the entry points.  Raises if it has not been built."""
    global _mod
    if _mod is None:
        lib()
        try:
            from . import _attn_bind
        except ImportError as e:
            raise RuntimeError(
                "_attn_bind.so is missing or does not fit this torch: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (there is no fallback)") from e
        _attn_bind.set_error(MxgError)
        _mod = _attn_bind
    return _mod


class KVCache:
    """A paged key/value cache: k and v of shape (pages, page_size, Hkv, D), or
    (layers, pages, page_size, Hkv, D), bf16, with equal strides.  It refers to
    the two tensors and owns nothing else.  kv_append takes all layers at once;
    qk_norm_rope and attn_tree take one, and refuse a cache of several."""

    __slots__ = ("k", "v")

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for t in (k, v):
            if not (t.is_cuda and t.dtype is torch.bfloat16 and t.dim() in (4, 5) and t.stride(-1) == 1):
                raise ValueError("a cache is CUDA bf16 ([layers,] pages, page_size, Hkv, D) with a unit inner stride")
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v of a cache differ in shape or strides")
        self.k, self.v = k, v

    def layer(self, i: int) -> "KVCache":
        """The cache of one layer."""
        return KVCache(self.k[i], self.v[i]) if self.k.dim() == 5 else self


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor | None = None,
                 cos_sin: torch.Tensor | None = None, *, wq=None, wk=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, v=None, cache: KVCache | None = None,
                 slots=None, dev_status=None, stream=None):
    """RMS norm (gains wq, wk (D,) bf16; None = no norm) and rotation of q
    (T, Hq, D) and k (T, Hkv, D); cos_sin (max_pos, rot) f32 with rows
    [cos | sin], pos (T,) int32.  With cache, k and v (T, Hkv, D) also go to
    the slots (T,) int64 (page * page_size + place; negative = not written) of
    this one-layer cache (cache.layer(i)).  q_out=q and k_out=k work in place.  Returns
    (q_out, k_out)."""
    ck, cv = (None, None) if cache is None else (cache.k, cache.v)
    return (_mod or _load()).qk_norm_rope(q, k, pos, cos_sin, wq, wk, eps, interleaved, q_out, k_out, v, ck, cv, slots,
                                          dev_status, stream)


def attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                scale: float | None = None, out=None, dev_status=None, timeout_ms: int = 0, debug_stall: int = 0,
                stream=None) -> torch.Tensor:
    """Causal attention of packed prompts: q (T, Hq, D), k, v (T, Hkv, D),
    sequence b = rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 (int32, on the
    device).  scale None = 1/sqrt(D).  Returns out (T, Hq, D)."""
    return (_mod or _load()).attn_prompt(q, k, v, cu_seqlens, scale, out, dev_status, timeout_ms, debug_stall, stream)


def mxg_attn_tree_workspace_bytes(D: int) -> int:
    """Workspace of attn_tree on the current device (it does not depend on the
    batch)."""
    return int(lib().mxg_attn_tree_workspace_bytes(D))


def attn_tree(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_nodes: torch.Tensor, mask: torch.Tensor,
              cache: KVCache, block_table: torch.Tensor, ctx_len: torch.Tensor, *, scale: float | None = None,
              out=None, ws=None, dev_status=None, timeout_ms: int = 0, debug_stall: int = 0,
              stream=None) -> torch.Tensor:
    """Attention of drafted trees over a paged cache: the nodes' q (N, Hq, D),
    k, v (N, Hkv, D), sequence b = nodes cu_nodes[b] .. cu_nodes[b+1] - 1 (at
    most 64), mask (N,) int64: bit j = node sees the sequence's node j; the
    cached tokens 0 .. ctx_len[b] - 1 of the pages block_table[b] (int32) are
    seen by all.  cache: one layer (cache.layer(i)).  ws None = mxg_attn_tree_workspace_bytes(D) bytes from torch's
    allocator.  Returns out (N, Hq, D)."""
    return (_mod or _load()).attn_tree(q, k, v, cu_nodes, mask, cache.k, cache.v, block_table, ctx_len, scale, out,
                                       dev_status, timeout_ms, debug_stall, ws, stream)


def kv_append(k: torch.Tensor, v: torch.Tensor, cu_nodes: torch.Tensor, accept: torch.Tensor, cache: KVCache,
              block_table: torch.Tensor, ctx_len: torch.Tensor, *, ctx_out=None, dev_status=None, stream=None):
    """The accepted nodes into the cache, in every layer: k, v (layers, N, Hkv,
    D), or (N, Hkv, D) with a one-layer cache; accept (B, most) int32: the
    nodes, counted from the sequence's first, that become tokens ctx_len[b],
    ctx_len[b] + 1, ... (the first negative entry ends the list, and so does
    one that cannot be written: no such node, or no page for the token).
    Returns ctx_out (B,) = ctx_len + tokens written."""
    return (_mod or _load()).kv_append(k, v, cu_nodes, accept, cache.k, cache.v, block_table, ctx_len, ctx_out,
                                       dev_status, stream)
