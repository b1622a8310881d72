"""The attention operators between the qkv projection and o_proj -- Python
binding of ``include/mxattn.h``, in the manner of the package's other entry
points: checks of dtypes and shapes, outputs allocated with torch, one call of
the C entry point of the same name.

Tensors of heads are (tokens, heads, D) bf16 with a unit inner stride; the
other strides are free (multiples of 8 elements), so a slice of the packed qkv
projection is passed as it is.  A paged cache is a `KVCache`, made once from
its two tensors.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, _need, _ptr, _stream, lib, workspace

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


def _heads(t: torch.Tensor, name: str):
    _need(t.dtype is torch.bfloat16 and t.is_cuda and t.dim() == 3, f"{name} must be a CUDA bf16 (tokens, heads, D) tensor")
    a, b, c = t.stride()
    _need(c == 1, f"{name} must have a unit inner stride")
    return Heads(t.data_ptr(), a, b)


def _ints(t: torch.Tensor, name: str, dim: int = 1, dtype=torch.int32):
    _need(t.dtype is dtype and t.is_cuda and t.dim() == dim and (t.numel() == 0 or t.stride(-1) == 1),
          f"{name} must be a CUDA {dtype} tensor of {dim} dimension(s) with a unit inner stride")
    return t.data_ptr()


def _table(t: torch.Tensor, seqs: int, name: str):
    p = _ints(t, name, 2)
    _need(t.shape[0] == seqs, f"{name} must have a row for each sequence")
    return p, (t.stride(0) if t.shape[0] > 1 else t.shape[1]), t.shape[1]


class KVCache:
    """A paged key/value cache: k and v of shape (pages, page_size, Hkv, D), or
    (layers, pages, page_size, Hkv, D), bf16, with equal strides.  It refers to
    the two tensors and owns nothing else; make it once and pass it on."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for t in (k, v):
            _need(t.is_cuda and t.dtype is torch.bfloat16 and t.dim() in (4, 5) and t.stride(-1) == 1,
                  "a cache is CUDA bf16 ([layers,] pages, page_size, Hkv, D) with a unit inner stride")
        _need(k.shape == v.shape and k.stride() == v.stride(), "k and v of a cache differ in shape or strides")
        self.k, self.v = k, v
        self.layers = k.shape[0] if k.dim() == 5 else 1
        self.pages, self.page_size, self.hkv, self.d = k.shape[-4:]
        st = k.stride()
        self.desc = CacheDesc(k.data_ptr(), v.data_ptr(), st[0] if k.dim() == 5 else 0, st[-4], st[-3], st[-2],
                              self.layers, self.pages, self.page_size)
        self.ref = ctypes.byref(self.desc)

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
    the slots (T,) int64 (page * page_size + place; negative = not written).
    q_out=q and k_out=k work in place.  Returns (q_out, k_out)."""
    qd, kd = _heads(q, "q"), _heads(k, "k")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    _need(k.shape == (T, Hkv, D), "k must be (T, Hkv, D)")
    if q_out is None:
        q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=q.device)
    if k_out is None:
        k_out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=q.device)
    qo, ko = _heads(q_out, "q_out"), _heads(k_out, "k_out")
    _need(q_out.shape == q.shape and k_out.shape == k.shape, "q_out / k_out shape")
    for w in (wq, wk):
        _need(w is None or (w.is_cuda and w.dtype is torch.bfloat16 and w.shape == (D,) and w.is_contiguous()),
              "wq / wk must be contiguous CUDA bf16 (D,) vectors")
    max_pos = rot = 0
    pp = None
    if cos_sin is not None:
        _need(cos_sin.is_cuda and cos_sin.dtype is torch.float32 and cos_sin.dim() == 2 and cos_sin.is_contiguous(),
              "cos_sin must be a contiguous CUDA f32 (max_pos, rot) tensor")
        max_pos, rot = cos_sin.shape
        _need(pos is not None, "a rotation needs pos")
        pp = _ints(pos, "pos")
        _need(pos.numel() == T, "pos must have one entry a token")
    vd = cd = sp = None
    if cache is not None:
        _need(v is not None and slots is not None, "a cache needs v and slots")
        _need(v.shape == k.shape and cache.hkv == Hkv and cache.d == D, "v or the cache does not fit k")
        vd, cd, sp = _heads(v, "v"), cache.ref, _ints(slots, "slots", 1, torch.int64)
        _need(slots.numel() == T, "slots must have one entry a token")
    _check("qk_norm_rope", lib().qk_norm_rope(
        qd, kd, T, Hq, Hkv, D, _ptr(wq), _ptr(wk), eps, pp, _ptr(cos_sin), max_pos, rot, int(interleaved), qo, ko,
        vd, cd, sp, _ptr(dev_status), _stream(stream)))
    return q_out, k_out


def _qkv(q, k, v, out):
    qd, kd, vd = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    _need(k.shape == (T, Hkv, D) and v.shape == k.shape, "k and v must be (T, Hkv, D)")
    if out is None:
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=q.device)
    _need(out.shape == q.shape, "out must have q's shape")
    return qd, kd, vd, _heads(out, "out"), out, T, Hq, Hkv, D


def _opts(ws, dev_status, timeout_ms, debug_stall):
    return AttnOpts(0 if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size(),
                    0 if dev_status is None else dev_status.data_ptr(), timeout_ms, debug_stall)


def attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                scale: float | None = None, out=None, dev_status=None, timeout_ms: int = 0, debug_stall: int = 0,
                stream=None) -> torch.Tensor:
    """Causal attention of packed prompts: q (T, Hq, D), k, v (T, Hkv, D),
    sequence b = rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 (int32, on the
    device).  scale None = 1/sqrt(D).  Returns out (T, Hq, D)."""
    qd, kd, vd, od, out, T, Hq, Hkv, D = _qkv(q, k, v, out)
    cu = _ints(cu_seqlens, "cu_seqlens")
    _check("attn_prompt", lib().attn_prompt(
        qd, kd, vd, cu, cu_seqlens.numel() - 1, T, Hq, Hkv, D, 1.0 / math.sqrt(D) if scale is None else scale, od,
        _opts(None, dev_status, timeout_ms, debug_stall), _stream(stream)))
    return out


_tree_ws: dict = {}


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
    seen by all.  Returns out (N, Hq, D)."""
    qd, kd, vd, od, out, N, Hq, Hkv, D = _qkv(q, k, v, out)
    cu, mp, cl = _ints(cu_nodes, "cu_nodes"), _ints(mask, "mask", 1, torch.int64), _ints(ctx_len, "ctx_len")
    B = ctx_len.numel()
    _need(cu_nodes.numel() == B + 1 and mask.numel() == N, "cu_nodes needs B + 1 entries, mask one a node")
    _need(cache.hkv == Hkv and cache.d == D, "the cache does not fit k")
    tp, ld, cols = _table(block_table, B, "block_table")
    if ws is None:
        key = (q.device, D)
        if key not in _tree_ws:
            _tree_ws[key] = mxg_attn_tree_workspace_bytes(D)
        ws = workspace(_tree_ws[key], q.device)
    _check("attn_tree", lib().attn_tree(
        qd, kd, vd, cu, mp, B, N, cache.ref, tp, ld, cols, cl, Hq, Hkv, D,
        1.0 / math.sqrt(D) if scale is None else scale, od, _opts(ws, dev_status, timeout_ms, debug_stall),
        _stream(stream)))
    return out


def kv_append(k: torch.Tensor, v: torch.Tensor, cu_nodes: torch.Tensor, accept: torch.Tensor, cache: KVCache,
              block_table: torch.Tensor, ctx_len: torch.Tensor, *, ctx_out=None, dev_status=None, stream=None):
    """The accepted nodes into the cache, in every layer: k, v (layers, N, Hkv,
    D), or (N, Hkv, D) with a one-layer cache; accept (B, most) int32: the
    nodes, counted from the sequence's first, that become tokens ctx_len[b],
    ctx_len[b] + 1, ... (the first negative entry ends the list).  Returns
    ctx_out (B,) = ctx_len + accepted."""
    _need(k.shape == v.shape and k.dim() in (3, 4), "k and v must be ([layers,] N, Hkv, D)")
    k0, v0, kl, vl = k, v, 0, 0
    if k.dim() == 4:
        _need(k.shape[0] == cache.layers, "k and the cache differ in layers")
        k0, v0, kl, vl = k[0], v[0], k.stride(0), v.stride(0)
    else:
        _need(cache.layers == 1, "k and the cache differ in layers")
    kd, vd = _heads(k0, "k"), _heads(v0, "v")
    N, Hkv, D = k0.shape
    _need(cache.hkv == Hkv and cache.d == D, "the cache does not fit k")
    B = ctx_len.numel()
    cu, cl = _ints(cu_nodes, "cu_nodes"), _ints(ctx_len, "ctx_len")
    _need(cu_nodes.numel() == B + 1, "cu_nodes needs B + 1 entries")
    ap, la, most = _table(accept, B, "accept")
    tp, ld, cols = _table(block_table, B, "block_table")
    if ctx_out is None:
        ctx_out = torch.empty_like(ctx_len)
    op = _ints(ctx_out, "ctx_out")
    _need(ctx_out.numel() == B, "ctx_out needs an entry a sequence")
    _check("kv_append", lib().kv_append(
        kd, kl, vd, vl, cu, B, N, ap, la, most, cache.ref, tp, ld, cols, cl, Hkv, D, op, _ptr(dev_status),
        _stream(stream)))
    return ctx_out
