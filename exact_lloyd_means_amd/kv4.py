"""A paged key/value cache held in 4 bits, and attention over it.

Low-bit KV quantisation is one of the uses the pages name for exact batched
k-means (papernotes.org notes, 研究背景与动机; 7minutos.es article, "Casos de
uso").  Here a codebook is what k-means gives for the normalised values of
one head: 16 centroids, so a value is kept as a 4-bit index and every row
(one token, one head) as its codes and one scale.

Two layers, as elsewhere in the package: functions named as the C ABI of
include/fk_kv4.h, which only check and marshal their tensors, and
``KV4Cache``, which holds the buffers of a serving loop:

    codebook = learn_codebook(k_sample, v_sample)
    cache = KV4Cache(pages, 64, kv_heads, head_dim, codebook, max_requests, max_len)
    step = cache.plan(new_lens, tokens)        # block tables, slots, positions
    cache.append(k, v)                         # (tokens, kv_heads, head_dim)
    out = cache.attend(q, max_q)               # (tokens, q_heads, head_dim)

Nothing here waits for the GPU.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (DTYPES, _check, _need_gpu, _P, _stream, _want, _want_ws, lib)

__all__ = ["fk_kv_plan", "fk_kv4_write", "fk_kv4_read",
           "fk_kv4_attention", "kv_plan_workspace", "kv4_attention_workspace"]

_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class Kv4CacheArgs(ctypes.Structure):
    _fields_ = [("codes", _P), ("scales", _P), ("codebook", _P), ("pages", _I64),
                ("page_size", _I32), ("kv_heads", _I32), ("head_dim", _I32), ("dtype", _I32)]


class Kv4AttnArgs(ctypes.Structure):
    _fields_ = [("B", _I64), ("T", _I64), ("q_heads", _I32), ("max_q", _I32), ("max_pages", _I64),
                ("q_token", _I64), ("q_head", _I64), ("q", _P), ("cu_q", _P), ("seq_lens", _P),
                ("block_table", _P), ("scale", ctypes.c_float), ("causal", _I32),
                ("window", _I32), ("out", _P), ("lse", _P)]


_CP, _AP = ctypes.POINTER(Kv4CacheArgs), ctypes.POINTER(Kv4AttnArgs)
for _name, (_args, _res) in {
    "fk_kv_plan_workspace_bytes": ([_I64], _SZ),
    "fk_kv_plan": ([_I64, _I64, _I32, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P,
                    _SZ, _P], ctypes.c_int),
    "fk_kv4_write": ([_CP, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "fk_kv4_read": ([_CP, _I64, _P, _P, _P, _P], ctypes.c_int),
    "fk_kv4_attn_workspace_bytes": ([_CP, _I64, _I64, _I32, _I32], _SZ),
    "fk_kv4_attention": ([_CP, _AP, _P, _SZ, _P], ctypes.c_int),
}.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

_HALVES = (torch.float16, torch.bfloat16)


def _cache_args(codebook, codes, scales):
    """The C description of a cache, from its three tensors."""
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a torch tensor")
    if codes.dtype != torch.uint8 or codes.dim() != 5 or codes.shape[2] != 2:
        raise ValueError("codes must be uint8 (pages, kv_heads, 2, page_size / 32, 16 * head_dim)")
    pages, H, _, blocks, row = codes.shape
    if row % 16:
        raise ValueError("the last dimension of codes must be 16 * head_dim")
    dev = codes.device
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    _want(scales, "scales", _HALVES, (pages, H, 2, 32 * blocks), dev)
    if codebook is not None:
        _want(codebook, "codebook", torch.float16, (2, H, 16), dev)
    return Kv4CacheArgs(codes.data_ptr(), scales.data_ptr(),
                        None if codebook is None else codebook.data_ptr(), pages, 32 * blocks, H,
                        row // 16, DTYPES[scales.dtype]), dev


def _want_rows(t, name, dtype, shape, dev):
    """A (tokens, heads, head_dim) tensor whose rows are contiguous; tokens
    and heads may be strided (a slice of a fused projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.stride(2) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")


def kv_plan_workspace(B: int, device=None) -> torch.Tensor:
    """A caller-owned workspace for fk_kv_plan of B requests."""
    return torch.empty(max(1, lib.fk_kv_plan_workspace_bytes(B)), dtype=torch.uint8,
                       device=device or "cuda")


def fk_kv_plan(ctx_lens, new_lens, page_size: int, free_pages, free_count, block_table, seq_lens,
               cu_new, slots, positions, free_left, status, ws=None, stream=None) -> None:
    """Block tables and slot maps of one step from the lengths on the GPU
    (all int32): writes the needed entries of block_table (B, max_pages),
    seq_lens (B), cu_new (B + 1), slots and positions (any length; positions
    may be None), free_left (1) and status (4)."""
    if not isinstance(ctx_lens, torch.Tensor):
        raise TypeError("ctx_lens must be a torch tensor")
    dev, i32 = ctx_lens.device, torch.int32
    B = ctx_lens.numel()
    _want(ctx_lens, "ctx_lens", i32, (B,), dev)
    _want(new_lens, "new_lens", i32, (B,), dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a (B, max_pages) tensor")
    M = block_table.shape[1]
    _want(block_table, "block_table", i32, (B, M), dev)
    _want(seq_lens, "seq_lens", i32, (B,), dev)
    _want(cu_new, "cu_new", i32, (B + 1,), dev)
    for t, name in ((free_pages, "free_pages"), (slots, "slots")):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise ValueError(f"{name} must be a 1-D tensor")
        _want(t, name, i32, t.shape, dev)
    _want(positions, "positions", i32, slots.shape, dev, optional=True)
    _want(free_count, "free_count", i32, (1,), dev)
    _want(free_left, "free_left", i32, (1,), dev)
    _want(status, "status", i32, (4,), dev)
    _want_ws(ws, dev)
    _need_gpu(dev)
    ws = kv_plan_workspace(B, dev) if ws is None else ws
    _check(lib.fk_kv_plan(B, M, int(page_size), ctx_lens.data_ptr(), new_lens.data_ptr(),
                          free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(),
                          block_table.data_ptr(), seq_lens.data_ptr(), cu_new.data_ptr(),
                          slots.data_ptr(), None if positions is None else positions.data_ptr(),
                          slots.numel(), free_left.data_ptr(), status.data_ptr(), ws.data_ptr(),
                          ws.numel(), _stream(stream)), "fk_kv_plan")


def fk_kv4_write(k, v, slots, codebook, codes, scales, stream=None) -> None:
    """Rows k, v (T, kv_heads, head_dim) into the slots (T) of the cache."""
    c, dev = _cache_args(codebook, codes, scales)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D tensor")
    T = slots.numel()
    _want(slots, "slots", torch.int32, (T,), dev)
    _want_rows(k, "k", scales.dtype, (T, c.kv_heads, c.head_dim), dev)
    _want_rows(v, "v", scales.dtype, (T, c.kv_heads, c.head_dim), dev)
    _need_gpu(dev)
    _check(lib.fk_kv4_write(c, T, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                            v.stride(0), v.stride(1), slots.data_ptr(), _stream(stream)),
           "fk_kv4_write")


def fk_kv4_read(slots, codebook, codes, scales, k, v, stream=None) -> None:
    """The rows of the slots (T) as values: k, v (T, kv_heads, head_dim)."""
    c, dev = _cache_args(codebook, codes, scales)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D tensor")
    T = slots.numel()
    _want(slots, "slots", torch.int32, (T,), dev)
    _want(k, "k", scales.dtype, (T, c.kv_heads, c.head_dim), dev)
    _want(v, "v", scales.dtype, (T, c.kv_heads, c.head_dim), dev)
    _need_gpu(dev)
    _check(lib.fk_kv4_read(c, T, slots.data_ptr(), k.data_ptr(), v.data_ptr(), _stream(stream)),
           "fk_kv4_read")


def kv4_attention_workspace(q, seq_lens, codes, max_q: int) -> torch.Tensor:
    """A caller-owned workspace for fk_kv4_attention of these sizes."""
    T, Hq, D = q.shape
    pages, H, _, blocks, _ = codes.shape
    c = Kv4CacheArgs(None, None, None, pages, 32 * blocks, H, D, DTYPES.get(q.dtype, -1))
    n = lib.fk_kv4_attn_workspace_bytes(c, seq_lens.numel(), T, Hq, int(max_q))
    if n == 0:
        raise ValueError(lib.fk_last_error().decode())
    return torch.empty(n, dtype=torch.uint8, device=codes.device)


def fk_kv4_attention(q, cu_q, seq_lens, block_table, codebook, codes, scales, out, max_q: int,
                     scale: float | None = None, causal: bool = True, window: int = 0, lse=None,
                     ws=None, stream=None) -> None:
    """Attention of the query tokens q (T, q_heads, head_dim), request b's at
    cu_q[b] .. cu_q[b + 1] - 1, over the cached tokens of their requests; out
    like q, contiguous; lse (T, q_heads) fp32 or None; scale None: 1 /
    sqrt(head_dim)."""
    c, dev = _cache_args(codebook, codes, scales)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a (T, q_heads, head_dim) tensor")
    T, Hq, D = q.shape
    _want_rows(q, "q", scales.dtype, (T, Hq, c.head_dim), dev)
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be a 1-D tensor")
    B, i32 = seq_lens.numel(), torch.int32
    _want(seq_lens, "seq_lens", i32, (B,), dev)
    _want(cu_q, "cu_q", i32, (B + 1,), dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a (B, max_pages) tensor")
    M = block_table.shape[1]
    _want(block_table, "block_table", i32, (B, M), dev)
    _want(out, "out", scales.dtype, (T, Hq, D), dev)
    _want(lse, "lse", torch.float32, (T, Hq), dev, optional=True)
    _want_ws(ws, dev)
    _need_gpu(dev)
    ws = kv4_attention_workspace(q, seq_lens, codes, max_q) if ws is None else ws
    a = Kv4AttnArgs(B, T, Hq, int(max_q), M, q.stride(0), q.stride(1), q.data_ptr(),
                    cu_q.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                    1.0 / math.sqrt(D) if scale is None else float(scale), int(bool(causal)),
                    int(window), out.data_ptr(), None if lse is None else lse.data_ptr())
    _check(lib.fk_kv4_attention(c, a, ws.data_ptr(), ws.numel(), _stream(stream)),
           "fk_kv4_attention")
