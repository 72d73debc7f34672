"""Binding of include/fk_serve.h: rotary positions, attention of requests that
share a prefix, verification of drafted tokens, and pages of the cache forked,
returned, copied and compacted.  A serving step on the 4-bit cache is

    slots, positions, cu = cache.plan(new_lens, tokens)
    cache.rotate(q, k, turns)                            # fk_rope
    cache.append(k, v)
    out = cache.attend(q, max_q, shared=(cu_groups, prefix_lens))
    accepted, emitted = cache.verify(tokens, target, draft, accept, pick)

with cache.fork(rows, sources) where requests continue each other, and
cache.compact() between steps.  The functions here check and marshal their
tensors, as those of kv4.py do; nothing waits for the GPU.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import DTYPES, _check, _FLOATS, _on, _P, lib
from .kv4 import (_at, _ATTN, _CACHE, _cache, _device_of, _I32, _i32, _I64, _on_gpu, _rows_at, _stream_of, _SZ, _tensor,
                  _ws_at)

__all__ = ["fk_rope", "rope_turns", "fk_verify", "verify_workspace", "fk_kv_fork", "kv_fork_workspace", "fk_kv_compact",
           "kv_compact_workspace", "fk_kv4_copy", "fk_kv4_attention_shared", "kv4_attention_shared_workspace"]

# the structs of the C ABI, packed field by field (see kv4.py)
_ROPE = struct.Struct("@qiiiiifPP")
_ROPE_ROWS = struct.Struct("@PPqqqqii")
_VERIFY = struct.Struct("@qqqPPPPqqiiPPPPPP")
_POOL = struct.Struct("@qqqiiPPPPP")

for _name, (_args, _res) in {
    "fk_rope": ([_P, _I32, _P, _P], ctypes.c_int),
    "fk_verify_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "fk_verify": ([_P, _P, _SZ, _P], ctypes.c_int),
    "fk_kv_fork_workspace_bytes": ([_I64, _P], _SZ),
    "fk_kv_fork": ([_P, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "fk_kv_compact_workspace_bytes": ([_I64], _SZ),
    "fk_kv_compact": ([_P, _P, _P, _P, _P, _P, _I64, _P, _SZ, _P], ctypes.c_int),
    "fk_kv4_copy": ([_P, _I64, _P, _P], ctypes.c_int),
    "fk_kv4_attn_shared_workspace_bytes": ([_P, _I64, _I64, _I32, _I32, _I64], _SZ),
    "fk_kv4_attention_shared": ([_P, _P, _I64, _P, _P, _P, _SZ, _P], ctypes.c_int),
}.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

_f32, _i64 = torch.float32, torch.int64


def _sized(n: int) -> int:
    if n == 0:
        raise ValueError(lib.fk_last_error().decode())
    return n


# ---- rotary positions ------------------------------------------------------------

def rope_turns(rot_dim: int, base: float = 10000.0, stretch: float = 1.0, trained: int = 0, slow: float = 1.0,
               fast: float = 32.0, device="cuda") -> torch.Tensor:
    """The turns table of fk_rope (rot_dim / 2, int64): pair i advances by
    base^(-2 i / rot_dim) radians a position.  For contexts `stretch` times as
    long as the `trained` length, pairs that turn `slow` times or less over it
    advance stretch times slower, those that turn `fast` times or more as
    before, and those between by a mean of both, weighted by the turns; trained
    0: all stretch times slower.  That is interpolation "by parts" as published by
    Peng et al. (YaRN, 2023), whose factor beside it is 1 + 0.1 ln(stretch);
    positions that are all interpolated are trained = 0.  Other frequencies w
    (radians a position) are round(w / 2 pi 2^64) modulo 2^64, as int64."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not base > 0 or not stretch > 0 or not math.isfinite(base) or not math.isfinite(stretch):
        raise ValueError("base and stretch must be positive and finite")
    if trained and not fast > slow:
        raise ValueError("fast must be greater than slow")
    turns = []
    for i in range(rot_dim // 2):
        w = base ** (-2.0 * i / rot_dim)
        share = 0.0
        if trained:
            share = min(1.0, max(0.0, (trained * w / (2 * math.pi) - slow) / (fast - slow)))
        w = w * share + w / stretch * (1.0 - share)
        t = round(w / (2 * math.pi) * 2.0 ** 64) % 2 ** 64          # a float holds it to 2^-53 of its value
        turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    return torch.tensor(turns, dtype=_i64, device=device)


def fk_rope(q, k, positions, turns, q_out=None, k_out=None, interleaved: bool = False, inverse: bool = False,
            factor: float = 1.0, stream=None) -> None:
    """Rotary positions of q (T, q_heads, head_dim) and, unless None, k (T,
    kv_heads, head_dim), into q_out and k_out (None: in place); positions (T)
    int32, negative: the row is copied; turns from rope_turns, of 2 len(turns)
    elements of a head.  inverse rotates back, which is also what takes the
    gradient of the outputs to that of the inputs.  Tokens and heads may be
    strided."""
    T, Hq, D = shape = _tensor(q, "q", 3)
    if q.dtype not in _FLOATS:
        raise ValueError(f"q must be float32, float16 or bfloat16, got {q.dtype}")
    index, rows = q.get_device(), []
    for x, y, name in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            if y is not None:
                raise ValueError(f"{name}_out is given without {name}")
            continue
        if name == "k":
            shape = torch.Size((T, _tensor(k, "k", 3)[1], D))
        at, token, head = _rows_at(x, name, q.dtype, shape, index)
        to, token2, head2 = (at, token, head) if y is None else _rows_at(y, name + "_out", q.dtype, shape, index)
        rows.append(_ROPE_ROWS.pack(at, to, token, head, token2, head2, shape[1], 0))
    pairs = _tensor(turns, "turns", 1)
    try:
        args = _ROPE.pack(T, D, 2 * pairs[0], DTYPES[q.dtype], bool(interleaved), bool(inverse), factor,
                          _at(positions, "positions", _i32, torch.Size((T,)), index), _at(turns, "turns", _i64, pairs, index))
    except (struct.error, OverflowError) as e:
        raise ValueError(f"factor is no fp32 number: {e}") from None
    _on_gpu(index)
    status = lib.fk_rope(args, len(rows), b"".join(rows), _stream_of(stream, index))
    if status:
        _check(status, "fk_rope")


# ---- verification of drafts ---------------------------------------------------------

def _distribution(t, name, dtype, shape, index):
    """Address and row stride of (T, V) values whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected {_device_of(index)}")
    if t.stride(1) != 1 and shape[1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), t.stride(0)


def verify_workspace(cu, target) -> torch.Tensor:
    """A caller-owned workspace for fk_verify of these sizes and smaller ones."""
    T, V = _tensor(target, "target", 2)
    return torch.empty(_sized(lib.fk_verify_workspace_bytes(_tensor(cu, "cu", 1)[0] - 1, T, V)), dtype=torch.uint8,
                       device=target.device)


def fk_verify(cu, tokens, target, accepted, emitted, draft=None, accept=None, pick=None, seq_lens=None, keep=None, ws=None,
              stream=None) -> None:
    """Which drafts the target keeps.  Request b has rows cu[b] .. cu[b + 1] -
    1 (cu int32); tokens (T) int32 are the step's input tokens, those of a
    request after its first being drafts; target (T, V) the probabilities of
    the token after each row, draft (T, V) those that the drafts were drawn
    from or None where they are certain; accept (T) and pick (B) fp32 uniform
    numbers, or both None for greedy decoding (target may then be logits).  A
    draft that is no token (-1, say) stands for none: it is refused, and the
    token is drawn from the target alone.
    Writes accepted (B), emitted (T: the drafts kept, a token more, then -1)
    and, unless None, keep (B): seq_lens without the drafts refused, as
    KV4Cache.release takes it."""
    T, V = shape = _tensor(target, "target", 2)
    if target.dtype not in _FLOATS:
        raise ValueError(f"target must be float32, float16 or bfloat16, got {target.dtype}")
    B, index = _tensor(cu, "cu", 1)[0] - 1, target.get_device()
    rows, one = torch.Size((T,)), torch.Size((B,)) if B > 0 else None
    if one is None:
        raise ValueError("cu must have an entry more than there are requests")
    if (accept is None) != (pick is None):
        raise ValueError("accept and pick come together")
    if keep is not None and seq_lens is None:
        raise ValueError("keep needs seq_lens")
    p, p_row = _distribution(target, "target", target.dtype, shape, index)
    q, q_row = (0, 0) if draft is None else _distribution(draft, "draft", target.dtype, shape, index)
    args = _VERIFY.pack(
        B, T, V, _at(cu, "cu", _i32, torch.Size((B + 1,)), index), _at(tokens, "tokens", _i32, rows, index), p, q, p_row, q_row,
        DTYPES[target.dtype], 0, 0 if accept is None else _at(accept, "accept", _f32, rows, index),
        0 if pick is None else _at(pick, "pick", _f32, one, index),
        0 if seq_lens is None else _at(seq_lens, "seq_lens", _i32, one, index), _at(accepted, "accepted", _i32, one, index),
        _at(emitted, "emitted", _i32, rows, index), 0 if keep is None else _at(keep, "keep", _i32, one, index))
    _on_gpu(index)
    if ws is None:
        with _on(stream, target.device):
            ws = verify_workspace(cu, target)
    _check(lib.fk_verify(args, *_ws_at(ws, index), _stream_of(stream, index)), "fk_verify")


# ---- pages ------------------------------------------------------------------------------

def _pool(page_size, block_table, lens, shares, free_pages, free_count):
    """The C description of a pool and its device."""
    R, M = table = _tensor(block_table, "block_table", 2)
    pages = _tensor(shares, "shares", 1)
    index = block_table.get_device()
    return _POOL.pack(R, M, pages[0], int(page_size), 0, _at(block_table, "block_table", _i32, table, index),
                      _at(lens, "lens", _i32, torch.Size((R,)), index), _at(shares, "shares", _i32, pages, index),
                      _at(free_pages, "free_pages", _i32, pages, index),
                      _at(free_count, "free_count", _i32, torch.Size((1,)), index)), index


def kv_fork_workspace(n: int, block_table, shares, page_size: int = 32) -> torch.Tensor:
    """A caller-owned workspace for fk_kv_fork of up to n pairs."""
    R, M = _tensor(block_table, "block_table", 2)
    pool = _POOL.pack(R, M, _tensor(shares, "shares", 1)[0], page_size, 0, 0, 0, 0, 0, 0)
    return torch.empty(_sized(lib.fk_kv_fork_workspace_bytes(n, pool)), dtype=torch.uint8, device=block_table.device)


def fk_kv_fork(rows, sources, keep, page_size: int, block_table, lens, shares, free_pages, free_count, copies, seq=None, ws=None,
               stream=None) -> None:
    """Row rows[i] of the table becomes the first keep[i] tokens of row
    sources[i], all at once (all int32); sources None: of itself.  Whole pages
    are shared (shares: rows that hold a page, beyond the first), pages that
    nobody holds any more go to the list, and copies (n, 3) says which partly
    filled pages fk_kv4_copy must copy, in every cache that the table serves.
    seq: lengths to be kept in step, or None."""
    (n,) = one = _tensor(rows, "rows", 1)
    pool, index = _pool(page_size, block_table, lens, shares, free_pages, free_count)
    args = (_at(rows, "rows", _i32, one, index), None if sources is None else _at(sources, "sources", _i32, one, index),
            _at(keep, "keep", _i32, one, index), _at(copies, "copies", _i32, torch.Size((n, 3)), index),
            None if seq is None else _at(seq, "seq", _i32, lens.shape, index))
    _on_gpu(index)
    if ws is None:
        with _on(stream, block_table.device):
            ws = kv_fork_workspace(n, block_table, shares, page_size)
    _check(lib.fk_kv_fork(pool, n, *args, *_ws_at(ws, index), _stream_of(stream, index)), "fk_kv_fork")


def kv_compact_workspace(shares) -> torch.Tensor:
    """A caller-owned workspace for fk_kv_compact of a pool."""
    return torch.empty(_sized(lib.fk_kv_compact_workspace_bytes(_tensor(shares, "shares", 1)[0])), dtype=torch.uint8,
                       device=shares.device)


def fk_kv_compact(page_size: int, block_table, lens, shares, free_pages, free_count, new_table, new_shares, new_free, free_left,
                  moves, ws=None, stream=None) -> None:
    """Numbers the pages in use 0, 1, ...: the table, shares, list and its
    length with the new numbers (each may be its input), and moves (n, 3), n >=
    pages / 2, for fk_kv4_copy."""
    pool, index = _pool(page_size, block_table, lens, shares, free_pages, free_count)
    n, _ = many = _tensor(moves, "moves", 2)
    if many[1] != 3:
        raise ValueError("moves must have shape (n, 3)")
    args = (_at(new_table, "new_table", _i32, block_table.shape, index), _at(new_shares, "new_shares", _i32, shares.shape, index),
            _at(new_free, "new_free", _i32, shares.shape, index), _at(free_left, "free_left", _i32, torch.Size((1,)), index),
            _at(moves, "moves", _i32, many, index))
    _on_gpu(index)
    if ws is None:
        with _on(stream, block_table.device):
            ws = kv_compact_workspace(shares)
    _check(lib.fk_kv_compact(pool, *args, n, *_ws_at(ws, index), _stream_of(stream, index)), "fk_kv_compact")


def fk_kv4_copy(copies, codes, scales, stream=None) -> None:
    """Pages of a cache to other pages of it: copies (n, 3) int32 as fk_kv_fork
    and fk_kv_compact write them, (source, destination, tokens)."""
    pages, H, two, blocks, row = _tensor(codes, "codes", 5)
    index = codes.get_device()
    if codes.dtype is not torch.uint8 or two != 2 or row % 16:
        raise ValueError("codes must be uint8 (pages, kv_heads, 2, page_size / 32, 16 * head_dim)")
    _at(codes, "codes", torch.uint8, codes.shape, index)
    if scales.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("scales must be float16 or bfloat16")
    _at(scales, "scales", scales.dtype, torch.Size((pages, H, 2, 32 * blocks)), index)
    n, three = many = _tensor(copies, "copies", 2)
    if three != 3:
        raise ValueError("copies must have shape (n, 3)")
    at = _at(copies, "copies", _i32, many, index)
    _on_gpu(index)
    # a copy looks nothing up: any address does for the codebook
    c = _CACHE.pack(codes.data_ptr(), scales.data_ptr(), codes.data_ptr(), pages, 32 * blocks, H, row // 16, DTYPES[scales.dtype])
    status = lib.fk_kv4_copy(c, n, at, _stream_of(stream, index))
    if status:
        _check(status, "fk_kv4_copy")


# ---- attention of requests that share a prefix ------------------------------------------

def kv4_attention_shared_workspace(q, seq_lens, prefix_lens, codes, max_q: int) -> torch.Tensor:
    """A caller-owned workspace for fk_kv4_attention_shared of these sizes, and of
    fewer requests and groups; of fewer tokens too where max_q q_heads /
    kv_heads is at most 48 (16 for 256 dimensions)."""
    T, Hq, D = _tensor(q, "q", 3)
    pages, H, _, blocks, _ = _tensor(codes, "codes", 5)
    c = _CACHE.pack(0, 0, 0, pages, 32 * blocks, H, D, DTYPES.get(q.dtype, -1))
    n = _sized(lib.fk_kv4_attn_shared_workspace_bytes(c, seq_lens.numel(), T, Hq, int(max_q), prefix_lens.numel()))
    return torch.empty(n, dtype=torch.uint8, device=codes.device)


def fk_kv4_attention_shared(q, cu_q, seq_lens, block_table, cu_groups, prefix_lens, codebook, codes, scales, out, max_q: int,
                            scale: float | None = None, causal: bool = True, window: int = 0, lse=None, ws=None,
                            stream=None) -> None:
    """fk_kv4_attention where the requests cu_groups[g] .. cu_groups[g + 1] - 1
    (int32, ascending; others share nothing) have their first prefix_lens[g]
    tokens in common: those are read once for all of them, through the table's
    row of the first.  For prefixes that are long beside the requests' own tokens
    and the table's room; short ones in a wide table are faster without."""
    c, H, D, dtype, index = _cache(codebook, codes, scales)
    T, Hq, _ = _tensor(q, "q", 3)
    rows = torch.Size((T, Hq, D))
    at, token, head = _rows_at(q, "q", dtype, rows, index)
    (B,) = one = _tensor(seq_lens, "seq_lens", 1)
    table = _tensor(block_table, "block_table", 2)
    (groups,) = some = _tensor(prefix_lens, "prefix_lens", 1)
    try:
        args = _ATTN.pack(
            B, T, Hq, max_q, table[1], token, head, at, _at(cu_q, "cu_q", _i32, torch.Size((B + 1,)), index),
            _at(seq_lens, "seq_lens", _i32, one, index), _at(block_table, "block_table", _i32, torch.Size((B, table[1])), index),
            1.0 / math.sqrt(D) if scale is None else scale, bool(causal), window, _at(out, "out", dtype, rows, index),
            0 if lse is None else _at(lse, "lse", _f32, torch.Size((T, Hq)), index))
    except struct.error as e:
        raise ValueError(f"max_q, window or scale is no number of its range: {e}") from None
    more = (_at(cu_groups, "cu_groups", _i32, torch.Size((groups + 1,)), index), _at(prefix_lens, "prefix_lens", _i32, some, index))
    _on_gpu(index)
    if ws is None:
        with _on(stream, codes.device):
            ws = kv4_attention_shared_workspace(q, seq_lens, prefix_lens, codes, max_q)
    _check(lib.fk_kv4_attention_shared(c, args, groups, *more, *_ws_at(ws, index), _stream_of(stream, index)),
           "fk_kv4_attention_shared")
