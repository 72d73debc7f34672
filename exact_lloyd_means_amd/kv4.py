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

Nothing here waits for the GPU.  With stream= a call runs there, and what it
allocates, its results among them, belongs to that stream; its inputs must be
ready there.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import DTYPES, _check, _need_gpu, _on, _P, _stream, _want, _want_ws, lib

__all__ = ["KV4Cache", "learn_codebook", "fk_kv_plan", "fk_kv4_write", "fk_kv4_read", "fk_kv4_attention", "kv_plan_workspace",
           "kv4_attention_workspace"]

_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
# fk_kv4_cache and fk_kv4_attn of the C ABI, packed field by field: a decode
# step makes several calls of a few microseconds, and a ctypes.Structure costs
# more to fill than the rest of a call
_CACHE = struct.Struct("@PPPqiiii")
_ATTN = struct.Struct("@qqiiqqqPPPPfiiPP")

for _name, (_args, _res) in {
    "fk_kv_plan_workspace_bytes": ([_I64], _SZ),
    "fk_kv_plan": ([_I64, _I64, _I32, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P,
                    _SZ, _P], ctypes.c_int),
    "fk_kv_plan_kept": ([_I64, _I64, _I32, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P,
                         _P, _P, _SZ, _P], ctypes.c_int),
    "fk_kv4_write": ([_P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "fk_kv4_read": ([_P, _I64, _P, _P, _P, _P], ctypes.c_int),
    "fk_kv4_attn_workspace_bytes": ([_P, _I64, _I64, _I32, _I32], _SZ),
    "fk_kv4_attention": ([_P, _P, _P, _SZ, _P], ctypes.c_int),
}.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

_HALVES = (torch.float16, torch.bfloat16)
_i32, _f16, _u8 = torch.int32, torch.float16, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device_of(index):
    return torch.device("cuda", index) if index >= 0 else torch.device("cpu")


def _at(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this dtype and shape on the device
    of this index (-1: CPU).  Anything else goes to the binding's checks,
    which say what is wrong with it."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == index
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _want(t, name, dtype, shape, _device_of(index))
    return t.data_ptr()


def _rows_at(t, name, dtype, shape, index):
    """Address and strides of a (tokens, heads, head_dim) tensor whose rows
    are contiguous; tokens and heads may be strided (a slice of a fused
    projection)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index:
            token, head, one = t.stride()
            if one == 1:
                return t.data_ptr(), token, head
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected {_device_of(index)}")
    raise ValueError(f"the last dimension of {name} must be contiguous")


def _tensor(t, name, dims):
    """The shape of a tensor of so many dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(shape)}")
    return shape


def _on_gpu(index):
    if index < 0:
        _need_gpu(_device_of(index))


def _stream_of(stream, index):
    if stream is None and _raw_stream is not None:
        return _raw_stream(index)
    return _stream(stream)


def _ws_at(ws, index):
    if ws.dtype is not _u8 or ws.dim() != 1 or ws.get_device() != index:
        _want_ws(ws, _device_of(index))
    return ws.data_ptr(), ws.numel()


def _cache(codebook, codes, scales):
    """The C description of a cache, its heads, head_dim, dtype and device."""
    try:
        pages, H, two, blocks, row = codes.shape
        dtype, index = scales.dtype, codes.get_device()
        if (codes.dtype is _u8 and two == 2 and not row % 16 and codes.is_contiguous()
                and dtype in _HALVES and scales.shape == (pages, H, 2, 32 * blocks)
                and scales.get_device() == index and scales.is_contiguous()
                and codebook.dtype is _f16 and codebook.shape == (2, H, 16)
                and codebook.get_device() == index and codebook.is_contiguous()):
            return (_CACHE.pack(codes.data_ptr(), scales.data_ptr(), codebook.data_ptr(), pages,
                                32 * blocks, H, row // 16, DTYPES[dtype]),
                    H, row // 16, dtype, index)
    except (AttributeError, TypeError, ValueError):
        pass
    # says what is wrong
    pages, H, two, blocks, row = _tensor(codes, "codes", 5)
    if codes.dtype is not _u8 or two != 2 or row % 16:
        raise ValueError("codes must be uint8 (pages, kv_heads, 2, page_size / 32, 16 * head_dim)")
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    _want(scales, "scales", _HALVES, (pages, H, 2, 32 * blocks), codes.device)
    _want(codebook, "codebook", _f16, (2, H, 16), codes.device)
    raise ValueError("codes, scales and codebook do not describe a cache")


def kv_plan_workspace(B: int, device=None) -> torch.Tensor:
    """A caller-owned workspace for fk_kv_plan of B requests."""
    return torch.empty(max(1, lib.fk_kv_plan_workspace_bytes(B)), dtype=torch.uint8,
                       device=device or "cuda")


def fk_kv_plan(ctx_lens, new_lens, page_size: int, free_pages, free_count, block_table, seq_lens,
               cu_new, slots, positions, free_left, status, ws=None, stream=None,
               kept_lens=None) -> None:
    """Block tables and slot maps of one step from the lengths on the GPU
    (all int32): writes the needed entries of block_table (B, max_pages),
    seq_lens (B), cu_new (B + 1), slots and positions (any length; positions
    may be None), free_left (1), status (4) and, unless None, kept_lens (B):
    what the cache then holds, the next step's ctx_lens (seq_lens unless pages
    ran out)."""
    (B,) = one = _tensor(ctx_lens, "ctx_lens", 1)
    table = _tensor(block_table, "block_table", 2)
    free = _tensor(free_pages, "free_pages", 1)
    cap = _tensor(slots, "slots", 1)
    index = ctx_lens.get_device()
    args = (B, table[1], int(page_size), _at(ctx_lens, "ctx_lens", _i32, one, index),
            _at(new_lens, "new_lens", _i32, one, index), _at(free_pages, "free_pages", _i32, free, index),
            free[0], _at(free_count, "free_count", _i32, (1,), index),
            _at(block_table, "block_table", _i32, (B, table[1]), index),
            _at(seq_lens, "seq_lens", _i32, one, index), _at(cu_new, "cu_new", _i32, (B + 1,), index),
            _at(slots, "slots", _i32, cap, index),
            None if positions is None else _at(positions, "positions", _i32, cap, index), cap[0],
            _at(free_left, "free_left", _i32, (1,), index), _at(status, "status", _i32, (4,), index),
            None if kept_lens is None else _at(kept_lens, "kept_lens", _i32, one, index))
    _on_gpu(index)
    if ws is None:
        with _on(stream, ctx_lens.device):
            ws = kv_plan_workspace(B, ctx_lens.device)
    _check(lib.fk_kv_plan_kept(*args, *_ws_at(ws, index), _stream_of(stream, index)), "fk_kv_plan")


def fk_kv4_write(k, v, slots, codebook, codes, scales, stream=None) -> None:
    """Rows k, v (T, kv_heads, head_dim) into the slots (T) of the cache."""
    c, H, D, dtype, index = _cache(codebook, codes, scales)
    (T,) = one = _tensor(slots, "slots", 1)
    at = _at(slots, "slots", _i32, one, index)
    rows = (T, H, D)
    ka, kt, kh = _rows_at(k, "k", dtype, rows, index)
    va, vt, vh = _rows_at(v, "v", dtype, rows, index)
    _on_gpu(index)
    status = lib.fk_kv4_write(c, T, ka, kt, kh, va, vt, vh, at, _stream_of(stream, index))
    if status:
        _check(status, "fk_kv4_write")


def fk_kv4_read(slots, codebook, codes, scales, k, v, stream=None) -> None:
    """The rows of the slots (T) as values: k, v (T, kv_heads, head_dim)."""
    c, H, D, dtype, index = _cache(codebook, codes, scales)
    (T,) = one = _tensor(slots, "slots", 1)
    args = (_at(slots, "slots", _i32, one, index), _at(k, "k", dtype, (T, H, D), index),
            _at(v, "v", dtype, (T, H, D), index))
    _on_gpu(index)
    _check(lib.fk_kv4_read(c, T, *args, _stream_of(stream, index)), "fk_kv4_read")


def kv4_attention_workspace(q, seq_lens, codes, max_q: int) -> torch.Tensor:
    """A caller-owned workspace for fk_kv4_attention of these sizes."""
    T, Hq, D = _tensor(q, "q", 3)
    pages, H, _, blocks, _ = _tensor(codes, "codes", 5)
    c = _CACHE.pack(0, 0, 0, pages, 32 * blocks, H, D, DTYPES.get(q.dtype, -1))
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
    sqrt(head_dim).  max_q: most query tokens of a request, or more; those
    from max_q on get no rows of out and lse."""
    c, H, D, dtype, index = _cache(codebook, codes, scales)
    T, Hq, _ = _tensor(q, "q", 3)
    rows = (T, Hq, D)
    at, token, head = _rows_at(q, "q", dtype, rows, index)
    (B,) = one = _tensor(seq_lens, "seq_lens", 1)
    table = _tensor(block_table, "block_table", 2)
    try:
        args = _ATTN.pack(
            B, T, Hq, max_q, table[1], token, head, at, _at(cu_q, "cu_q", _i32, (B + 1,), index),
            _at(seq_lens, "seq_lens", _i32, one, index),
            _at(block_table, "block_table", _i32, (B, table[1]), index),
            1.0 / math.sqrt(D) if scale is None else scale, bool(causal), window,
            _at(out, "out", dtype, rows, index),
            0 if lse is None else _at(lse, "lse", torch.float32, (T, Hq), index))
    except struct.error as e:
        raise ValueError(f"max_q, window or scale is no number of its range: {e}") from None
    _on_gpu(index)
    if ws is None:
        with _on(stream, codes.device):
            ws = kv4_attention_workspace(q, seq_lens, codes, max_q)
    _check(lib.fk_kv4_attention(c, args, *_ws_at(ws, index), _stream_of(stream, index)),
           "fk_kv4_attention")


def learn_codebook(k, v, iters: int = 30, stream=None) -> torch.Tensor:
    """Codebook (2, kv_heads, 16) fp16 from sample rows k, v (tokens,
    kv_heads, head_dim) on the GPU: exact Lloyd k-means (K = 16, d = 1, one
    problem a head, k and v) on the values over their row's largest
    magnitude, from equally spaced levels, in the library's deterministic
    mode.  A row with a value that is not finite counts as zeros.  Preparing
    the values is done with torch, on `stream` too, which waits for the current
    stream first and is waited for by it at the end."""
    from .api import batch_kmeans_euclid
    T, H, D = _tensor(k, "k", 3)
    if _tensor(v, "v", 3) != k.shape:
        raise ValueError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    _on_gpu(k.get_device())
    here = torch.cuda.current_stream(k.device)
    with _on(stream, k.device):
        there = torch.cuda.current_stream(k.device)
        there.wait_stream(here)
        x = torch.stack((k, v)).float()
        most = x.abs().amax(-1, keepdim=True)
        x = torch.where(most < math.inf, x / most.clamp(min=torch.finfo(torch.float32).tiny), 0.0)
        x = x.permute(0, 2, 1, 3).reshape(2 * H, T * D, 1).contiguous()
        first = torch.linspace(-1, 1, 16, device=x.device).view(16, 1)
        _, c, _ = batch_kmeans_euclid(x, 16, iters, init=first, deterministic=True, stream=stream)
        c = c.view(2, H, 16).sort(-1).values.half().contiguous()
    here.wait_stream(there)
    c.record_stream(here)
    return c


class KV4Cache:
    """The buffers of a serving loop around the functions above.

    pages x page_size tokens are shared by max_requests rows of a block table
    with room for max_len tokens each.  A step is plan(), append(), attend();
    release() returns a row's pages.  Lengths, tables and the list of free
    pages live on the GPU and no call waits for it.  The calls follow each
    other on one stream; a caller that changes streams orders them."""

    def __init__(self, pages: int, page_size: int, kv_heads: int, head_dim: int,
                 codebook: torch.Tensor, max_requests: int, max_len: int,
                 dtype=torch.bfloat16, device="cuda"):
        if page_size < 32 or page_size % 32:
            raise ValueError("page_size must be a multiple of 32")
        if dtype not in _HALVES:
            raise ValueError("dtype must be float16 or bfloat16")
        self.page_size = int(page_size)
        M = -(-int(max_len) // self.page_size)
        i32 = dict(dtype=torch.int32, device=device)
        # every byte is a valid code and no scale may be NaN
        self.codes = torch.zeros(pages, kv_heads, 2, page_size // 32, 16 * head_dim,
                                 dtype=torch.uint8, device=device)
        self.scales = torch.zeros(pages, kv_heads, 2, page_size, dtype=dtype, device=device)
        self.codebook = codebook
        self.block_table = torch.full((max_requests, M), -1, **i32)
        self.free_pages = torch.arange(pages - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), pages, **i32)
        self.status = torch.zeros(4, **i32)
        self.cu = torch.zeros(max_requests + 1, **i32)
        self._lens = [torch.zeros(max_requests, **i32) for _ in range(2)]
        self._seq = torch.zeros(max_requests, **i32)
        self._plan_ws = kv_plan_workspace(max_requests, device)
        self.slots = self.positions = None

    @property
    def lens(self) -> torch.Tensor:
        """Tokens of each row of the table (int32, on the GPU)."""
        return self._lens[0]

    def plan(self, new_lens: torch.Tensor, tokens: int, stream=None):
        """Makes room for new_lens (max_requests, int32, on the GPU) more
        tokens, `tokens` of them in all or more (the rest is padding), never
        fewer (the last would have pages and no rows).  Returns
        (slots, positions, cu): self.status says how many tokens found no
        page.  append() and attend() use this plan.  Tokens without a page are
        the last of their request; they are not in the cache, lens does not
        count them, and a later plan may bring them again."""
        device = self.codes.device
        with _on(stream, device):
            self.slots = torch.empty(tokens, dtype=torch.int32, device=device)
            self.positions = torch.empty(tokens, dtype=torch.int32, device=device)
        now, then = self._lens
        fk_kv_plan(now, new_lens, self.page_size, self.free_pages, self.free_count,
                   self.block_table, self._seq, self.cu, self.slots, self.positions,
                   self.free_count, self.status, ws=self._plan_ws, stream=stream, kept_lens=then)
        self._lens = [then, now]
        return self.slots, self.positions, self.cu

    def append(self, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        """Rows of the planned tokens, (tokens, kv_heads, head_dim)."""
        if self.slots is not None and not self.slots.numel() and not len(k) and not len(v):
            return                                    # a step without tokens
        fk_kv4_write(k, v, self.slots, self.codebook, self.codes, self.scales, stream=stream)

    def attend(self, q: torch.Tensor, max_q: int, scale: float | None = None, causal: bool = True,
               window: int = 0, lse: torch.Tensor | None = None, ws: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
        """Attention of the planned tokens' queries (tokens, q_heads,
        head_dim) over their requests, the planned tokens among them."""
        with _on(stream, q.device):
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if not len(q):
            return out
        fk_kv4_attention(q, self.cu, self._seq, self.block_table, self.codebook, self.codes,
                         self.scales, out, max_q, scale=scale, causal=causal, window=window,
                         lse=lse, ws=ws, stream=stream)
        return out

    def release(self, rows, keep=None, stream=None) -> None:
        """Shortens these rows of the table (integers, on the GPU; one named
        twice counts once, one that is none not at all) to their first `keep`
        tokens, a number or a tensor of one for each row, and returns the
        pages that hold none of them to the list.  None: no token is kept, the request is
        over.  Drafts that were rejected are taken back this way; the lengths
        are not to be lowered by hand, since the pages would be lost."""
        with _on(stream, self.codes.device):
            self._release(rows, keep)

    def _release(self, rows, keep) -> None:
        table, lens, (R, M) = self.block_table, self.lens, self.block_table.shape
        ints = dict(dtype=torch.int64, device=table.device)
        rows = torch.as_tensor(rows, device=table.device)
        if rows.dtype is torch.bool:
            rows = torch.where(rows, torch.arange(R, **ints), R)
        rows = torch.where(rows < 0, rows + R, rows).long()
        rows = torch.where((rows >= 0) & (rows < R), rows, R)        # R: none of them
        n = rows.numel()
        if not isinstance(keep, torch.Tensor):                       # filled there: a copy would wait
            keep = lens.new_full((n,), max(0, keep or 0))
        keep = keep.int().clamp(min=0).expand(n)
        left = torch.cat((lens, lens.new_zeros(1))).scatter_reduce_(0, rows, keep, "amin")
        turn = torch.arange(n, **ints)
        first = torch.full((R + 1,), n, **ints).scatter_reduce_(0, rows, turn, "amin")[rows] == turn
        row, page = rows.clamp(max=R - 1), torch.arange(M, **ints)
        entries, P = table[row], self.page_size
        mine = (first & (rows < R))[:, None] & (page >= ((left[rows] + P - 1) // P)[:, None])
        mine &= (page < ((lens[row] + P - 1) // P)[:, None]) & (entries >= 0)
        # where each returned page goes; entries that are not go to a place past the list
        at = self.free_count + mine.flatten().cumsum(0) - 1
        pages = self.free_pages.numel()
        longer = torch.cat((self.free_pages, self.free_pages.new_empty(1)))
        longer[torch.where(mine.flatten(), at, pages)] = entries.flatten()
        self.free_pages.copy_(longer[:pages])
        self.free_count += mine.sum().int()
        # a row named twice writes each entry as it is and as -1: the lesser stays
        table.view(-1).scatter_reduce_(0, (row[:, None] * M + page).flatten(),
                                       torch.where(mine, -1, entries).flatten(), "amin")
        self._seq.copy_(torch.where(left[:R] < lens, left[:R], self._seq))
        lens.copy_(left[:R])
