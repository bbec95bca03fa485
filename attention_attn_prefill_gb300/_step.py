"""Binding of the serving step: tables from request lengths, query/key norm with rotation, the 4-bit
paged cache and attention over it.

As in ``_lib``, these wrappers check shapes, types and devices, allocate what is not given and pass raw
pointers.  A call runs on the device its tensors live on, on that device's current stream unless
``stream`` is given; what it allocates for another stream is recorded there.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from ._lib import PAGE_TOKENS, _check, lib

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


def _ptr(t: torch.Tensor, dtype, name: str, device) -> int:
    """Pointer of a dense tensor on the call's device."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device(t, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _rows(t: torch.Tensor, name: str, device) -> tuple[int, int]:
    """(pointer, token stride) of bf16 rows [T, H, d] whose heads are dense."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    T, H, d = t.shape
    token, head, channel = t.stride()
    if channel != 1 or (head != d and H > 1):
        raise ValueError(f"the heads of a token of {name} must be dense")
    return t.data_ptr(), token if T > 1 else H * d


def _run(fn: str, device, stream, args, made=()) -> None:
    """Calls the C entry point with the stream appended, with `device` current."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _run(fn, device, stream, args, made)
    if stream is None:
        handle = torch.cuda.current_stream(device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    _check(getattr(lib(), fn)(*args, handle), fn)
    if stream is not None:
        # memory allocated here belongs to the current stream: it may not be reused before `stream` is done
        on = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(handle, device=device)
        for t in made:
            t.record_stream(on)


class StepTables(NamedTuple):
    seq_lens: torch.Tensor    # [N] int32
    cu_seqlens: torch.Tensor  # [N + 1] int32
    positions: torch.Tensor   # [num_tokens] int32
    slots: torch.Tensor       # [num_tokens] int32, -1 behind the last request
    pages_used: torch.Tensor  # [1] int32


def step_tables(cached_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                block_table: torch.Tensor, num_tokens: int, num_blocks: int, out: StepTables | None = None,
                stream=None) -> StepTables:
    """Tables of one serving step from request lengths [N]; `block_table` [N, max_blocks] is extended in
    place by pages from the front of `free_pages`.  All int32.  `num_tokens` >= sum(new_lens)."""
    device = _device(cached_lens, "cached_lens")
    N = cached_lens.numel()
    if cached_lens.dim() != 1 or new_lens.shape != (N,) or free_pages.dim() != 1:
        raise ValueError("cached_lens and new_lens must be [N], free_pages [num_free]")
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError("block_table must be [N, max_blocks]")
    made = ()
    if out is None:
        buf = torch.empty(2 * num_tokens + 2 * N + 2, dtype=_I32, device=device)  # one allocation for all five
        out = StepTables(*buf.split([N, N + 1, num_tokens, num_tokens, 1]))
        made = (buf,)
    elif [t.shape for t in out] != [(N,), (N + 1,), (num_tokens,), (num_tokens,), (1,)]:
        raise ValueError("out must have the shapes of StepTables for these lengths")
    args = [_ptr(cached_lens, _I32, "cached_lens", device), _ptr(new_lens, _I32, "new_lens", device),
            _ptr(free_pages, _I32, "free_pages", device), _ptr(block_table, _I32, "block_table", device),
            *(_ptr(t, _I32, "out", device) for t in out), N, int(num_tokens), free_pages.numel(), PAGE_TOKENS,
            block_table.shape[1], int(num_blocks)]
    _run("attn_step_tables", device, stream, args, made)
    return out


def rope_table(max_positions: int, rot: int, theta: float = 10000.0, device=None, stream=None) -> torch.Tensor:
    """Rotation table [max_positions, rot] f32 for qk_norm_rope (cosines, then sines; angles in double)."""
    device = torch.device("cuda") if device is None else torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    table = torch.empty((max_positions, rot), dtype=_F32, device=device)
    _run("attn_rope_table", device, stream, [table.data_ptr(), int(max_positions), int(rot), float(theta)], (table,))
    return table


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor | None, table: torch.Tensor | None,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, v: torch.Tensor | None = None, k_cache: torch.Tensor | None = None,
                 v_cache: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """RMS norm of each head of q [T,Hq,d] and k [T,Hkv,d] (with a weight [d]) and rotation of the first
    table.shape[1] channels, one pass -> (q_out, k_out).

    q, k and v may be views of one projection's output (heads dense, any token stride that is a multiple
    of 8).  With k_cache and v_cache [num_blocks,16,Hkv,d], v and slots [T], K and V are written to the
    paged cache as well; k_out is then None unless given.  q_out and k_out may be q and k themselves.
    """
    device = _device(q, "q")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, d):
        raise ValueError("k must be [T, Hkv, d] matching q")
    paged = k_cache is not None or v_cache is not None
    made = []
    if q_out is None:
        q_out = torch.empty((T, Hq, d), dtype=_BF16, device=device)
        made.append(q_out)
    if k_out is None and not paged:
        k_out = torch.empty((T, Hkv, d), dtype=_BF16, device=device)
        made.append(k_out)
    if q_out.shape != q.shape or (k_out is not None and k_out.shape != k.shape):
        raise ValueError("q_out and k_out must have the shapes of q and k")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and w.shape != (d,):
            raise ValueError(f"{name} must be [d]")
    rot = max_positions = 0
    if table is not None:
        if table.dim() != 2 or positions is None or positions.shape != (T,):
            raise ValueError("table must be [max_positions, rot] and positions [T]")
        max_positions, rot = table.shape
    num_blocks, page = 0, PAGE_TOKENS
    vp = (None, 0)
    if paged:
        if v is None or slots is None or k_cache is None or v_cache is None:
            raise ValueError("writing to a cache takes v, slots, k_cache and v_cache")
        num_blocks, page = k_cache.shape[:2]
        if k_cache.shape != (num_blocks, page, Hkv, d) or v_cache.shape != k_cache.shape:
            raise ValueError("caches must be [num_blocks, page, Hkv, d] matching k")
        if v.shape != k.shape or slots.shape != (T,):
            raise ValueError("v must have the shape of k and slots be [T]")
        vp = _rows(v, "v", device)
    args = [*_rows(q, "q", device), *_rows(k, "k", device), *vp,
            None if q_weight is None else _ptr(q_weight, _BF16, "q_weight", device),
            None if k_weight is None else _ptr(k_weight, _BF16, "k_weight", device), float(eps),
            None if table is None else _ptr(positions, _I32, "positions", device),
            None if table is None else _ptr(table, _F32, "table", device), max_positions, rot,
            1 if interleaved else 0, *_rows(q_out, "q_out", device),
            *((None, 0) if k_out is None else _rows(k_out, "k_out", device)),
            *((_ptr(k_cache, _BF16, "k_cache", device), _ptr(v_cache, _BF16, "v_cache", device),
               _ptr(slots, _I32, "slots", device)) if paged else (None, None, None)),
            T, Hq, Hkv, d, page, num_blocks]
    _run("attn_qk_norm_rope", device, stream, args, made)
    return q_out, k_out


def cache_q4_empty(num_blocks: int, Hkv: int, d: int, device=None) -> torch.Tensor:
    """A 4-bit paged cache [num_blocks, Hkv, 17 d] uint8 (zeroed: every value reads back as 0)."""
    size = int(lib().attn_cache_q4_record_bytes(d))
    if size == 0:
        raise ValueError("d must be 64, 128 or 256")
    return torch.zeros((num_blocks, Hkv, size), dtype=_U8, device="cuda" if device is None else device)


def _cache(cache: torch.Tensor, d: int, device) -> tuple[int, int, int]:
    """(pointer, num_blocks, Hkv) of a 4-bit cache."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3 or cache.shape[2] != 17 * d:
        raise ValueError("cache must be [num_blocks, Hkv, 17 d]")
    return _ptr(cache, _U8, "cache", device), cache.shape[0], cache.shape[1]


def cache_append_q4(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, stream=None) -> None:
    """Writes k, v [T,Hkv,d] bf16 (heads dense, any token stride that is a multiple of 8) into the 4-bit
    cache at slots [T] int32 (negative: not written)."""
    device = _device(cache, "cache")
    T, Hkv, d = k.shape
    ptr, num_blocks, heads = _cache(cache, d, device)
    if heads != Hkv or v.shape != k.shape or slots.shape != (T,):
        raise ValueError("k and v must be [T, Hkv, d] with the cache's Hkv, and slots [T]")
    args = [*_rows(k, "k", device), *_rows(v, "v", device), _ptr(slots, _I32, "slots", device), ptr, T, Hkv, d,
            PAGE_TOKENS, num_blocks]
    _run("attn_cache_append_q4", device, stream, args)


def _paged(cache, block_table, seq_lens, d, device):
    ptr, num_blocks, Hkv = _cache(cache, d, device)
    N = seq_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != N or seq_lens.dim() != 1:
        raise ValueError("block_table must be [N, max_blocks] and seq_lens [N]")
    return (ptr, _ptr(block_table, _I32, "block_table", device), _ptr(seq_lens, _I32, "seq_lens", device), N, Hkv,
            block_table.shape[1], num_blocks)


def cache_gather_q4(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """Reads sequences back: (k, v) [N, max_blocks * 16, Hkv, d] bf16; rows behind a sequence's end are
    left as they were (uninitialised if allocated here)."""
    device = _device(cache, "cache")
    if cache.dim() != 3 or cache.shape[2] % 17:
        raise ValueError("cache must be [num_blocks, Hkv, 17 d]")
    d = cache.shape[2] // 17
    cp, bt, sl, N, Hkv, max_blocks, num_blocks = _paged(cache, block_table, seq_lens, d, device)
    shape = (N, max_blocks * PAGE_TOKENS, Hkv, d)
    made = []
    if k_out is None:
        k_out = torch.empty(shape, dtype=_BF16, device=device)
        made.append(k_out)
    if v_out is None:
        v_out = torch.empty(shape, dtype=_BF16, device=device)
        made.append(v_out)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError("k_out and v_out must be [N, max_blocks * 16, Hkv, d]")
    args = [cp, bt, sl, _ptr(k_out, _BF16, "k_out", device), _ptr(v_out, _BF16, "v_out", device), N, Hkv, d,
            PAGE_TOKENS, max_blocks, num_blocks]
    _run("attn_cache_gather_q4", device, stream, args, made)
    return k_out, v_out


_decode_ws: dict[tuple[int, int], int] = {}


def decode_q4_workspace_bytes(d: int, device=None) -> int:
    """Bytes of workspace decode_paged_q4 needs on a device (the current one if not given)."""
    index = torch.cuda.current_device() if device is None or device.index is None else device.index
    if (index, d) not in _decode_ws:
        with torch.cuda.device(index):
            _decode_ws[index, d] = int(lib().attn_decode_q4_workspace_bytes(d))
    return _decode_ws[index, d]


def decode_paged_q4(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    return_lse: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """Single-token attention over the 4-bit cache: q [N,Hq,d] bf16 -> (o [N,Hq,d], lse [N,Hq])."""
    device = _device(q, "q")
    N, Hq, d = q.shape
    cp, bt, sl, num_seqs, Hkv, max_blocks, num_blocks = _paged(cache, block_table, seq_lens, d, device)
    if num_seqs != N:
        raise ValueError("seq_lens must be [N] matching q")
    made = []
    if out is None:
        out = torch.empty((N, Hq, d), dtype=_BF16, device=device)
        made.append(out)
    if lse is None and return_lse:
        lse = torch.empty((N, Hq), dtype=_F32, device=device)
        made.append(lse)
    if out.shape != q.shape or (lse is not None and lse.shape != (N, Hq)):
        raise ValueError("out must be [N, Hq, d] and lse [N, Hq]")
    if workspace is None:
        workspace = torch.empty(decode_q4_workspace_bytes(d, device), dtype=_U8, device=device)
        made.append(workspace)
    args = [_ptr(q, _BF16, "q", device), cp, bt, sl, _ptr(out, _BF16, "out", device),
            None if lse is None else _ptr(lse, _F32, "lse", device), N, Hq, Hkv, d, PAGE_TOKENS, max_blocks,
            num_blocks, 1.0 / math.sqrt(d) if scale is None else float(scale),
            _ptr(workspace, _U8, "workspace", device), workspace.numel()]
    _run("attn_decode_paged_q4", device, stream, args, made)
    return out, lse


def prefill_q4_workspace_bytes(num_seqs: int, Hkv: int, d: int, max_blocks: int) -> int:
    return int(lib().attn_prefill_q4_workspace_bytes(num_seqs, Hkv, d, max_blocks))


def prefill_paged_q4(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                     seq_lens: torch.Tensor, max_seqlen_q: int, scale: float | None = None, causal: bool = True,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = True,
                     workspace: torch.Tensor | None = None, stream=None):
    """Chunked prefill over the 4-bit cache: new tokens q [T,Hq,d] (their K/V already appended) against
    all cached tokens of their sequences -> (o [T,Hq,d], lse [Hq,T])."""
    device = _device(q, "q")
    T, Hq, d = q.shape
    cp, bt, sl, N, Hkv, max_blocks, num_blocks = _paged(cache, block_table, seq_lens, d, device)
    if cu_seqlens_q.shape != (N + 1,):
        raise ValueError("cu_seqlens_q must be [N + 1]")
    made = []
    if out is None:
        out = torch.empty((T, Hq, d), dtype=_BF16, device=device)
        made.append(out)
    if lse is None and return_lse:
        lse = torch.empty((Hq, T), dtype=_F32, device=device)
        made.append(lse)
    if out.shape != q.shape or (lse is not None and lse.shape != (Hq, T)):
        raise ValueError("out must be [T, Hq, d] and lse [Hq, T]")
    if workspace is None:
        workspace = torch.empty(max(1, prefill_q4_workspace_bytes(N, Hkv, d, max_blocks)), dtype=_U8, device=device)
        made.append(workspace)
    args = [_ptr(q, _BF16, "q", device), cp, bt, _ptr(cu_seqlens_q, _I32, "cu_seqlens_q", device), sl,
            _ptr(out, _BF16, "out", device), None if lse is None else _ptr(lse, _F32, "lse", device), N,
            int(max_seqlen_q), T, Hq, Hkv, d, PAGE_TOKENS, max_blocks, num_blocks,
            1.0 / math.sqrt(d) if scale is None else float(scale), 1 if causal else 0,
            _ptr(workspace, _U8, "workspace", device), workspace.numel()]
    _run("attn_prefill_paged_q4", device, stream, args, made)
    return out, lse
