"""Binding of the 8-bit paged cache, attention over it, and the selection of the blocks a query attends to.

As in ``_step``: these wrappers check shapes, types and devices, allocate what is not given and pass raw pointers, on
the device their tensors live on and its current stream unless ``stream`` is given.
"""
from __future__ import annotations

import torch

from ._lib import PAGE_TOKENS, _empty_on, lib
from ._step import _BF16, _I32, _U8, _cuda_index, _explain, _outputs, _run, _stride

RECORD_TAIL = 16  # bytes of a record behind its 32 d codes


def cache_f8_empty(num_blocks: int, Hkv: int, d: int, device=None) -> torch.Tensor:
    """An 8-bit paged cache [num_blocks, Hkv, 32 d + 16] uint8 (zeroed: every value reads back as 0)."""
    size = int(lib().attn_cache_f8_record_bytes(d))
    if size == 0:
        raise ValueError("d must be 64, 128 or 256")
    return torch.zeros((num_blocks, Hkv, size), dtype=_U8, device="cuda" if device is None else device)


def key_bounds_empty(num_blocks: int, Hkv: int, d: int, device=None) -> torch.Tensor:
    """Key bounds of a cache's pages [num_blocks, Hkv, 2, d] bf16 (zeroed), for cache_append_f8 and select_blocks."""
    if int(lib().attn_cache_f8_record_bytes(d)) == 0:
        raise ValueError("d must be 64, 128 or 256")
    return torch.zeros((num_blocks, Hkv, 2, d), dtype=_BF16, device="cuda" if device is None else device)


def cache_append_f8(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
                    bounds: torch.Tensor | None = None, stream=None) -> None:
    """Writes k, v [T,Hkv,d] bf16 (heads dense, any token stride that is a multiple of 8) into the 8-bit cache at
    slots [T] int32 (negative: not written), and keeps the pages' key bounds if given.

    A page's scale belongs to all its tokens: those of a call that go to one page stand next to each other with
    consecutive slots, as step_tables gives them.  Rows of the page before them stay, rows behind them are void."""
    dev = cache.get_device()
    if (dev < 0 or cache.dtype is not _U8 or slots.dtype is not _I32 or slots.get_device() != dev
            or not cache.is_contiguous() or not slots.is_contiguous()):
        _explain(dev, (cache, _U8, "cache"), (slots, _I32, "slots"))
    T, Hkv, d = k.shape
    if cache.dim() != 3 or cache.shape[1:] != (Hkv, 32 * d + RECORD_TAIL):
        raise ValueError("cache must be [num_blocks, Hkv, 32 d + 16] matching k")
    if v.shape != k.shape or slots.shape != (T,):
        raise ValueError("k and v must be [T, Hkv, d] and slots [T]")
    bp = 0
    if bounds is not None:
        if bounds.dtype is not _BF16 or bounds.get_device() != dev or not bounds.is_contiguous():
            _explain(dev, (bounds, _BF16, "bounds"))
        if bounds.shape != (cache.shape[0], Hkv, 2, d):
            raise ValueError("bounds must be [num_blocks, Hkv, 2, d] matching the cache")
        bp = bounds.data_ptr()
    ks, vs = _stride(k, "k", dev), _stride(v, "v", dev)
    if T == 0:  # a step without tokens
        return
    _run("attn_cache_append_f8", dev, stream, k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(), cache.data_ptr(),
         bp, T, Hkv, d, PAGE_TOKENS, cache.shape[0])


def _check_tables(dev, block_table, seq_lens, N):
    if (dev < 0 or block_table.dtype is not _I32 or seq_lens.dtype is not _I32 or block_table.get_device() != dev
            or seq_lens.get_device() != dev or not block_table.is_contiguous() or not seq_lens.is_contiguous()):
        _explain(dev, (block_table, _I32, "block_table"), (seq_lens, _I32, "seq_lens"))
    if block_table.dim() != 2 or block_table.shape[0] != N or seq_lens.shape != (N,):
        raise ValueError("block_table must be [N, max_blocks] and seq_lens [N]")


def _check_paged(dev, d, cache, block_table, seq_lens, N):
    """(num_blocks, Hkv, max_blocks) of an 8-bit cache and the tables that address it."""
    if dev < 0 or cache.dtype is not _U8 or cache.get_device() != dev or not cache.is_contiguous():
        _explain(dev, (cache, _U8, "cache"))
    if cache.dim() != 3 or cache.shape[2] != 32 * d + RECORD_TAIL:
        raise ValueError("cache must be [num_blocks, Hkv, 32 d + 16]")
    _check_tables(dev, block_table, seq_lens, N)
    num_blocks, Hkv, _ = cache.shape
    return num_blocks, Hkv, block_table.shape[1]


def _check_rows(dev, q, cu_seqlens_q, N):
    """Pointer of cu_seqlens_q [N + 1], or 0 where each sequence has one query row."""
    if q.dtype is not _BF16 or q.get_device() != dev or not q.is_contiguous():
        _explain(dev, (q, _BF16, "q"))
    if cu_seqlens_q is None:
        if q.shape[0] != N:
            raise ValueError("q must have a row for each sequence where cu_seqlens_q is not given")
        return 0
    if cu_seqlens_q.dtype is not _I32 or cu_seqlens_q.get_device() != dev or not cu_seqlens_q.is_contiguous():
        _explain(dev, (cu_seqlens_q, _I32, "cu_seqlens_q"))
    if cu_seqlens_q.shape != (N + 1,):
        raise ValueError("cu_seqlens_q must be [N + 1]")
    return cu_seqlens_q.data_ptr()


def cache_gather_f8(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """Reads sequences back: (k, v) [N, max_blocks * 16, Hkv, d] bf16; rows behind a sequence's end are
    left as they were (uninitialised if allocated here)."""
    dev, N = cache.get_device(), seq_lens.numel()
    d = (cache.shape[-1] - RECORD_TAIL) // 32
    num_blocks, Hkv, max_blocks = _check_paged(dev, d, cache, block_table, seq_lens, N)
    shape = (N, max_blocks * PAGE_TOKENS, Hkv, d)
    if k_out is None:
        k_out = _empty_on(shape, _BF16, dev, stream)
    if v_out is None:
        v_out = _empty_on(shape, _BF16, dev, stream)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError("k_out and v_out must be [N, max_blocks * 16, Hkv, d]")
    if (k_out.dtype is not _BF16 or v_out.dtype is not _BF16 or k_out.get_device() != dev
            or v_out.get_device() != dev or not k_out.is_contiguous() or not v_out.is_contiguous()):
        _explain(dev, (k_out, _BF16, "k_out"), (v_out, _BF16, "v_out"))
    if N == 0:  # a step without sequences
        return k_out, v_out
    _run("attn_cache_gather_f8", dev, stream, cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
         k_out.data_ptr(), v_out.data_ptr(), N, Hkv, d, PAGE_TOKENS, max_blocks, num_blocks)
    return k_out, v_out


_decode_ws: dict[tuple[int, int], int] = {}


def decode_f8_workspace_bytes(d: int, device=None) -> int:
    """Bytes of workspace decode_paged_f8 and decode_blocks_f8 need on a device (the current one if not given)."""
    index = _cuda_index(device)
    if (index, d) not in _decode_ws:
        with torch.cuda.device(index):
            _decode_ws[index, d] = int(lib().attn_decode_f8_workspace_bytes(d))
    return _decode_ws[index, d]


def decode_paged_f8(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    return_lse: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """Single-token attention over the 8-bit cache: q [N,Hq,d] bf16 -> (o [N,Hq,d], lse [N,Hq]).  Few short sequences are
    faster in a block table that is no wider than the longest of them needs."""
    dev = q.get_device()
    N, Hq, d = q.shape
    num_blocks, Hkv, max_blocks = _check_paged(dev, d, cache, block_table, seq_lens, N)
    if q.dtype is not _BF16 or not q.is_contiguous():
        _explain(dev, (q, _BF16, "q"))
    out, lse, workspace = _outputs(dev, q, out, lse, (N, Hq), return_lse, workspace,
                                   _decode_ws.get((dev, d)) or decode_f8_workspace_bytes(d, dev), stream)
    if N == 0:  # a step without sequences
        return out, lse
    _run("attn_decode_paged_f8", dev, stream, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(),
         seq_lens.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), N, Hq, Hkv, d, PAGE_TOKENS,
         max_blocks, num_blocks, d ** -0.5 if scale is None else scale, workspace.data_ptr(), workspace.numel())
    return out, lse


def decode_blocks_f8(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                     blocks: torch.Tensor, cu_seqlens_q: torch.Tensor | None = None, scale: float | None = None,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = True,
                     workspace: torch.Tensor | None = None, stream=None):
    """Attention of q [T,Hq,d] bf16 over the blocks [T,Hkv,K] int32 that each row and KV head names (select_blocks)
    -> (o [T,Hq,d], lse [T,Hq]).

    Row i of sequence n's rows cu_seqlens_q[n] .. (without it: row n) sees the tokens up to its own; the rows are
    the sequence's last tokens, appended before.  Negative entries are passed over.  Rows of q behind the last
    sequence are left as they were in out and lse."""
    dev, N = q.get_device(), seq_lens.numel()
    T, Hq, d = q.shape
    num_blocks, Hkv, max_blocks = _check_paged(dev, d, cache, block_table, seq_lens, N)
    cu = _check_rows(dev, q, cu_seqlens_q, N)
    if blocks.dtype is not _I32 or blocks.get_device() != dev or not blocks.is_contiguous():
        _explain(dev, (blocks, _I32, "blocks"))
    if blocks.dim() != 3 or blocks.shape[:2] != (T, Hkv):
        raise ValueError("blocks must be [T, Hkv, K]")
    out, lse, workspace = _outputs(dev, q, out, lse, (T, Hq), return_lse, workspace,
                                   _decode_ws.get((dev, d)) or decode_f8_workspace_bytes(d, dev), stream)
    if T == 0:  # a step without tokens
        return out, lse
    _run("attn_decode_blocks_f8", dev, stream, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), cu,
         seq_lens.data_ptr(), blocks.data_ptr(), blocks.shape[2], out.data_ptr(), 0 if lse is None else lse.data_ptr(),
         T, N, Hq, Hkv, d, PAGE_TOKENS, max_blocks, num_blocks, d ** -0.5 if scale is None else scale,
         workspace.data_ptr(), workspace.numel())
    return out, lse


def prefill_f8_workspace_bytes(num_seqs: int, Hkv: int, d: int, max_blocks: int) -> int:
    return int(lib().attn_prefill_f8_workspace_bytes(num_seqs, Hkv, d, max_blocks))


def prefill_paged_f8(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                     seq_lens: torch.Tensor, max_seqlen_q: int, scale: float | None = None, causal: bool = True,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = True,
                     workspace: torch.Tensor | None = None, stream=None):
    """Chunked prefill over the 8-bit cache: new tokens q [T,Hq,d] (their K/V already appended) against
    all cached tokens of their sequences -> (o [T,Hq,d], lse [Hq,T]).

    The workspace holds N * max_blocks pages as bf16: pass block_table[:, :pages].contiguous() where the
    table is much wider than the longest sequence needs."""
    dev, N = q.get_device(), seq_lens.numel()
    T, Hq, d = q.shape
    num_blocks, Hkv, max_blocks = _check_paged(dev, d, cache, block_table, seq_lens, N)
    if cu_seqlens_q is None:
        raise ValueError("cu_seqlens_q must be a tensor")
    cu = _check_rows(dev, q, cu_seqlens_q, N)
    out, lse, workspace = _outputs(dev, q, out, lse, (Hq, T), return_lse, workspace,
                                   max(1, prefill_f8_workspace_bytes(N, Hkv, d, max_blocks)), stream)
    if T == 0:  # a step without tokens
        return out, lse
    _run("attn_prefill_paged_f8", dev, stream, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), cu,
         seq_lens.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), N, max_seqlen_q, T, Hq, Hkv, d,
         PAGE_TOKENS, max_blocks, num_blocks, d ** -0.5 if scale is None else scale, 1 if causal else 0,
         workspace.data_ptr(), workspace.numel())
    return out, lse


def select_blocks_workspace_bytes(num_tokens: int, num_seqs: int, max_seqlen_q: int, Hkv: int, d: int,
                                  max_blocks: int) -> int:
    return int(lib().attn_select_blocks_workspace_bytes(num_tokens, num_seqs, max_seqlen_q, Hkv, d, max_blocks))


def select_blocks(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  num_selected: int, first: int = 1, last: int = 2, cu_seqlens_q: torch.Tensor | None = None,
                  max_seqlen_q: int | None = None, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Blocks [T,Hkv,num_selected] int32 that each row of q [T,Hq,d] bf16 and KV head is to attend to, ascending, -1
    behind: the first `first` and last `last` blocks that the row sees, and those whose key bounds
    [num_blocks,Hkv,2,d] allow the highest scores; all where there are no more than num_selected.

    cu_seqlens_q as for decode_blocks_f8, with at most max_seqlen_q rows a sequence (without it any number: a bound of
    up to four rows takes a faster way).  The workspace holds a score for each row, KV head and column of the table: 1.1 GB
    for a chunk of 4096 tokens over 131072 and 8 KV heads, so give a long chunk in parts, and
    block_table[:, :pages].contiguous() where the table is much wider than the longest sequence needs."""
    dev, N = q.get_device(), seq_lens.numel()
    T, Hq, d = q.shape
    if dev < 0 or bounds.dtype is not _BF16 or bounds.get_device() != dev or not bounds.is_contiguous():
        _explain(dev, (bounds, _BF16, "bounds"))
    if bounds.dim() != 4 or bounds.shape[2:] != (2, d):
        raise ValueError("bounds must be [num_blocks, Hkv, 2, d] matching q")
    num_blocks, Hkv = bounds.shape[:2]
    _check_tables(dev, block_table, seq_lens, N)
    cu = _check_rows(dev, q, cu_seqlens_q, N)
    if max_seqlen_q is None:
        max_seqlen_q = 1 if cu_seqlens_q is None else max(1, T)
    if out is None:
        out = _empty_on((T, Hkv, num_selected), _I32, dev, stream)
    elif (out.shape != (T, Hkv, num_selected) or out.dtype is not _I32 or out.get_device() != dev
          or not out.is_contiguous()):
        _explain(dev, (out, _I32, "out (of shape [T, Hkv, num_selected])"))
    if workspace is None:
        need = select_blocks_workspace_bytes(T, N, max_seqlen_q, Hkv, d, block_table.shape[1])
        workspace = _empty_on(max(1, need), _U8, dev, stream, returned=False)
    elif workspace.dtype is not _U8 or workspace.get_device() != dev or not workspace.is_contiguous():
        _explain(dev, (workspace, _U8, "workspace"))
    if T == 0:  # a step without tokens
        return out
    _run("attn_select_blocks", dev, stream, q.data_ptr(), bounds.data_ptr(), block_table.data_ptr(), cu,
         seq_lens.data_ptr(), out.data_ptr(), num_selected, first, last, T, N, max_seqlen_q, Hq, Hkv, d, PAGE_TOKENS,
         block_table.shape[1], num_blocks, workspace.data_ptr(), workspace.numel())
    return out
