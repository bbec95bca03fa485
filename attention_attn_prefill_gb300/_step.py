"""Binding of the serving step: tables from request lengths, query/key norm with rotation, the 4-bit
paged cache and attention over it.

As in ``_lib``, these wrappers check shapes, types and devices, allocate what is not given and pass raw
pointers.  A call runs on the device its tensors live on, on that device's current stream unless
``stream`` is given (what that asks of the caller, and where a call's own memory then comes from, is as
in ``_lib``).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._lib import PAGE_TOKENS, _check, _empty_on, _stream_handle, lib

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


# A call here takes a few microseconds on the GPU, about what the interpreter needs for it, so the checks
# are one expression a call over the tensors that were given; _explain finds which of them failed.
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream().cuda_stream without the Stream object
_current_device = torch._C._cuda_getDevice
_entry = {}


def _explain(dev: int, *tensors) -> None:
    """Raises for the first of (tensor, dtype, name) that is not a dense tensor of its type on the call's device."""
    for t, dtype, name in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor")
        if dev < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{tensors[0][2]} has another shape or device than the call needs")


def _stride(t: torch.Tensor, name: str, dev: int) -> int:
    """Token stride of bf16 rows [T, H, d] whose heads are dense."""
    if t.dtype is not _BF16 or t.get_device() != dev:
        _explain(dev, (t, _BF16, name))
    T, H, d = t.shape
    token, head, channel = t.stride()
    if channel != 1 or (head != d and H > 1):
        raise ValueError(f"the heads of a token of {name} must be dense")
    return token if T > 1 else H * d


def _run(fn: str, dev: int, stream, *args) -> None:
    """Calls the C entry point with the stream appended, with device `dev` current."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _run(fn, dev, stream, *args)
    call = _entry.get(fn)
    if call is None:
        call = _entry[fn] = getattr(lib(), fn)
    status = call(*args, _raw_stream(dev) if stream is None else _stream_handle(stream))
    if status:
        _check(status, fn)


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
    place by pages from the front of `free_pages`.  All int32.  `num_tokens` >= sum(new_lens).  `out` takes
    the results in given tensors, none of which may overlap an input (seq_lens is not cached_lens)."""
    dev, N = cached_lens.get_device(), cached_lens.numel()
    if (dev < 0 or new_lens.get_device() != dev or free_pages.get_device() != dev or block_table.get_device() != dev
            or cached_lens.dtype is not _I32 or new_lens.dtype is not _I32 or free_pages.dtype is not _I32
            or block_table.dtype is not _I32 or not cached_lens.is_contiguous() or not new_lens.is_contiguous()
            or not free_pages.is_contiguous() or not block_table.is_contiguous()):
        _explain(dev, (cached_lens, _I32, "cached_lens"), (new_lens, _I32, "new_lens"),
                 (free_pages, _I32, "free_pages"), (block_table, _I32, "block_table"))
    if cached_lens.dim() != 1 or new_lens.shape != (N,) or free_pages.dim() != 1:
        raise ValueError("cached_lens and new_lens must be [N], free_pages [num_free]")
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError("block_table must be [N, max_blocks]")
    if out is None:
        made = _empty_on(2 * (num_tokens + N + 1), _I32, dev, stream)  # one allocation for all five
        sl = made.data_ptr()
        cu, pos = sl + 4 * N, sl + 4 * (2 * N + 1)
        slots = pos + 4 * num_tokens
        used = slots + 4 * num_tokens
        out = StepTables(*torch.unsafe_split_with_sizes(made, (N, N + 1, num_tokens, num_tokens, 1)))
    else:
        if [t.shape for t in out] != [(N,), (N + 1,), (num_tokens,), (num_tokens,), (1,)]:
            raise ValueError("out must have the shapes of StepTables for these lengths")
        if any(t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous() for t in out):
            _explain(dev, *((t, _I32, "out") for t in out))
        sl, cu, pos, slots, used = (t.data_ptr() for t in out)
    _run("attn_step_tables", dev, stream, cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
         block_table.data_ptr(), sl, cu, pos, slots, used, N, num_tokens, free_pages.numel(), PAGE_TOKENS,
         block_table.shape[1], num_blocks)
    return out


def _cuda_index(device) -> int:
    """Index of a CUDA device given as an index, a name, a torch device or None (the current one)."""
    if isinstance(device, int):
        return device
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"device must be a CUDA device, got {device}")
    return torch.cuda.current_device() if device.index is None else device.index


def rope_table(max_positions: int, rot: int, theta: float = 10000.0, device=None, stream=None) -> torch.Tensor:
    """Rotation table [max_positions, rot] f32 for qk_norm_rope (cosines, then sines; angles in double)."""
    dev = _cuda_index(device)
    table = _empty_on((max_positions, rot), _F32, dev, stream)
    _run("attn_rope_table", dev, stream, table.data_ptr(), max_positions, rot, float(theta))
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
    dev = q.get_device()
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    qs, ks = _stride(q, "q", dev), _stride(k, "k", dev)
    if dev < 0 or k.shape != (T, Hkv, d):
        raise ValueError("q must be a CUDA tensor [T, Hq, d] and k [T, Hkv, d]")
    paged = k_cache is not None or v_cache is not None
    if q_out is None:
        q_out, qos = _empty_on((T, Hq, d), _BF16, dev, stream), Hq * d
    else:
        qos = _stride(q_out, "q_out", dev)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
    kop = kos = 0
    if k_out is None and not paged:
        k_out, kos = _empty_on((T, Hkv, d), _BF16, dev, stream), Hkv * d
        kop = k_out.data_ptr()
    elif k_out is not None:
        kop, kos = k_out.data_ptr(), _stride(k_out, "k_out", dev)
        if k_out.shape != k.shape:
            raise ValueError("k_out must have the shape of k")
    qwp = kwp = 0
    if q_weight is not None:
        if q_weight.dtype is not _BF16 or q_weight.get_device() != dev or not q_weight.is_contiguous():
            _explain(dev, (q_weight, _BF16, "q_weight"))
        if q_weight.shape != (d,):
            raise ValueError("q_weight must be [d]")
        qwp = q_weight.data_ptr()
    if k_weight is not None:
        if k_weight.dtype is not _BF16 or k_weight.get_device() != dev or not k_weight.is_contiguous():
            _explain(dev, (k_weight, _BF16, "k_weight"))
        if k_weight.shape != (d,):
            raise ValueError("k_weight must be [d]")
        kwp = k_weight.data_ptr()
    rot = max_positions = pp = tp = 0
    if table is not None:
        if table.dim() != 2 or positions is None or positions.shape != (T,):
            raise ValueError("table must be [max_positions, rot] and positions [T]")
        if (positions.dtype is not _I32 or table.dtype is not _F32 or positions.get_device() != dev
                or table.get_device() != dev or not positions.is_contiguous() or not table.is_contiguous()):
            _explain(dev, (positions, _I32, "positions"), (table, _F32, "table"))
        max_positions, rot = table.shape
        pp, tp = positions.data_ptr(), table.data_ptr()
    num_blocks, page = 0, PAGE_TOKENS
    vptr = vs = kcp = vcp = sp = 0
    if paged:
        if v is None or slots is None or k_cache is None or v_cache is None:
            raise ValueError("writing to a cache takes v, slots, k_cache and v_cache")
        num_blocks, page = k_cache.shape[:2]
        if k_cache.shape != (num_blocks, page, Hkv, d) or v_cache.shape != k_cache.shape:
            raise ValueError("caches must be [num_blocks, page, Hkv, d] matching k")
        if v.shape != k.shape or slots.shape != (T,):
            raise ValueError("v must have the shape of k and slots be [T]")
        vptr, vs = v.data_ptr(), _stride(v, "v", dev)
        if (slots.dtype is not _I32 or k_cache.dtype is not _BF16 or v_cache.dtype is not _BF16
                or slots.get_device() != dev or k_cache.get_device() != dev or v_cache.get_device() != dev
                or not slots.is_contiguous() or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
            _explain(dev, (k_cache, _BF16, "k_cache"), (v_cache, _BF16, "v_cache"), (slots, _I32, "slots"))
        kcp, vcp, sp = k_cache.data_ptr(), v_cache.data_ptr(), slots.data_ptr()
    if T == 0:  # a step without tokens
        return q_out, k_out
    _run("attn_qk_norm_rope", dev, stream, q.data_ptr(), qs, k.data_ptr(), ks, vptr, vs, qwp, kwp, eps, pp, tp,
         max_positions, rot, 1 if interleaved else 0, q_out.data_ptr(), qos, kop, kos, kcp, vcp, sp, T, Hq, Hkv, d,
         page, num_blocks)
    return q_out, k_out


def cache_q4_empty(num_blocks: int, Hkv: int, d: int, device=None) -> torch.Tensor:
    """A 4-bit paged cache [num_blocks, Hkv, 17 d] uint8 (zeroed: every value reads back as 0)."""
    size = int(lib().attn_cache_q4_record_bytes(d))
    if size == 0:
        raise ValueError("d must be 64, 128 or 256")
    return torch.zeros((num_blocks, Hkv, size), dtype=_U8, device="cuda" if device is None else device)


def cache_append_q4(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, stream=None) -> None:
    """Writes k, v [T,Hkv,d] bf16 (heads dense, any token stride that is a multiple of 8) into the 4-bit
    cache at slots [T] int32 (negative: not written)."""
    dev = cache.get_device()
    if (dev < 0 or cache.dtype is not _U8 or slots.dtype is not _I32 or slots.get_device() != dev
            or not cache.is_contiguous() or not slots.is_contiguous()):
        _explain(dev, (cache, _U8, "cache"), (slots, _I32, "slots"))
    T, Hkv, d = k.shape
    if cache.dim() != 3 or cache.shape[1:] != (Hkv, 17 * d):
        raise ValueError("cache must be [num_blocks, Hkv, 17 d] matching k")
    if v.shape != k.shape or slots.shape != (T,):
        raise ValueError("k and v must be [T, Hkv, d] and slots [T]")
    ks, vs = _stride(k, "k", dev), _stride(v, "v", dev)
    if T == 0:  # a step without tokens
        return
    _run("attn_cache_append_q4", dev, stream, k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(), cache.data_ptr(),
         T, Hkv, d, PAGE_TOKENS, cache.shape[0])


def _check_paged(dev, d, cache, block_table, seq_lens, N):
    """(num_blocks, Hkv, max_blocks) of a 4-bit cache and the tables that address it."""
    if (dev < 0 or cache.dtype is not _U8 or block_table.dtype is not _I32 or seq_lens.dtype is not _I32
            or cache.get_device() != dev or block_table.get_device() != dev or seq_lens.get_device() != dev
            or not cache.is_contiguous() or not block_table.is_contiguous() or not seq_lens.is_contiguous()):
        _explain(dev, (cache, _U8, "cache"), (block_table, _I32, "block_table"), (seq_lens, _I32, "seq_lens"))
    if cache.dim() != 3 or cache.shape[2] != 17 * d:
        raise ValueError("cache must be [num_blocks, Hkv, 17 d]")
    if block_table.dim() != 2 or block_table.shape[0] != N or seq_lens.shape != (N,):
        raise ValueError("block_table must be [N, max_blocks] and seq_lens [N]")
    num_blocks, Hkv, _ = cache.shape
    return num_blocks, Hkv, block_table.shape[1]


def cache_gather_q4(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """Reads sequences back: (k, v) [N, max_blocks * 16, Hkv, d] bf16; rows behind a sequence's end are
    left as they were (uninitialised if allocated here)."""
    dev, N = cache.get_device(), seq_lens.numel()
    d = cache.shape[-1] // 17
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
    _run("attn_cache_gather_q4", dev, stream, cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
         k_out.data_ptr(), v_out.data_ptr(), N, Hkv, d, PAGE_TOKENS, max_blocks, num_blocks)
    return k_out, v_out


def _outputs(dev, q, out, lse, lse_shape, return_lse, workspace, need, stream):
    """(out, lse, workspace), allocated where not given."""
    if out is None:
        out = _empty_on(q.shape, _BF16, dev, stream)
    elif out.shape != q.shape or out.dtype is not _BF16 or out.get_device() != dev or not out.is_contiguous():
        _explain(dev, (out, _BF16, "out (of q's shape)"))
    if lse is not None:
        if lse.shape != lse_shape or lse.dtype is not _F32 or lse.get_device() != dev or not lse.is_contiguous():
            _explain(dev, (lse, _F32, f"lse (of shape {list(lse_shape)})"))
    elif return_lse:
        lse = _empty_on(lse_shape, _F32, dev, stream)
    if workspace is None:
        workspace = _empty_on(need, _U8, dev, stream, returned=False)
    elif workspace.dtype is not _U8 or workspace.get_device() != dev or not workspace.is_contiguous():
        _explain(dev, (workspace, _U8, "workspace"))
    return out, lse, workspace


_decode_ws: dict[tuple[int, int], int] = {}


def decode_q4_workspace_bytes(d: int, device=None) -> int:
    """Bytes of workspace decode_paged_q4 needs on a device (the current one if not given)."""
    index = _cuda_index(device)
    if (index, d) not in _decode_ws:
        with torch.cuda.device(index):
            _decode_ws[index, d] = int(lib().attn_decode_q4_workspace_bytes(d))
    return _decode_ws[index, d]


def decode_paged_q4(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    return_lse: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """Single-token attention over the 4-bit cache: q [N,Hq,d] bf16 -> (o [N,Hq,d], lse [N,Hq])."""
    dev = q.get_device()
    N, Hq, d = q.shape
    num_blocks, Hkv, max_blocks = _check_paged(dev, d, cache, block_table, seq_lens, N)
    if q.dtype is not _BF16 or not q.is_contiguous():
        _explain(dev, (q, _BF16, "q"))
    out, lse, workspace = _outputs(dev, q, out, lse, (N, Hq), return_lse, workspace,
                                   _decode_ws.get((dev, d)) or decode_q4_workspace_bytes(d, dev), stream)
    _run("attn_decode_paged_q4", dev, stream, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(),
         seq_lens.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), N, Hq, Hkv, d, PAGE_TOKENS,
         max_blocks, num_blocks, d ** -0.5 if scale is None else scale, workspace.data_ptr(), workspace.numel())
    return out, lse


def prefill_q4_workspace_bytes(num_seqs: int, Hkv: int, d: int, max_blocks: int) -> int:
    return int(lib().attn_prefill_q4_workspace_bytes(num_seqs, Hkv, d, max_blocks))


def prefill_paged_q4(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                     seq_lens: torch.Tensor, max_seqlen_q: int, scale: float | None = None, causal: bool = True,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = True,
                     workspace: torch.Tensor | None = None, stream=None):
    """Chunked prefill over the 4-bit cache: new tokens q [T,Hq,d] (their K/V already appended) against
    all cached tokens of their sequences -> (o [T,Hq,d], lse [Hq,T]).

    The workspace holds N * max_blocks pages as bf16: pass block_table[:, :pages].contiguous() where the
    table is much wider than the longest sequence needs."""
    dev, N = q.get_device(), seq_lens.numel()
    T, Hq, d = q.shape
    num_blocks, Hkv, max_blocks = _check_paged(dev, d, cache, block_table, seq_lens, N)
    if q.dtype is not _BF16 or not q.is_contiguous():
        _explain(dev, (q, _BF16, "q"))
    if cu_seqlens_q.dtype is not _I32 or cu_seqlens_q.get_device() != dev or not cu_seqlens_q.is_contiguous():
        _explain(dev, (cu_seqlens_q, _I32, "cu_seqlens_q"))
    if cu_seqlens_q.shape != (N + 1,):
        raise ValueError("cu_seqlens_q must be [N + 1]")
    out, lse, workspace = _outputs(dev, q, out, lse, (Hq, T), return_lse, workspace,
                                   max(1, prefill_q4_workspace_bytes(N, Hkv, d, max_blocks)), stream)
    if T == 0:  # a step without tokens
        return out, lse
    _run("attn_prefill_paged_q4", dev, stream, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(),
         cu_seqlens_q.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), N,
         max_seqlen_q, T, Hq, Hkv, d, PAGE_TOKENS, max_blocks, num_blocks, d ** -0.5 if scale is None else scale,
         1 if causal else 0, workspace.data_ptr(), workspace.numel())
    return out, lse
