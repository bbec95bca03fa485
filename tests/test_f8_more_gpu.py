"""The 8-bit cache and block selection where sizes, offsets, streams and shares make a difference.

Attention is compared with 64-bit sums over the values read back from the cache (which tests/test_f8_ops_gpu.py
compares with their definition), by that file's tolerance; selections with 64-bit scores, exactly.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.f8 as o8
from attention_attn_prefill_gb300._lib import _SIGNATURES
from test_streams_gpu import _busy_with_freed_blocks

pytestmark = pytest.mark.gpu
PAGE = 16


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _randn(shape, gen, dev):
    return torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)


def _setup(attn, dev, lens, Hkv, d, seed, width=None, blocks=None, first_page=0):
    """A cache of sequences on shuffled pages from `first_page` on, with its bounds, and the block table."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    need = [_pages(n) for n in lens]
    total = sum(need) + 2
    blocks = blocks or first_page + total
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32) + first_page
    table = torch.zeros((len(lens), width or max(max(need), 1)), dtype=torch.int32, device=dev)
    cache, bounds = attn.cache_f8_empty(blocks, Hkv, d, device=dev), attn.key_bounds_empty(blocks, Hkv, d, device=dev)
    slots, at = [], 0
    for n, length in enumerate(lens):
        table[n, :need[n]] = order[at:at + need[n]]
        t = torch.arange(length, device=dev)
        slots.append(table[n].long()[t // PAGE] * PAGE + t % PAGE)
        at += need[n]
    slots = torch.cat(slots).to(torch.int32)
    T = slots.numel()
    if T:
        attn.cache_append_f8(_randn((T, Hkv, d), gen, dev), _randn((T, Hkv, d), gen, dev), slots, cache, bounds=bounds)
    return gen, cache, bounds, table


def _exact(q, k, v, scale):
    """q [G, d], k, v [L, d] in 64 bits -> (o, lse, mean |p v|, largest sum |q k| scale)."""
    s = q @ k.T * scale
    p = torch.softmax(s, -1)
    return p @ v, torch.logsumexp(s, -1), p @ v.abs(), float((q.abs() @ k.abs().T).max() * scale) if k.shape[0] else 0.0


def _check_rows(o, lse, q, k, v, scale, d):
    wo, wl, mass, biggest = _exact(q.double(), k, v, scale)
    dot = (2 * d / 16 + 4) * 2.0 ** -22 * biggest
    tol = 2.0 ** -8 * wo.abs() + (2.0 ** -11 + 2 * (dot + 2.0 ** -16)) * mass + 2.0 ** -133
    err = (o.double() - wo).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse.double() - wl).abs() <= dot + 2.0 ** -16 + 2.0 ** -22 * wl.abs()).all()


def _values(attn, cache, table, lens, dev):
    k, v = attn.cache_gather_f8(cache, table, _i32(lens, dev))
    return k, v


# ---------------------------------------------------------------------------------------------- shares
@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ([20000], 4, 1, 128), ([20000, 9], 8, 4, 256), ([9000, 1, 250], 6, 2, 64), ([700, 20], 32, 2, 128),
    ([30000, 20001], 8, 2, 128), ([40000, 100, 30000], 16, 4, 64), ([9000] * 9, 8, 1, 128), ([333] * 40, 4, 2, 256),
    ([5] * 700, 2, 1, 64), ([(i * 271) % 199 for i in range(900)], 16, 2, 128),
    ([(i * 1543) % 4999 for i in range(9)], 18, 2, 128), ([122863, 6335], 16, 2, 256), ([17] * 300, 40, 8, 128),
])
def test_decode_in_many_shares(attn, gpu, lens, Hq, Hkv, d):
    """Sequences cut by shares, several in a share, more than a thread counts; and the same as listed blocks."""
    gen, cache, bounds, table = _setup(attn, gpu, lens, Hkv, d, seed=len(lens) + d)
    q = _randn((len(lens), Hq, d), gen, gpu)
    sl = _i32(lens, gpu)
    o, lse = attn.decode_paged_f8(q, cache, table, sl)
    width = table.shape[1]
    every = torch.arange(width, dtype=torch.int32, device=gpu).expand(len(lens), Hkv, width).contiguous()
    ob, lb = attn.decode_blocks_f8(q, cache, table, sl, every)
    G = Hq // Hkv
    for n, length in enumerate(lens):
        if length == 0:
            assert not o[n].any() and not ob[n].any() and (lse[n] == -math.inf).all() and (lb[n] == -math.inf).all()
            continue
        if len(lens) > 100 and n % 17:
            continue
        k, v = (x[0, :length].double() for x in _values(attn, cache, table[n:n + 1], [length], gpu))
        for h in range(Hkv):
            rows = slice(h * G, (h + 1) * G)
            _check_rows(o[n, rows], lse[n, rows], q[n, rows], k[:, h], v[:, h], d ** -0.5, d)
            _check_rows(ob[n, rows], lb[n, rows], q[n, rows], k[:, h], v[:, h], d ** -0.5, d)


@pytest.mark.parametrize("N,longest,Hq,Hkv,d", [
    (1, 130, 4, 1, 128), (20, 700, 8, 2, 64), (70, 900, 8, 2, 128), (100, 333, 20, 2, 128), (110, 600, 4, 2, 256),
    (200, 500, 16, 2, 128), (280, 300, 8, 2, 64), (600, 250, 5, 1, 64), (150, 200, 48, 3, 128), (260, 150, 8, 2, 256),
    (1300, 60, 4, 1, 128), (900, 64, 6, 1, 256), (449, 1800, 8, 2, 64)])
def test_decode_dealt_out(attn, gpu, N, longest, Hq, Hkv, d):
    """Rows and heads on either side of the numbers of CTAs that the device holds, with sequences without tokens between."""
    lens = [longest] + [0 if n % 5 == 3 else 1 + (n * 7919) % longest for n in range(1, N)]
    gen, cache, bounds, table = _setup(attn, gpu, lens, Hkv, d, seed=N)
    q, sl = _randn((N, Hq, d), gen, gpu), _i32(lens, gpu)
    o, lse = attn.decode_paged_f8(q, cache, table, sl)
    width = table.shape[1]
    every = torch.arange(width, dtype=torch.int32, device=gpu).expand(N, Hkv, width).contiguous()
    ob, lb = attn.decode_blocks_f8(q, cache, table, sl, every)
    G = Hq // Hkv
    for n in range(N) if N < 40 else sorted({0, 1, 3, 4, 8, N // 3, N // 2, N - 3, N - 2, N - 1}):
        if lens[n] == 0:
            assert not o[n].any() and not ob[n].any() and (lse[n] == -math.inf).all() and (lb[n] == -math.inf).all()
            continue
        k, v = (x[0, :lens[n]].double() for x in _values(attn, cache, table[n:n + 1], [lens[n]], gpu))
        for h in range(Hkv):
            rows = slice(h * G, (h + 1) * G)
            _check_rows(o[n, rows], lse[n, rows], q[n, rows], k[:, h], v[:, h], d ** -0.5, d)
            _check_rows(ob[n, rows], lb[n, rows], q[n, rows], k[:, h], v[:, h], d ** -0.5, d)
    assert attn.device_status() == 0


@pytest.mark.parametrize("N,rows,length,Hq,Hkv,d,K", [
    (3, 1, 9000, 8, 2, 128, 100), (40, 4, 2000, 4, 1, 64, 31), (2, 300, 4000, 16, 2, 128, 9), (700, 1, 40, 2, 1, 256, 2),
    (1, 1, 60000, 5, 1, 128, 999), (5, 7, 3000, 40, 4, 64, 64),
])
def test_decode_blocks_in_many_shares(attn, gpu, N, rows, length, Hq, Hkv, d, K):
    gen, cache, bounds, table = _setup(attn, gpu, [length] * N, Hkv, d, seed=K)
    T = N * rows
    q = _randn((T, Hq, d), gen, gpu)
    cu = torch.arange(0, T + 1, rows, dtype=torch.int32, device=gpu)
    nb = _pages(length)
    blocks = torch.rand((T, Hkv, nb), generator=gen, device=gpu).argsort(-1)[..., :K].to(torch.int32).contiguous()
    o, lse = attn.decode_blocks_f8(q, cache, table, _i32([length] * N, gpu), blocks, cu_seqlens_q=cu)
    G = Hq // Hkv
    for r in range(0, T, max(1, T // 12)):
        n, seen = r // rows, length - (rows - 1 - r % rows)
        k, v = (x[0].double() for x in _values(attn, cache, table[n:n + 1], [length], gpu))
        for h in range(Hkv):
            at = (blocks[r, h].long()[:, None] * PAGE + torch.arange(PAGE, device=gpu)).flatten()
            at = at[at < seen]
            sl = slice(h * G, (h + 1) * G)
            if at.numel() == 0:
                assert not o[r, sl].any() and (lse[r, sl] == -math.inf).all()
                continue
            _check_rows(o[r, sl], lse[r, sl], q[r, sl], k[at, h], v[at, h], d ** -0.5, d)


# ---------------------------------------------------------------------------------------------- selection
def _wanted(q, bounds, table, cu, lens, K, first, last):
    """Selections by 64-bit scores on the GPU, ties to the lowest."""
    T, Hq, d = q.shape
    H = bounds.shape[1]
    out = torch.full((T, H, K), -1, dtype=torch.int32, device=q.device)
    for n, length in enumerate(lens):
        for r in range(cu[n], cu[n + 1]):
            nb = max(0, _pages(length - (cu[n + 1] - 1 - r)))
            if nb <= K:
                out[r, :, :nb] = torch.arange(nb, dtype=torch.int32, device=q.device)
                continue
            x = q[r].double().view(H, -1, d)
            b = bounds[table[n, :nb].long()].double()                                    # nb, H, 2, d
            s = (x.clamp(max=0).sum(1) * b[:, :, 0]).sum(-1) + (x.clamp(min=0).sum(1) * b[:, :, 1]).sum(-1)
            s[:first], s[nb - last:] = math.inf, math.inf
            out[r] = torch.argsort(s, dim=0, descending=True, stable=True)[:K].sort(0).values.T.to(torch.int32)
    return out


@pytest.mark.parametrize("seed", range(12))
def test_select_random(attn, gpu, seed):
    """Random shapes; bounds of which some are far above the rest, in one block or in a tenth of them."""
    rng = np.random.default_rng(seed)
    d, Hkv, G = [64, 128, 256][seed % 3], int(rng.integers(1, 4)), int(rng.integers(1, 9))
    N = int(rng.integers(1, 5))
    max_q = [1, 3, 4, 5, 16, 70][seed % 6]
    rows = [int(rng.integers(0 if max_q > 1 else 1, max_q + 1)) for _ in range(N)]
    lens = [int(rng.integers(max(1, m), 6000)) for m in rows]
    first, last = int(rng.integers(0, 3)), int(rng.integers(1, 3))
    K = first + last + int(rng.integers(0, 60))
    gen = torch.Generator(device=gpu).manual_seed(seed)
    need = [_pages(n) for n in lens]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=gen, device=gpu).to(torch.int32)
    table = torch.full((N, max(need) + seed % 4), 2 ** 30, dtype=torch.int32, device=gpu)
    at = 0
    for n, m in enumerate(need):
        table[n, :m] = order[at:at + m]
        at += m
    b = torch.randn((blocks, Hkv, 2, d), generator=gen, device=gpu).sort(2).values
    if seed % 4 == 1:
        b[order[0].long()] *= 1e6                                  # a first page unlike all others
    if seed % 4 == 2:
        b *= torch.exp(4 * torch.randn((blocks, Hkv, 1, 1), generator=gen, device=gpu))
    if seed % 4 == 3:
        b[torch.rand(blocks, generator=gen, device=gpu) < 0.1] *= 1000.0
    bounds = b.to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    if cu[-1] == 0:
        return
    q = _randn((cu[-1], Hkv * G, d), gen, gpu)
    got = attn.select_blocks(q, bounds, table, _i32(lens, gpu), K, first=first, last=last, cu_seqlens_q=_i32(cu, gpu),
                             max_seqlen_q=max_q)
    assert torch.equal(got, _wanted(q, bounds, table, cu, lens, K, first, last))


@pytest.mark.parametrize("N,length,Hkv,d,K", [(700, 900, 1, 64, 20), (500, 64, 2, 256, 3), (1, 210000, 2, 64, 300),
                                              (2, 200000, 1, 128, 6000), (65, 4000, 4, 128, 100)])
def test_select_of_many_and_of_long_sequences(attn, gpu, N, length, Hkv, d, K):
    """More sequences than a thread counts; tables past what shared memory holds of a row's scores."""
    gen = torch.Generator(device=gpu).manual_seed(N)
    nb = _pages(length)
    bounds = torch.randn((nb * 3, Hkv, 2, d), generator=gen, device=gpu).sort(2).values.to(torch.bfloat16)
    table = torch.stack([torch.randperm(nb * 3, generator=gen, device=gpu)[:nb] for _ in range(N)]).to(torch.int32)
    lens = [length - 16 * (i % 7) for i in range(N)]
    q = _randn((N, 2 * Hkv, d), gen, gpu)
    got = attn.select_blocks(q, bounds, table, _i32(lens, gpu), K)
    some = sorted({0, 1 % N, N // 2, N - 1})
    for n in some:
        want = _wanted(q[n:n + 1], bounds, table[n:n + 1], [0, 1], [lens[n]], K, 1, 2)
        assert torch.equal(got[n:n + 1], want), n
    # pages that are all alike, in tables of this width: the lowest numbers
    got = attn.select_blocks(q, bounds[:1].expand(nb * 3, -1, -1, -1).contiguous(), table, _i32(lens, gpu), K)
    for n in some:
        blocks = max(0, _pages(lens[n]))
        alike = list(range(K - 2)) + [blocks - 2, blocks - 1] if blocks > K else list(range(blocks)) + [-1] * (K - blocks)
        assert (got[n] == torch.tensor(alike, dtype=torch.int32, device=gpu)).all(), n
    if min(lens) < 0:                                              # 64 - 16 * 6: no blocks, and recorded
        assert attn.device_status(clear=True) == 5


@pytest.mark.parametrize("N,Hkv,d,width", [
    (1, 1, 128, 258), (1, 1, 128, 259), (1, 2, 64, 266), (3, 5, 256, 370), (2, 8, 128, 378), (16, 8, 128, 1274), (38, 8, 64, 300),
    (304, 1, 256, 40), (305, 1, 256, 40), (51, 6, 128, 256), (76, 8, 128, 256), (77, 8, 128, 256), (608, 1, 64, 100),
    (609, 1, 64, 100), (400, 1, 128, 257), (100, 4, 256, 255)])
def test_select_of_one_row_each(attn, gpu, N, Hkv, d, width):
    """Either side of the sizes that one launch takes: some sequences without a row, without tokens, with fewer blocks than
    are chosen, with bounds that are no numbers or infinite, and with queries of zeros."""
    gen = torch.Generator(device=gpu).manual_seed(N * width + d)
    rng = np.random.default_rng(N * width + d)
    K, first, last = 17, 2, 1
    lens = [int(x) for x in rng.integers(1, 16 * width + 1, N)]
    lens[0], lens[-1] = 16 * width, lens[-1] if N < 4 else 0
    for n in range(2, N, 9):
        lens[n] = int(rng.integers(1, 16 * K + 20))
    rows = [0 if N > 4 and n % 11 == 5 else 1 for n in range(N)]
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    blocks = 3 * width
    b = torch.randn((blocks, Hkv, 2, d), generator=gen, device=gpu).sort(2).values.to(torch.bfloat16)
    b[torch.rand(blocks, generator=gen, device=gpu) < 0.3] = b[0].clone()                  # many alike
    table = torch.randint(0, blocks, (N, width), generator=gen, device=gpu, dtype=torch.int32)
    q = _randn((cu[-1], 3 * Hkv, d), gen, gpu)
    q[cu[-1] // 3] = 0
    out = torch.full((cu[-1], Hkv, K), 7, dtype=torch.int32, device=gpu)
    for odd in (None, math.inf, math.nan):
        if odd is not None:
            b[1, :, 1, 3] = odd                            # a query that is 0 there has 0 inf in its sum: not a number
            q[:, :, 3] = q[:, :, 3].abs().clamp(min=0.5)
        got = attn.select_blocks(q, b, table, _i32(lens, gpu), K, first=first, last=last, cu_seqlens_q=_i32(cu, gpu),
                                 max_seqlen_q=1, out=out)
        for n in range(N) if N < 20 else sorted({0, 1, 2, 5, 11, N // 2, N - 2, N - 1}):
            if rows[n]:
                want = _wanted_odd(q[cu[n]:cu[n] + 1], b, table[n:n + 1], lens[n], K, first, last)
                assert torch.equal(got[cu[n]], want), (odd, n)
    assert attn.device_status() == 0


@pytest.mark.parametrize("N,Hkv,d,width,most", [(41, 4, 128, 90, 70), (160, 1, 128, 40, 128), (20, 4, 128, 260, 5), (45, 4, 64, 60, 65),
                                                (39, 4, 256, 33, 40), (41, 4, 128, 90, 129), (2, 2, 128, 300, 1000)])
def test_select_of_chunks_of_many_sequences(attn, gpu, N, Hkv, d, width, most):
    """Chunks of different lengths, some of none, and sequences shorter than their rows or their choice; what lies behind the
    results and behind the workspace stays as it was."""
    gen = torch.Generator(device=gpu).manual_seed(N + width)
    rng = np.random.default_rng(N + width)
    rows = [int(x) for x in rng.integers(0, most + 1, N)]
    rows[0], rows[1] = most, 0
    lens = [max(1, int(x)) for x in rng.integers(1, 16 * width + 1, N)]
    lens[0] = 16 * width
    K, blocks = 12, 4 * width
    b = torch.randn((blocks, Hkv, 2, d), generator=gen, device=gpu).sort(2).values.to(torch.bfloat16)
    table = torch.randint(0, blocks, (N, width), generator=gen, device=gpu, dtype=torch.int32)
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    T = cu[-1]
    q = _randn((T + 3, 2 * Hkv, d), gen, gpu)
    out = torch.full((T + 3, Hkv, K), -7, dtype=torch.int32, device=gpu)
    need = attn.select_blocks_workspace_bytes(T + 3, N, most, Hkv, d, width)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=gpu)
    attn.select_blocks(q, b, table, _i32(lens, gpu), K, cu_seqlens_q=_i32(cu, gpu), max_seqlen_q=most, out=out, workspace=ws[:need])
    assert (ws[need:] == 0x5A).all() and (out[T:] == -7).all() and attn.device_status() == 0
    for n in sorted({0, 2 % N, 3 % N, N // 2, N - 1}):
        picked = sorted({0, rows[n] // 2, rows[n] - 1}) if rows[n] else []
        for r in picked:
            seen = lens[n] - (rows[n] - 1 - r)
            if seen <= 0:
                assert (out[cu[n] + r] == -1).all()
                continue
            want = _wanted_odd(q[cu[n] + r:cu[n] + r + 1], b, table[n:n + 1], seen, K, 1, 2)
            assert torch.equal(out[cu[n] + r], want), (n, r)


@pytest.mark.parametrize("rows,Hq,Hkv,d,width,K", [
    (700, 4, 2, 128, 60, 9), (1100, 3, 1, 64, 512, 40), (600, 8, 2, 256, 513, 33), (520, 4, 2, 128, 1024, 64),
    (400, 3, 3, 64, 1300, 700), (350, 15, 3, 128, 1850, 5), (260, 8, 4, 128, 2560, 90), (1050, 2, 1, 256, 2561, 20)])
@pytest.mark.parametrize("kind", ["plain", "far", "alike", "close", "odd"])
def test_select_of_many_rows(attn, gpu, rows, Hq, Hkv, d, width, K, kind):
    """As many rows and heads as are taken a warp each.  far: a few pages are far above all others; alike: a third of the pages
    are copies of one, whose scores tie; close: those copies differ in a channel that adds a part in 10^11 to 10^13 to
    the scores, which 64 bits (a part in 10^16, 512 additions) resolve; odd: bounds that are infinite or no number, queries of zeros and infinities."""
    gen = torch.Generator(device=gpu).manual_seed(rows + width)
    parts = [rows - 90, 0, 90]
    lens, cu = [16 * width - 5, 30, 16 * (width // 2)], [0, rows - 90, rows - 90, rows]
    first, last = 1, 2
    blocks = width + 7
    b = torch.randn((blocks, Hkv, 2, d), generator=gen, device=gpu).sort(2).values
    if kind == "far":
        b[torch.randperm(blocks, generator=gen, device=gpu)[:3]] *= 1e4
    b = b.to(torch.bfloat16)
    if kind in ("alike", "close"):
        copies = torch.rand(blocks, generator=gen, device=gpu) < 0.34
        b[copies] = b[0].clone()
        if kind == "close":
            b[copies, :, :, 7] = torch.randn((int(copies.sum()), Hkv, 1), generator=gen, device=gpu).to(torch.bfloat16)
    table = torch.stack([torch.randperm(blocks, generator=gen, device=gpu)[:width] for _ in lens]).to(torch.int32)
    q = _randn((rows, Hq, d), gen, gpu)
    some = sorted({0, 1, 17, rows // 3, rows - 91, rows - 90, rows - 2, rows - 1})
    if kind == "close":
        q[:, :, 7] = q[:, :, 7].abs().clamp(min=0.1) * 1e-10
    if kind == "odd":
        q[:, :, 3] = q[:, :, 3].abs().clamp(min=0.5)
        b[2, :, 1, 3], b[5, :, 1, 3] = math.inf, math.nan
        q[17], q[rows - 2, 0, 5] = 0, math.inf
    got = attn.select_blocks(q, b, table, _i32(lens, gpu), K, first=first, last=last, cu_seqlens_q=_i32(cu, gpu),
                             max_seqlen_q=rows - 90)
    assert attn.device_status() == 0
    for r in some:
        n = 0 if r < rows - 90 else 2
        want = _wanted_odd(q[r:r + 1], b, table[n:n + 1], lens[n] - (cu[n + 1] - 1 - r), K, first, last)
        assert torch.equal(got[r], want), r
    nb = torch.tensor([_pages(lens[0 if r < rows - 90 else 2] - (cu[1 if r < rows - 90 else 3] - 1 - r)) for r in range(rows)],
                      device=gpu)[:, None, None]
    assert ((got >= 0).sum(-1, keepdim=True) == nb.clamp(max=K)).all() and (got < nb).all()
    full = got[(nb > K).flatten()]
    assert (full[..., 1:] > full[..., :-1]).all()


def _wanted_odd(q, bounds, table, length, K, first, last):
    """_wanted for one row, with NaN above all other scores."""
    nb = _pages(length)
    if nb <= K:
        return _wanted(q, bounds, table, [0, 1], [length], K, first, last)[0]
    H, d = bounds.shape[1], q.shape[-1]
    x, b = q[0].double().view(H, -1, d), bounds[table[0, :nb].long()].double()
    s = (x.clamp(max=0).sum(1) * b[:, :, 0]).sum(-1) + (x.clamp(min=0).sum(1) * b[:, :, 1]).sum(-1)
    key = torch.where(s.isnan(), math.inf, s)
    key[:first], key[nb - last:] = math.inf, math.inf
    order = [sorted(range(nb), key=lambda i: (0 if i < first or i >= nb - last else 1 if nan[i] else 2, -col[i], i))[:K]
             for nan, col in zip(s.isnan().T.tolist(), key.T.tolist())]
    return torch.tensor([sorted(o) for o in order], dtype=torch.int32, device=q.device)


def test_select_of_a_chunk_in_a_wide_table(attn, gpu):
    """A prompt's chunk whose sequence fills a small part of its table, beside one that fills it."""
    gen = torch.Generator(device=gpu).manual_seed(5)
    rows, lens, d = [70, 0, 130], [5000, 40, 100000], 128
    table = torch.randint(0, 6000, (3, 6250), generator=gen, device=gpu, dtype=torch.int32)
    bounds = torch.randn((6000, 1, 2, d), generator=gen, device=gpu).sort(2).values.to(torch.bfloat16)
    cu = [0, 70, 70, 200]
    q = _randn((200, 4, d), gen, gpu)
    got = attn.select_blocks(q, bounds, table, _i32(lens, gpu), 40, cu_seqlens_q=_i32(cu, gpu), max_seqlen_q=130)
    assert torch.equal(got, _wanted(q, bounds, table, cu, lens, 40, 1, 2))


# ---------------------------------------------------------------------------------------------- offsets
def test_pages_and_rows_past_32_bits(attn, gpu):
    """Pages past 2^32 bytes of a cache and of its bounds, and token rows past 2^32 bytes of their tensor."""
    Hkv, d, Hq, lens = 8, 128, 16, [600, 37]
    first = 1_060_000                                              # 4.3 GB of bounds, 34.9 GB of records
    gen, cache, bounds, table = _setup(attn, gpu, lens, Hkv, d, seed=1, first_page=first)
    assert first * Hkv * 4 * d > 2 ** 32
    T, stride = sum(lens), 4 << 20
    flat = torch.empty((T - 1) * stride + Hkv * d, dtype=torch.bfloat16, device=gpu)
    k = flat.as_strided((T, Hkv, d), (stride, d, 1))
    assert (T - 1) * stride * 2 > 2 ** 32
    dense, v = _randn((T, Hkv, d), gen, gpu), _randn((T, Hkv, d), gen, gpu)
    k.copy_(dense)
    t = [torch.arange(n, device=gpu) for n in lens]
    slots = torch.cat([table[n].long()[x // PAGE] * PAGE + x % PAGE for n, x in enumerate(t)]).to(torch.int32)
    attn.cache_append_f8(k, v, slots, cache, bounds=bounds)
    # the same in a small cache
    small, sb = attn.cache_f8_empty(50, Hkv, d, device=gpu), attn.key_bounds_empty(50, Hkv, d, device=gpu)
    st, ss = table - first, slots - first * PAGE
    st = torch.where(table > 0, st, 0).contiguous()
    attn.cache_append_f8(dense, v, ss, small, bounds=sb)
    del flat, k
    q = _randn((2, Hq, d), gen, gpu)
    sl, cu = _i32(lens, gpu), _i32([0, 1, 2], gpu)
    results = []
    for c, b, tab in ((cache, bounds, table), (small, sb, st)):
        picked = attn.select_blocks(q, b, tab, sl, 7)
        many = attn.select_blocks(q.repeat_interleave(8, 0), b, tab, sl, 7, cu_seqlens_q=_i32([0, 8, 16], gpu), max_seqlen_q=8)
        kk, vv = attn.cache_gather_f8(c, tab, sl)
        results.append((picked, many, *attn.decode_paged_f8(q, c, tab, sl), *attn.decode_blocks_f8(q, c, tab, sl, picked),
                        *attn.prefill_paged_f8(q, c, tab, cu, sl, 1), kk[0, :600], vv[0, :600], kk[1, :37], vv[1, :37]))
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------------- streams
def _calls(attn, dev):
    N, Hq, Hkv, d = 2, 8, 2, 128
    lens = [300, 150]
    gen, cache, bounds, table = _setup(attn, dev, lens, Hkv, d, seed=3)
    q1, q = _randn((N, Hq, d), gen, dev), _randn((64, Hq, d), gen, dev)
    sl, cu = _i32(lens, dev), _i32([0, 40, 64], dev)
    picked = attn.select_blocks(q1, bounds, table, sl, 5)
    return {
        "decode_paged_f8": lambda **s: attn.decode_paged_f8(q1, cache, table, sl, **s),
        "decode_blocks_f8": lambda **s: attn.decode_blocks_f8(q1, cache, table, sl, picked, **s),
        "prefill_paged_f8": lambda **s: attn.prefill_paged_f8(q, cache, table, cu, sl, 40, **s),
        "cache_gather_f8": lambda **s: [x[n, :lens[n]] for x in attn.cache_gather_f8(cache, table, sl, **s) for n in range(N)],
        "select_blocks": lambda **s: [attn.select_blocks(q1, bounds, table, sl, 5, **s)],
        "select_blocks chunk": lambda **s: [attn.select_blocks(q, bounds, table, sl, 5, cu_seqlens_q=cu, max_seqlen_q=40, **s)],
    }


NAMES = ["decode_paged_f8", "decode_blocks_f8", "prefill_paged_f8", "cache_gather_f8", "select_blocks", "select_blocks chunk"]


@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_a_side_stream_has_memory_of_its_own(attn, gpu, name):
    calls = _calls(attn, gpu)
    assert list(calls) == NAMES
    call, side = calls[name], torch.cuda.Stream()
    want = [x.clone() for x in call()]
    torch.cuda.synchronize()
    first = call(stream=side)                                  # the side stream's pool gets its memory
    del first
    torch.cuda.synchronize()
    for _ in range(2):
        seen = _busy_with_freed_blocks(gpu)
        busy = torch.cuda.Event()
        busy.record()
        got = call(stream=side)
        side.synchronize()
        assert not busy.query()                                # the call did not wait for the current stream
        kept = [x.clone() for x in got]
        torch.cuda.synchronize()
        assert all((b == 0xFF).all() for b in seen)
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_two_calls_at_once_and_a_captured_fork(attn, gpu):
    """Two streams at a time, each with a workspace of its own; and inside a capture, on a forked stream."""
    calls = _calls(attn, gpu)
    want = {n: [x.clone() for x in calls[n]()] for n in NAMES}
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        got = [(n, calls[n](stream=s)) for n in NAMES for s in (a, b)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for n, g in got for x, y in zip(g, want[n]))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = {n: calls[n](stream=side) for n in NAMES}
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for n in NAMES:
            for x in got[n]:
                x.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for n in NAMES for x, y in zip(got[n], want[n]))


def test_steps_without_tokens(attn, gpu):
    gen, cache, bounds, table = _setup(attn, gpu, [40, 20], 2, 64, seed=9)
    sl, cu = _i32([40, 20], gpu), _i32([0, 0, 0], gpu)
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=gpu)
    assert attn.select_blocks(q, bounds, table, sl, 4, cu_seqlens_q=cu).shape == (0, 2, 4)
    o, lse = attn.decode_blocks_f8(q, cache, table, sl, torch.zeros((0, 2, 4), dtype=torch.int32, device=gpu), cu_seqlens_q=cu)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = attn.prefill_paged_f8(q, cache, table, cu, sl, 1)
    assert o.shape == (0, 4, 64)


# ---------------------------------------------------------------------------------------------- waits that run out
WAIT_LIMIT_NS = 2_000_000


@pytest.fixture(scope="module")
def waitlib():
    """A test-only build with a limit of 2 ms and copies that can be left out; nothing faults, traps or hangs."""
    from attention_attn_prefill_gb300.build import build
    path = build(variant="waittest", extra_flags=["-DATTN_TEST_DROP_COPY", f"-DATTN_WAIT_LIMIT_NS={WAIT_LIMIT_NS}ull"])
    handle = ctypes.CDLL(path)
    for name in ("attn_decode_paged_f8", "attn_decode_blocks_f8", "attn_decode_f8_workspace_bytes", "attn_device_status",
                 "attn_select_blocks", "attn_select_blocks_workspace_bytes"):
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = _SIGNATURES[name]
    for name in ("attn_test_drop_copy_f8", "attn_test_drop_copy_select"):
        getattr(handle, name).restype, getattr(handle, name).argtypes = ctypes.c_int, [ctypes.c_int]
    return handle


def _status(lib):
    code = ctypes.c_uint32(0)
    assert lib.attn_device_status(ctypes.byref(code), 1) == 0
    return int(code.value)


def _timed(call):
    start, end = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    torch.cuda.synchronize()
    start.record()
    assert call() == 0                  # the launch itself is fine; the error is recorded on the device
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end)


@pytest.mark.parametrize("drop", [1, 2])
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("N,length,Hq,Hkv,d", [(3, 700, 8, 2, 128), (9000, 16, 4, 2, 64), (9000, 16, 5, 1, 128),
                                               (5000, 16, 2, 1, 256), (300, 16, 4, 2, 64), (200, 100, 5, 1, 128),
                                               (120, 40, 4, 2, 256), (3, 3000, 8, 2, 128), (2, 2500, 5, 1, 64),
                                               (3, 2500, 4, 1, 256)])
def test_decode_waits_that_run_out(attn, gpu, waitlib, drop, listed, N, length, Hq, Hkv, d):
    lib = waitlib
    gen, cache, bounds, table = _setup(attn, gpu, [length] * 3, Hkv, d, seed=2)
    table = table[torch.arange(N, device=gpu) % 3].contiguous()
    q, sl = _randn((N, Hq, d), gen, gpu), _i32([length] * N, gpu)
    o = torch.empty_like(q)
    need = lib.attn_decode_f8_workspace_bytes(d)
    ws = torch.zeros(need, dtype=torch.uint8, device=gpu)
    width = table.shape[1]
    blocks = torch.arange(width, dtype=torch.int32, device=gpu).expand(N, Hkv, width).contiguous()
    stream = torch.cuda.current_stream().cuda_stream
    tail = (N, Hq, Hkv, d, PAGE, width, cache.shape[0], d ** -0.5, ws.data_ptr(), need, stream)

    def call():
        if listed:
            return lib.attn_decode_blocks_f8(q.data_ptr(), cache.data_ptr(), table.data_ptr(), 0, sl.data_ptr(), blocks.data_ptr(),
                                             width, o.data_ptr(), 0, N, *tail)
        return lib.attn_decode_paged_f8(q.data_ptr(), cache.data_ptr(), table.data_ptr(), sl.data_ptr(), o.data_ptr(), 0, *tail)

    assert _status(lib) == 0
    quick = _timed(call)
    want = o.clone()
    assert _status(lib) == 0 and torch.isfinite(want).all()
    assert lib.attn_test_drop_copy_f8(drop) == 0
    o.fill_(float("nan"))
    ms = _timed(call)
    assert lib.attn_test_drop_copy_f8(0) == 0
    assert _status(lib) == 1            # kDevWaitTimeout
    # a warp's own wait, one for each of the others' and the loading warp's, the drain of its slots: 6 limits
    assert ms < 8 * WAIT_LIMIT_NS * 1e-6 + quick, ms
    if N > 3:
        same = (o == want).all(-1).all(-1)
        assert int(same.sum()) > N - N // 100 - 3 and same[N // 2:].all()
    _timed(call)
    assert _status(lib) == 0 and torch.equal(o, want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_select_waits_that_run_out(attn, gpu, waitlib, d):
    lib = waitlib
    gen = torch.Generator(device=gpu).manual_seed(d)
    rows, length, Hq, Hkv, K = 200, 6000, 4, 2, 20
    nb = _pages(length)
    bounds = torch.randn((nb, Hkv, 2, d), generator=gen, device=gpu).sort(2).values.to(torch.bfloat16)
    table = torch.randperm(nb, generator=gen, device=gpu).to(torch.int32)[None].contiguous()
    q, cu, sl = _randn((rows, Hq, d), gen, gpu), _i32([0, rows], gpu), _i32([length], gpu)
    out = torch.empty((rows, Hkv, K), dtype=torch.int32, device=gpu)
    need = lib.attn_select_blocks_workspace_bytes(rows, 1, rows, Hkv, d, nb)
    ws = torch.zeros(need, dtype=torch.uint8, device=gpu)
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        return lib.attn_select_blocks(q.data_ptr(), bounds.data_ptr(), table.data_ptr(), cu.data_ptr(), sl.data_ptr(),
                                      out.data_ptr(), K, 1, 2, rows, 1, rows, Hq, Hkv, d, PAGE, nb, nb, ws.data_ptr(), need, stream)

    assert _status(lib) == 0
    quick = _timed(call)
    want = out.clone()
    assert _status(lib) == 0 and torch.equal(want, _wanted(q, bounds, table, [0, rows], [length], K, 1, 2))
    assert lib.attn_test_drop_copy_select(1) == 0
    ms = _timed(call)
    assert lib.attn_test_drop_copy_select(0) == 0
    assert _status(lib) == 1
    # the issuing warp's wait, the epilogue's and the loading warp's, and the last copies'
    assert ms < 8 * WAIT_LIMIT_NS * 1e-6 + quick, ms
    _timed(call)
    assert _status(lib) == 0 and torch.equal(out, want)
