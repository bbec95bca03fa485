"""The serving-step operators against their float64 definitions.

Tolerances, fixed before the first run (u = 2^-24, half a float32 step; a bf16 rounding is off by at
most 2^-8 relative):
  norm + rotation: the sum of squares takes at most 13 roundings (halved by the root), the mean, eps and
    rsqrt (2 ulp) 6 more, the two factors 2, the table entry 1, the rotation 3: under 20 u relative to
    the terms |a| + |b| of an output, taken as 2^-19; then one bf16 rounding.
  decode over the 4-bit cache: a group's product sums 64 terms |q| (16 + c) <= 31 |q| in float32, every
    addition allowed a whole ulp (2 u), so a score is off by at most B = scale * sum_g s_g * 31 * sum|q| *
    70 * 2 u, and a probability relatively by B + 2^-16 (ex2, the merge).  A weighted mean of terms t moves
    by at most 2 (B + 2^-16) max|t|.  The terms are what the kernel sums, x (c - 8) less x (z - 8) with x =
    p s, a value of 0 (c = z) being a difference of two: max|t| is taken as 31 max s of the group.  x enters
    both as the same fp16 number, off by half a step of 11 bits, 2^-12 relative: 2^-12 max|v| for the mean.
    Below 2^-20 max s (at p = 1) it is off by 2^-31 max s instead: |c - z| <= 15 times L tokens of that are
    under 2^-11 max s for L <= 2^16, less than half of 2^-16 * 31 max s.  The LSE moves by at most
    B + 2^-20 (1 + |lse|).
  whole numbers, 4-bit codes and what they stand for: equal.
"""
import math

import numpy as np
import pytest
import torch

import oracle.attention as oa
import oracle.step as os_

pytestmark = pytest.mark.gpu

PAGE = 16


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _randn(shape, seed, dev, gain=None):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    return (x if gain is None else x * gain).to(torch.bfloat16).to(dev)


def _pages(n):
    return (n + PAGE - 1) // PAGE


# ------------------------------------------------------------------------------------------ tables
def _tables_case(cached, new, seed, extra_free=3, width_extra=2):
    rng = np.random.default_rng(seed)
    need = sum(_pages(c + w) - _pages(c) for c, w in zip(cached, new))
    held = sum(_pages(c) for c in cached)
    num_blocks = held + need + extra_free
    perm = rng.permutation(num_blocks).tolist()
    width = max(1, max(_pages(c + w) for c, w in zip(cached, new)) + width_extra)
    table = np.full((len(cached), width), -7, np.int64)
    for n, c in enumerate(cached):
        for j in range(_pages(c)):
            table[n, j] = perm.pop(0)
    return table, perm, num_blocks


@pytest.mark.parametrize("cached,new,pad", [
    ([0], [0], 0), ([0], [1], 0), ([0], [1], 63), ([15], [1], 0), ([16], [1], 1), ([31, 0, 5], [2, 33, 0], 4),
    ([0] * 7, [0] * 7, 5), ([100], [5000], 0), ([0, 17, 40, 16], [1024, 1, 1024, 1023], 1000),
    ([(i * 37) % 300 for i in range(600)], [1] * 600, 0),
    ([(i * 37) % 300 for i in range(1500)], [(i * 7) % 23 if i % 5 else 0 for i in range(1500)], 77),
    ([3] * 300, [0] * 299 + [2050], 0),                      # one owner behind many without tokens
])
def test_tables(attn, gpu, cached, new, pad):
    table, free, num_blocks = _tables_case(cached, new, len(cached))
    T = sum(new) + pad
    bt = _i32(table.tolist(), gpu)
    for _ in range(2):                                        # repeated on the same inputs: the same tables
        out = attn.step_tables(_i32(cached, gpu), _i32(new, gpu), _i32(free, gpu), bt, T, num_blocks)
        want = os_.step_tables(cached, new, free, table, T)
        for got, w in zip(out, want[:5]):
            assert np.array_equal(got.cpu().numpy().reshape(-1), np.reshape(w, -1))
        assert np.array_equal(bt.cpu().numpy(), want[5])


def test_tables_without_free_pages(attn, gpu):
    bt = _i32([[4, 0]], gpu)
    out = attn.step_tables(_i32([3], gpu), _i32([5], gpu), _i32([], gpu), bt, 5, 8)
    assert out.slots.tolist() == [67, 68, 69, 70, 71] and int(out.pages_used) == 0


def test_tables_report_what_does_not_fit(attn, gpu):
    """Device status 6; the request at fault takes part in nothing, the others are served."""
    def step(cached, new, free, width, T, num_blocks=64):
        bt = torch.arange(len(cached) * width, dtype=torch.int32, device=gpu).view(len(cached), width)
        before = bt.clone()
        out = attn.step_tables(_i32(cached, gpu), _i32(new, gpu), _i32(free, gpu), bt, T, num_blocks)
        return out, bt, before, attn.device_status(clear=True)

    # too long for the table; its tokens keep their rows
    out, bt, before, code = step([0, 30, 1], [1, 5, 1], [50, 51, 52], 2, 7)
    assert code == 6 and out.seq_lens.tolist() == [1, 30, 2] and out.cu_seqlens.tolist() == [0, 1, 6, 7]
    assert out.slots.tolist() == [800] + [-1] * 5 + [4 * 16 + 1] and int(out.pages_used) == 1
    assert torch.equal(bt[1:], before[1:])
    # negative lengths
    out, _, _, code = step([-1, 4, 2], [1, -3, 1], [50], 2, 2)
    assert code == 6 and out.seq_lens.tolist() == [0, 4, 3] and out.cu_seqlens.tolist() == [0, 1, 1, 2]
    assert out.slots.tolist() == [-1, 4 * 16 + 2]
    # the free pages run out at the second request; the third needs none
    out, bt, before, code = step([0, 16, 3], [16, 17, 1], [50, 51], 4, 34)
    assert code == 6 and out.seq_lens.tolist() == [16, 16, 4] and int(out.pages_used) == 1
    assert out.slots.tolist() == list(range(800, 816)) + [-1] * 17 + [8 * 16 + 3]
    assert torch.equal(bt[1:], before[1:])
    # more tokens than rows
    out, _, _, code = step([0, 0], [2, 2], [50, 51], 2, 3)
    assert code == 6 and out.slots.tolist() == [800, 801, -1] and out.cu_seqlens.tolist() == [0, 2, 4]
    # a free page outside the cache: status 2, its tokens are nowhere, the table is not written
    out, bt, before, code = step([0], [17], [70, 5], 2, 17)
    assert code == 2 and out.slots.tolist() == [-1] * 16 + [80] and bt.tolist() == [[0, 5]]


def test_tables_after_a_request_without_pages(attn, gpu):
    """A request that finds too few pages ends the taking of pages, also for a later one that needs fewer than are
    left; requests that need none are served."""
    cached, new = [0, 0, 3, 0, 16, 5], [16, 80, 1, 0, 1, 11]
    bt = torch.arange(36, dtype=torch.int32, device=gpu).view(6, 6)
    before = bt.clone()
    out = attn.step_tables(_i32(cached, gpu), _i32(new, gpu), _i32([50, 51, 52], gpu), bt, sum(new), 64)
    assert attn.device_status(clear=True) == 6
    assert out.seq_lens.tolist() == [16, 0, 4, 0, 16, 16] and int(out.pages_used) == 1
    assert out.cu_seqlens.tolist() == np.concatenate([[0], np.cumsum(new)]).tolist()
    assert out.slots.tolist() == (list(range(800, 816)) + [-1] * 80 + [12 * 16 + 3] + [-1]
                                  + list(range(30 * 16 + 5, 30 * 16 + 16)))
    before[0, 0] = 50
    assert torch.equal(bt, before)


# ------------------------------------------------------------------------------------------ norm + rotation
def test_rope_table(attn, gpu):
    """Within half a float32 step of the cosine and sine, far positions too."""
    t = _np(attn.rope_table(131073, 128, 500000.0, device=gpu))
    pos = np.array([0, 1, 2, 77, 8191, 65537, 131072])
    a = os_.rope_angles(pos, 128, 500000.0)
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    # the angle is at most 131072 with a few roundings in 64 bits: 131072 * 2^-51, next to 2^-25 of the entry
    assert np.abs(t[pos] - want).max() <= 2.0 ** -25 + 131072 * 2.0 ** -50


def _rope_case(T, Hq, Hkv, d, rot, seed, dev, max_pos=5000, theta=10000.0):
    qkv = _randn((T, (Hq + 2 * Hkv) * d + 8), seed, dev)     # token stride no multiple of d
    q = qkv[:, :Hq * d].view(T, Hq, d) if T > 1 else qkv[:, :Hq * d].reshape(T, Hq, d)
    cut = lambda at, H: qkv[:, at * d:(at + H) * d].unflatten(1, (H, d))  # noqa: E731
    q, k, v = cut(0, Hq), cut(Hq, Hkv), cut(Hq + Hkv, Hkv)
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, max_pos, T)
    pos[:2] = [0, max_pos - 1][:T]
    a = os_.rope_angles(pos, rot, theta) if rot else np.zeros((T, 0))
    return q, k, v, _i32(pos.tolist(), dev), np.cos(a), np.sin(a)


def _check_rope(got, x, weight, eps, cos, sin, inter, what):
    want, size = os_.norm_rope(_np(x), None if weight is None else _np(weight), eps, cos, sin, inter)
    err = np.abs(_np(got) - want)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size * (1 + 2.0 ** -8)
    assert (err <= tol).all(), f"{what}: {(err / np.maximum(tol, 1e-30)).max():.3g} of the tolerance"


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,norm", [
    (1, 1, 1, 64, 64, False, True), (1, 1, 1, 64, 64, True, True), (3, 5, 1, 128, 128, False, True),
    (33, 4, 2, 128, 64, False, True), (33, 4, 2, 128, 32, True, True), (7, 32, 8, 128, 128, False, True),
    (5, 16, 2, 256, 256, False, True), (6, 16, 2, 256, 64, True, True), (9, 3, 3, 256, 16, False, True),
    (65, 2, 1, 64, 48, False, False), (65, 2, 1, 64, 0, False, True), (4, 71, 1, 64, 16, True, True),
    (1000, 8, 2, 128, 128, False, False), (513, 3, 2, 64, 32, False, True), (40, 40, 10, 128, 80, False, True),
])
def test_norm_rope(attn, gpu, T, Hq, Hkv, d, rot, inter, norm):
    q, k, v, pos, cos, sin = _rope_case(T, Hq, Hkv, d, rot, T + d, gpu)
    table = attn.rope_table(5000, rot, 10000.0, device=gpu) if rot else None
    qw = (1 + 0.3 * torch.randn(d)).to(torch.bfloat16).to(gpu) if norm else None
    kw = (1 + 0.3 * torch.randn(d)).to(torch.bfloat16).to(gpu) if norm else None
    qo, ko = attn.qk_norm_rope(q, k, pos if rot else None, table, qw, kw, eps=1e-5, interleaved=inter)
    _check_rope(qo, q, qw, 1e-5, cos, sin, inter, "q")
    _check_rope(ko, k, kw, 1e-5, cos, sin, inter, "k")
    # the same into the paged cache: the same bits, nothing else touched, padded tokens not written
    num_blocks = _pages(T) + 2
    slots = torch.randperm(num_blocks * PAGE, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    slots[T // 2] = -1
    kc, vc = (torch.full((num_blocks, PAGE, Hkv, d), 7.0, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    q2, k2 = attn.qk_norm_rope(q, k, pos if rot else None, table, qw, kw, eps=1e-5, interleaved=inter, v=v,
                               k_cache=kc, v_cache=vc, slots=slots.to(gpu))
    assert k2 is None and torch.equal(q2, qo)
    want_k, want_v = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0)
    live = slots >= 0
    at = slots[live].long().to(gpu)
    want_k.view(-1, Hkv, d)[at] = ko[live.to(gpu)]
    want_v.view(-1, Hkv, d)[at] = v[live.to(gpu)]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    # in place
    q3, k3 = q.clone(), k.clone()
    attn.qk_norm_rope(q3, k3, pos if rot else None, table, qw, kw, eps=1e-5, interleaved=inter, q_out=q3, k_out=k3)
    assert torch.equal(q3, qo) and torch.equal(k3, ko)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("only", ["q", "k"])
def test_norm_of_one_side(attn, gpu, only, inter):
    """A weight for queries or for keys alone: the other side is turned without a norm."""
    T, Hq, Hkv, d, rot = 21, 10, 3, 128, 96
    q, k, v, pos, cos, sin = _rope_case(T, Hq, Hkv, d, rot, 5, gpu)
    table = attn.rope_table(5000, rot, 10000.0, device=gpu)
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(6))).to(torch.bfloat16).to(gpu)
    qw, kw = (w, None) if only == "q" else (None, w)
    qo, ko = attn.qk_norm_rope(q, k, pos, table, qw, kw, eps=1e-5, interleaved=inter)
    _check_rope(qo, q, qw, 1e-5, cos, sin, inter, "q")
    _check_rope(ko, k, kw, 1e-5, cos, sin, inter, "k")
    both, kboth = attn.qk_norm_rope(q, k, pos, table, w, w, eps=1e-5, interleaved=inter)
    none, knone = attn.qk_norm_rope(q, k, pos, table, interleaved=inter)
    assert torch.equal(qo, both if only == "q" else none) and torch.equal(ko, kboth if only == "k" else knone)


def test_norm_of_small_large_and_zero_rows(attn, gpu):
    """eps keeps a row of zeros at zero; large rows stay finite."""
    d = 128
    x = torch.zeros((4, 1, d), dtype=torch.bfloat16, device=gpu)
    x[1] = 1e-12
    x[2] = 3e15
    x[3, 0, 5] = -2.0
    w = torch.ones(d, dtype=torch.bfloat16, device=gpu)
    q, k = attn.qk_norm_rope(x, x, None, None, w, w, eps=1e-6)
    none = np.zeros((4, 0))
    _check_rope(q, x, w, 1e-6, none, none, False, "q")
    assert torch.equal(q, k) and (q[0] == 0).all()


def test_rope_reports_positions_and_slots(attn, gpu):
    x = _randn((3, 2, 64), 1, gpu)
    table = attn.rope_table(10, 64, device=gpu)
    q, _ = attn.qk_norm_rope(x, x, _i32([0, 10, -1], gpu), table)
    assert attn.device_status(clear=True) == 7
    want, _ = attn.qk_norm_rope(x, x, _i32([0, 9, 0], gpu), table)
    assert torch.equal(q, want)
    kc, vc = (torch.zeros((2, PAGE, 2, 64), dtype=torch.bfloat16, device=gpu) for _ in range(2))
    attn.qk_norm_rope(x, x, None, None, v=x, k_cache=kc, v_cache=vc, slots=_i32([31, 32, -5], gpu))
    assert attn.device_status(clear=True) == 8
    assert torch.equal(kc.view(-1, 2, 64)[31], x[0]) and int((kc != 0).sum()) == int((x[0] != 0).sum())


# ------------------------------------------------------------------------------------------ 4-bit cache
def _cache_case(lens, Hkv, d, seed, dev, gain=None):
    """An empty cache, shuffled pages and K, V of all tokens of the sequences."""
    rng = np.random.default_rng(seed)
    num_blocks = sum(_pages(n) for n in lens) + 3
    perm = rng.permutation(num_blocks).tolist()
    width = max(1, max(_pages(n) for n in lens))
    table = np.zeros((len(lens), width), np.int64)
    slots = []
    for n, length in enumerate(lens):
        for j in range(_pages(length)):
            table[n, j] = perm.pop()
        slots += [int(table[n, p // PAGE]) * PAGE + p % PAGE for p in range(length)]
    T = len(slots)
    k, v = _randn((T, Hkv, d), seed, dev, gain), _randn((T, Hkv, d), seed + 1, dev, gain)
    cache = torch.randint(0, 256, (num_blocks, Hkv, 17 * d), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(seed)).to(dev)
    return cache, _i32(table.tolist(), dev), _i32(lens, dev), k, v, _i32(slots, dev)


@pytest.mark.parametrize("lens,Hkv,d", [
    ([1], 1, 64), ([16], 1, 128), ([17, 0, 5], 2, 64), ([40, 3], 3, 128), ([33, 16, 1], 2, 256), ([200], 8, 128),
])
def test_cache_append_and_gather(attn, gpu, lens, Hkv, d):
    cache, table, sl, k, v, slots = _cache_case(lens, Hkv, d, 11 + d, gpu)
    before = cache.clone()
    attn.cache_append_q4(k, v, slots, cache)
    ko, vo = (torch.full((len(lens), table.shape[1] * PAGE, Hkv, d), 9.0, dtype=torch.bfloat16, device=gpu)
              for _ in range(2))
    attn.cache_gather_q4(cache, table, sl, k_out=ko, v_out=vo)
    wk, wv = os_.stored(_np(k)), os_.stored(_np(v))
    at = 0
    for n, length in enumerate(lens):
        assert np.array_equal(_np(ko)[n, :length], wk[at:at + length])
        assert np.array_equal(_np(vo)[n, :length], wv[at:at + length])
        assert (ko[n, length:] == 9).all() and (vo[n, length:] == 9).all()    # rows behind the end
        at += length
    # the layout, record by record, and the bytes of every other token as they were
    held = {int(s) for s in slots}
    for page in range(cache.shape[0]) if d < 256 else range(0):
        for h in range(Hkv):
            got, old = (os_.read_record(c[page, h].cpu().numpy(), d) for c in (cache, before))
            for tok in range(PAGE):
                s = page * PAGE + tok
                for which, x in ((0, wk), (1, wv)):
                    if s in held:
                        assert np.array_equal(got[which][tok], x[slots.tolist().index(s), h])
                    else:
                        assert np.array_equal(got[which][tok], old[which][tok], equal_nan=True)


def test_gather_from_a_wide_table(attn, gpu):
    """Rows of the table far longer than the sequences, and more records than warps are started for."""
    lens, Hkv, d, wide = [1, 0, 300, 16] + [40] * 700, 2, 64, 200
    cache, table, sl, k, v, slots = _cache_case(lens, Hkv, d, 17, gpu)
    attn.cache_append_q4(k, v, slots, cache)
    spread = torch.full((len(lens), wide), -1, dtype=torch.int32, device=gpu)
    spread[:, :table.shape[1]] = table
    for n, length in enumerate(lens):
        spread[n, _pages(length):] = -1
    k0, v0 = attn.cache_gather_q4(cache, table, sl)
    k1, v1 = attn.cache_gather_q4(cache, spread, sl)
    assert attn.device_status(clear=True) == 0
    at = 0
    for n, length in enumerate(lens):
        want_k, want_v = (os_.stored(_np(x[at:at + length])) for x in (k, v))
        assert (_np(k1[n, :length]) == want_k).all() and (_np(v1[n, :length]) == want_v).all()
        assert torch.equal(k0[n, :length], k1[n, :length]) and torch.equal(v0[n, :length], v1[n, :length])
        at += length


@pytest.mark.parametrize("order", ["shuffled", "reversed", "singles", "strided"])
def test_cache_append_orders_agree(attn, gpu, order):
    """Whatever the order and grouping of the tokens, and the stride of their rows, the same bytes."""
    cache, table, sl, k, v, slots = _cache_case([100, 7, 64], 2, 128, 5, gpu)
    want = cache.clone()
    attn.cache_append_q4(k, v, slots, want)
    T = k.shape[0]
    if order == "singles":
        for t in range(T):
            attn.cache_append_q4(k[t:t + 1], v[t:t + 1], slots[t:t + 1], cache)
    elif order == "strided":
        both = torch.cat([v.flatten(1), k.flatten(1), torch.zeros((T, 8), dtype=k.dtype, device=gpu)], 1)
        attn.cache_append_q4(both[:, 256:512].unflatten(1, (2, 128)), both[:, :256].unflatten(1, (2, 128)), slots, cache)
    else:
        at = torch.randperm(T) if order == "shuffled" else torch.arange(T - 1, -1, -1)
        at = at.to(gpu)
        attn.cache_append_q4(k[at].contiguous(), v[at].contiguous(), slots[at].contiguous(), cache)
    assert torch.equal(cache, want)


@pytest.mark.parametrize("d,Hkv", [(64, 20), (128, 11), (256, 5)])
@pytest.mark.parametrize("order", ["whole", "offset", "holes", "swapped", "shuffled", "tails"])
def test_append_by_pages_agrees_with_rows(attn, gpu, order, d, Hkv):
    """A call large enough to write whole pages at once gives the bytes of small calls, however the pages' tokens
    lie in the batch."""
    T, num_blocks = 997, 400
    rng = np.random.default_rng(d)
    pages = rng.permutation(num_blocks)
    slots = np.concatenate([p * PAGE + np.arange(PAGE) for p in pages[:T // PAGE + 1]])
    if order == "offset":                                     # a page starts 5 tokens into the batch
        slots = np.concatenate([[pages[-1] * PAGE + i for i in (3, 7, 2, 9, 15)], slots])
    elif order == "tails":                                    # short sequences between whole pages
        cut = [slots[i * PAGE:i * PAGE + (PAGE if i % 3 else 1 + i % 15)] for i in range(T // PAGE + 1)]
        slots = np.concatenate(cut + [pages[200 + i] * PAGE + np.arange(12) for i in range(60)])
    slots = slots[:T]
    if order == "holes":
        slots = np.where(rng.random(T) < 0.05, -1, slots)
    elif order == "swapped":                                  # two tokens of some pages in the other order
        for i in range(0, T - PAGE, 3 * PAGE):
            j = i + rng.integers(0, 15)
            slots[j], slots[j + 1] = slots[j + 1], slots[j]
    elif order == "shuffled":
        slots = rng.permutation(slots)
    slots = _i32(slots.tolist(), gpu)
    T = slots.numel()
    assert T * Hkv * d > 1 << 20 and 128 * Hkv * d <= 1 << 20   # by pages, and by rows
    k, v = _randn((T, Hkv, d), 1, gpu), _randn((T, Hkv, d), 2, gpu)
    cache = torch.randint(0, 256, (num_blocks, Hkv, 17 * d), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(d)).to(gpu)
    want = cache.clone()
    attn.cache_append_q4(k, v, slots, cache)
    for at in range(0, T, 128):
        attn.cache_append_q4(k[at:at + 128], v[at:at + 128], slots[at:at + 128], want)
    assert torch.equal(cache, want) and attn.device_status(clear=True) == 0
    # slots past the end are reported and skipped, with the rest of the batch written
    bad = slots.clone()
    bad[500:520] = num_blocks * PAGE + torch.arange(20, dtype=torch.int32, device=gpu)
    attn.cache_append_q4(k, v, bad, cache)
    assert torch.equal(cache, want) and attn.device_status(clear=True) == 8


def test_cache_values_at_the_edges(attn, gpu):
    """Zeros, one sign, ties, exact grids, tiny and large ranges; infinities and NaN spoil their group only."""
    d = 128
    rng = np.random.default_rng(0)
    rows = [np.zeros(d), np.full(d, 3.0), np.full(d, -0.001), np.abs(rng.standard_normal(d)) + 5,
            rng.integers(-15, 16, d) * 0.5, rng.integers(0, 31, d) * 0.5, rng.integers(-15, 1, d) * 12.0,
            rng.standard_normal(d) * 1e-30, rng.standard_normal(d) * 1e37, np.where(np.arange(d) == 3, 1e9, 1e-9),
            np.where(np.arange(d) == 70, -1.0, 0.0), rng.standard_normal(d) * 2.0 ** -128]
    x = torch.tensor(np.array(rows)).to(torch.bfloat16).view(-1, 1, d).to(gpu)
    T = x.shape[0]
    bad = x.clone()
    bad[0, 0, 5], bad[1, 0, 64], bad[2, 0, 127] = float("nan"), float("inf"), -float("inf")
    bad[3, 0, 0], bad[3, 0, 1] = 3e38, -3e38                    # the range overflows
    cache = attn.cache_q4_empty(1, 1, d, device=gpu)
    attn.cache_append_q4(x, bad, _i32(list(range(T)), gpu), cache)
    k, v = attn.cache_gather_q4(cache, _i32([[0]], gpu), _i32([T], gpu))
    assert np.array_equal(_np(k)[0, :T, 0], os_.stored(_np(x)[:, 0]))
    got, want = _np(v)[0, :T, 0], os_.stored(np.nan_to_num(_np(bad)[:, 0], nan=0.0, posinf=0.0, neginf=0.0))
    for r, half in ((0, 0), (1, 1), (2, 1), (3, 0)):
        assert np.isnan(got[r, half * 64:half * 64 + 64]).all()
        want[r, half * 64:half * 64 + 64] = np.nan
    assert np.array_equal(got, want, equal_nan=True)


def _bf16_between(lo, hi):
    """Every bf16 number x with lo <= x <= hi and |x| >= max(-lo, hi) / 120: all whose code is not the zero point's."""
    x = np.arange(1 << 16, dtype=np.uint32) << 16
    with np.errstate(invalid="ignore"):                       # NaN among them
        x = x.view(np.float32).astype(np.float64)
        return x[(x >= lo) & (x <= hi) & (np.abs(x) >= max(-lo, hi) / 120)]


def _groups_of_every_quotient(exponent):
    """Groups [n, 64] whose scale is m 2^(exponent - 3), m = 8 .. 15: for each zero point 0 .. 15 every bf16 number of
    the range, and for each bf16 number as the minimum one group."""
    rng = np.random.default_rng(exponent + 1000)
    out = []
    for m in range(8, 16):
        s = m * 2.0 ** (exponent - 3)
        for z in range(16):
            x = _bf16_between(-z * s, (15 - z) * s)
            x = np.concatenate([x, np.zeros(-len(x) % 62)]).reshape(-1, 62)
            ends = np.broadcast_to([-z * s, (15 - z) * s], (len(x), 2))
            out.append(np.concatenate([ends, x], 1))
        every = _bf16_between(-15 * s, 15 * s)
        for lo in every[(every < 0) & (every >= -15 * s)]:
            ok = every[(every >= lo) & (every <= 15 * s + lo)]
            if len(ok):
                out.append(np.concatenate([[lo, ok.max()], rng.choice(ok, 62)])[None])
    return np.concatenate(out)


# the middle of the range, the ends of what the product with a reciprocal takes (s from 10^-20 on), and past them
@pytest.mark.parametrize("exponent", [0, -66, -67, -70, -100, -120, 84, 119])
def test_cache_quotients(attn, gpu, exponent):
    """Every quotient of a bf16 number and a scale that does not round to 0, ties among them: the codes of the
    definition.  By rows and by pages."""
    x = _groups_of_every_quotient(exponent)
    x = np.stack([x, x[::-1]], 1)                             # two heads
    want = os_.stored(x)
    t = torch.from_numpy(x).to(torch.bfloat16).to(gpu)
    assert np.array_equal(_np(t), x)                          # bf16 numbers all
    T = t.shape[0]
    table = torch.arange(_pages(T), dtype=torch.int32, device=gpu).view(1, -1)
    slots = torch.arange(T, dtype=torch.int32, device=gpu)
    cache = attn.cache_q4_empty(_pages(T), 2, 64, device=gpu)
    paged = cache.clone()
    assert T > 1 << 13                                        # over 2^20 values go by pages
    attn.cache_append_q4(t, t, slots, paged)
    for at in range(0, T, 8192):
        attn.cache_append_q4(t[at:at + 8192], t[at:at + 8192], slots[at:at + 8192], cache)
    assert torch.equal(cache, paged)
    for got in attn.cache_gather_q4(cache, table, _i32([T], gpu)):
        assert np.array_equal(_np(got)[0, :T], want)


def test_cache_reports(attn, gpu):
    cache, table, sl, k, v, slots = _cache_case([20], 1, 64, 3, gpu)
    want = cache.clone()
    attn.cache_append_q4(k[:1], v[:1], slots[:1], want)
    some = slots.clone()
    some[1:] = -1
    some[2] = cache.shape[0] * PAGE
    attn.cache_append_q4(k, v, some, cache)
    assert attn.device_status(clear=True) == 8 and torch.equal(cache, want)
    attn.cache_append_q4(k, v, slots, cache)
    k0, _ = attn.cache_gather_q4(cache, torch.zeros_like(table), sl)
    bad = torch.zeros_like(table)
    bad[0, 1] = cache.shape[0]
    k1, _ = attn.cache_gather_q4(cache, bad, sl)
    assert attn.device_status(clear=True) == 2 and torch.equal(k0[0, :20], k1[0, :20])
    attn.cache_gather_q4(cache, table, _i32([33], gpu))
    assert attn.device_status(clear=True) == 5


# ------------------------------------------------------------------------------------------ decode
def _filled(attn, lens, Hkv, d, seed, dev, gain=None):
    """A filled cache whose rows behind every sequence's end hold garbage (NaN scales among it)."""
    cache, table, sl, k, v, slots = _cache_case(lens, Hkv, d, seed, dev, gain)
    cache[:, :, 16 * d:] = 0xFF                               # every parameter word reads as NaN
    if k.shape[0]:
        attn.cache_append_q4(k, v, slots, cache)
    return cache, table, sl, os_.stored(_np(k)), os_.stored(_np(v))


def _check_decode(o, lse, q, lens, k, v, scale, what=""):
    o, lse, q = _np(o), _np(lse), _np(q)
    Hq, d = q.shape[1:]
    Hkv = k.shape[1] if len(k) else 1
    at = 0
    for n, length in enumerate(lens):
        if length == 0:
            assert (o[n] == 0).all() and np.isneginf(lse[n]).all()
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kk, vv = k[at:at + length, g], v[at:at + length, g]
            s = scale * (kk @ q[n, h])
            m = s.max()
            p = np.exp(s - m)
            want, want_l = p @ vv / p.sum(), m + np.log(p.sum())
            # s_g <= 1.125 * range / 15, with the range at most twice the largest |k| of the group
            step = 1.125 * 2 * np.abs(kk).reshape(length, -1, 64).max((0, 2)) / 15
            B = scale * (step * 31 * np.abs(q[n, h]).reshape(-1, 64).sum(-1)).sum() * 70 * 2.0 ** -23
            terms = 31 * 1.125 * 2 * np.repeat(np.abs(vv).reshape(length, -1, 64).max((0, 2)), 64) / 15
            most = np.repeat(np.abs(vv).reshape(length, -1, 64).max((0, 2)), 64)
            tol = 2.0 ** -8 * np.abs(want) + 2.01 * (B + 2.0 ** -16) * terms + 2.0 ** -12 * most
            err = np.abs(o[n, h] - want)
            assert (err <= tol).all(), f"{what} n={n} h={h}: {(err / tol).max():.3g} of the tolerance"
            assert abs(lse[n, h] - want_l) <= B + 2.0 ** -20 * (1 + abs(want_l)), (what, n, h, lse[n, h], want_l)
        at += length


@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ([1], 1, 1, 64), ([1], 1, 1, 128), ([1], 1, 1, 256), ([2, 15, 16, 17], 4, 2, 64), ([0], 2, 1, 128),
    ([0, 33, 0, 0, 1], 8, 2, 128), ([127, 128, 129, 130], 8, 8, 128), ([1009], 32, 8, 128), ([1000, 3], 5, 1, 128),
    ([300, 77], 16, 2, 256), ([4100], 8, 1, 256), ([500], 11, 1, 64), ([700, 20], 32, 2, 128), ([90], 17, 1, 256),
    ([60] * 40, 4, 2, 128), ([5] * 700, 2, 1, 64), ([9000, 1, 250], 6, 2, 64), ([20000], 4, 1, 128),
    ([40000, 100, 30000], 16, 4, 64), ([30000, 20001], 8, 2, 128), ([9000] * 9, 8, 1, 128), ([20000], 8, 4, 256),
])
def test_decode_q4(attn, gpu, lens, Hq, Hkv, d):
    cache, table, sl, k, v = _filled(attn, lens, Hkv, d, 3 + d, gpu)
    q = _randn((len(lens), Hq, d), 7, gpu)
    scale = 1 / math.sqrt(d)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    start.record()
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 500                      # no wait ran into its limit of 2 s
    _check_decode(o, lse, q, lens, k, v, scale, f"{lens[:4]} {Hq}/{Hkv} d={d}")
    again, lse2 = attn.decode_paged_q4(q, cache, table, sl)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    only, none = attn.decode_paged_q4(q, cache, table, sl, return_lse=False)
    assert none is None and torch.equal(only, o)


def test_decode_q4_peaked_and_growing_scores(attn, gpu):
    """Large score ranges: the running maximum moves late, by much, and differently for each head."""
    d, L = 128, 3000
    cache, table, sl, k, v, slots = _cache_case([L], 2, d, 21, gpu)
    k = (k.float() * torch.linspace(0.1, 6, L, device=gpu)[:, None, None]).to(torch.bfloat16)
    attn.cache_append_q4(k, v, slots, cache)
    q = _randn((1, 8, d), 22, gpu, 3.0)
    o, lse = attn.decode_paged_q4(q, cache, table, sl, scale=0.25)
    _check_decode(o, lse, q, [L], os_.stored(_np(k)), os_.stored(_np(v)), 0.25, "growing")


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 1, 128), (8, 2, 128), (2, 2, 256), (5, 1, 256)])
@pytest.mark.parametrize("which", ["growing", "shrinking", "zeros", "groups", "largest", "smallest", "one_sided"])
def test_decode_q4_value_ranges(attn, gpu, which, Hq, Hkv, d):
    """Scales of V that change along a sequence, that differ between the groups of a token, and at both ends of
    the type's range.  Every group is held to its own scales."""
    lens = [2500, 35]
    cache, table, sl, k, v, slots = _cache_case(lens, Hkv, d, 61, gpu)
    T = v.shape[0]
    at = torch.arange(T, device=gpu, dtype=torch.float64) / T
    e = {"growing": 80 * at - 40, "shrinking": 40 - 80 * at, "largest": 0 * at + 122, "smallest": 0 * at - 118}
    if which in e:
        v = (v.double() * torch.exp2(torch.floor(e[which]))[:, None, None]).to(torch.bfloat16)
    elif which == "zeros":
        v[(torch.arange(T, device=gpu) // 48) % 2 == 0] = 0
    elif which == "groups":
        v = (v.double() * torch.exp2(60.0 - 40 * (torch.arange(d, device=gpu) // 64).double())).to(torch.bfloat16)
    else:
        v = v.abs()
    assert torch.isfinite(v).all()
    attn.cache_append_q4(k, v, slots, cache)
    q = _randn((2, Hq, d), 62, gpu)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    _check_decode(o, lse, q, lens, os_.stored(_np(k)), os_.stored(_np(v)), 1 / math.sqrt(d), which)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 1, 128), (8, 2, 128), (2, 2, 256), (5, 1, 256)])
@pytest.mark.parametrize("later", [None, -110, 3])
def test_decode_q4_subnormal_scales(attn, gpu, later, Hq, Hkv, d):
    """V whose scales all lie below 2^-126, or do so at first.  With queries of zero every probability is 1, x = s
    times a power of two is an fp16 number and a share's sums are of integers below 2^24, so that the output is off
    by its own rounding (2^-8 relative, 2^-134 below 2^-126) and by the merge of up to 80 partials in 32 bits (under
    2^-16).  Where larger scales follow, x of the small ones is off by 2^-31 of the largest: 15 of that at a token."""
    lens = [2500, 35, 3]
    cache, table, sl, k, v, slots = _cache_case(lens, Hkv, d, 65, gpu)
    v = v.double().abs() * 2.0 ** -128
    if later is not None:
        v[700:2500] *= 2.0 ** (later + 128)
    v = v.to(torch.bfloat16)
    attn.cache_append_q4(k, v, slots, cache)
    q = torch.zeros((3, Hq, d), dtype=torch.bfloat16, device=gpu)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    stored, scales = os_.stored(_np(v)), os_.quantise(_np(v))[1]
    at = 0
    for n, length in enumerate(lens):
        most = scales[at:at + length].max()
        assert most > 0 and (later is not None and n == 0 or most < 2.0 ** -126)
        want = stored[at:at + length].mean(0).repeat(Hq // Hkv, 0)
        tol = 2.0 ** -134 + (2.0 ** -8 + 2.0 ** -16) * want + (15 * 2.0 ** -31 * most if most >= 2.0 ** -120 else 0)
        assert (np.abs(_np(o[n]) - want) <= tol).all() and (want > 0).mean() > 0.9
        at += length
    assert np.abs(_np(lse) - np.log(lens)[:, None]).max() <= 2.0 ** -18
    # and with ordinary queries
    q = _randn((3, Hq, d), 66, gpu)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    _check_decode(o, lse, q, lens, os_.stored(_np(k)), stored, 1 / math.sqrt(d), "subnormal")


def test_decode_q4_huge_values_behind_other_values(attn, gpu):
    """A NaN page, then ordinary ones: only the NaN's group of channels is lost, whatever comes after it."""
    d, L = 256, 900
    cache, table, sl, k, v, slots = _cache_case([L], 1, d, 63, gpu)
    v[3, 0, 200] = float("inf")
    attn.cache_append_q4(k, v, slots, cache)
    q = _randn((1, 4, d), 64, gpu)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    assert torch.isnan(o[..., 192:]).all() and torch.isfinite(lse).all()
    v[3, 0, 200] = 0
    clean = torch.zeros_like(cache)
    attn.cache_append_q4(k, v, slots, clean)
    want, _ = attn.decode_paged_q4(q, clean, table, sl)
    assert torch.equal(o[..., :192], want[..., :192])


@pytest.mark.parametrize("seed", range(6))
def test_decode_q4_cut_anywhere(attn, gpu, seed):
    """Many lengths from nothing to a few pages beside long ones: shares begin and end at every kind of place."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, [40, 200, 40, 1000, 3, 5000][seed], [30, 90, 700, 25, 1100, 9][seed]).tolist()
    Hq, Hkv, d = [(4, 2, 64), (16, 2, 128), (2, 2, 64), (8, 1, 256), (3, 1, 64), (18, 2, 128)][seed]
    cache, table, sl, k, v = _filled(attn, lens, Hkv, d, 70 + seed, gpu)
    q = _randn((len(lens), Hq, d), 80 + seed, gpu)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    _check_decode(o, lse, q, lens, k, v, 1 / math.sqrt(d), str(seed))


def test_decode_q4_agrees_with_the_bf16_cache(attn, gpu):
    """The same values read back to a bf16 cache and decoded there."""
    lens, Hq, Hkv, d = [5, 700, 64, 1333], 16, 4, 128
    cache, table, sl, k, v = _filled(attn, lens, Hkv, d, 31, gpu)
    q = _randn((len(lens), Hq, d), 32, gpu)
    kb, vb = (torch.zeros((len(lens), table.shape[1] * PAGE, Hkv, d), dtype=torch.bfloat16, device=gpu) for _ in "kv")
    attn.cache_gather_q4(cache, table, sl, k_out=kb, v_out=vb)
    ident = torch.arange(table.numel(), dtype=torch.int32, device=gpu).view_as(table)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    ob, lb = attn.decode_paged(q, kb.view(-1, PAGE, Hkv, d), vb.view(-1, PAGE, Hkv, d), ident, sl)
    _check_decode(o, lse, q, lens, k, v, 1 / math.sqrt(d))
    # the bf16 decode rounds its probabilities to bf16 (2^-8 relative at most) and both outputs
    assert (np.abs(_np(o) - _np(ob)) <= 2.0 ** -7 * np.abs(_np(ob)) + 2.0 ** -7 * np.abs(v).max()).all()
    assert np.abs(_np(lse) - _np(lb)).max() <= 1e-3


def test_decode_q4_nan_in_a_value_reaches_its_head_only(attn, gpu):
    cache, table, sl, k, v, slots = _cache_case([40], 2, 128, 41, gpu)
    v[7, 1, 70] = float("nan")
    attn.cache_append_q4(k, v, slots, cache)
    q = _randn((1, 4, 128), 42, gpu)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    assert torch.isfinite(o[0, :2]).all() and torch.isfinite(o[0, 2:, :64]).all()
    assert torch.isnan(o[0, 2:, 64:]).all() and torch.isfinite(lse).all()


def test_decode_q4_reports(attn, gpu):
    cache, table, sl, k, v = _filled(attn, [40], 1, 64, 51, gpu)
    q = _randn((1, 2, 64), 52, gpu)
    bad, zero = table.clone(), table.clone()
    bad[0, 1], zero[0, 1] = -1, 0
    cache[0] = 0
    want, _ = attn.decode_paged_q4(q, cache, zero, sl)
    got, _ = attn.decode_paged_q4(q, cache, bad, sl)
    assert attn.device_status(clear=True) == 2 and torch.equal(got, want)
    attn.decode_paged_q4(q, cache, zero, _i32([-4], gpu))
    assert attn.device_status(clear=True) == 3
    with pytest.raises(attn.AttnError):
        attn.decode_paged_q4(q, cache, table, sl, workspace=torch.empty(64, dtype=torch.uint8, device=gpu))


def test_far_pages(attn, gpu):
    """Pages past 2^32 bytes of a cache, and token rows past 2^32 bytes of their tensor."""
    Hkv, d, num_blocks = 8, 256, 130000
    cache = attn.cache_q4_empty(num_blocks, Hkv, d, device=gpu)
    assert cache.numel() > 1 << 32
    pages = [num_blocks - 1, 3, num_blocks - 2, num_blocks - 7]
    L = 50
    rows = torch.empty((L, 1 << 26), dtype=torch.bfloat16, device=gpu)   # 128 MB apart
    k, v = (rows[:, at:at + Hkv * d].unflatten(1, (Hkv, d)) for at in (0, 1 << 25))
    k.copy_(_randn((L, Hkv, d), 91, gpu))
    v.copy_(_randn((L, Hkv, d), 92, gpu))
    slots = _i32([pages[t // PAGE] * PAGE + t % PAGE for t in range(L)], gpu)
    table, sl = _i32([pages], gpu), _i32([L], gpu)
    attn.cache_append_q4(k, v, slots, cache)
    want = [os_.stored(_np(x)) for x in (k, v)]
    got = attn.cache_gather_q4(cache, table, sl)
    assert all((_np(g[0, :L]) == w).all() for g, w in zip(got, want))
    q = _randn((1, Hkv, d), 93, gpu)
    o, lse = attn.decode_paged_q4(q, cache, table, sl)
    _check_decode(o, lse, q, [L], *want, 1 / math.sqrt(d), "far")
    kc, vc = (torch.zeros((20, PAGE, Hkv, d), dtype=torch.bfloat16, device=gpu) for _ in "kv")
    _, kn = attn.qk_norm_rope(v, k, None, None, v=v, k_cache=kc, v_cache=vc, slots=_i32(list(range(L)), gpu),
                              k_out=torch.empty_like(rows)[:, :Hkv * d].unflatten(1, (Hkv, d)))
    assert torch.equal(kn, k) and torch.equal(kc.view(-1, Hkv, d)[:L], k) and torch.equal(vc.view(-1, Hkv, d)[:L], v)
    assert attn.device_status(clear=True) == 0


# ------------------------------------------------------------------------------------------ prefill
@pytest.mark.parametrize("ctx,new,Hq,Hkv,d", [
    ([1], [1], 1, 1, 64), ([130, 40], [130, 3], 4, 2, 128), ([500, 16, 257], [100, 0, 257], 8, 2, 128),
    ([300, 1], [17, 1], 3, 1, 64), ([400], [129], 4, 1, 256),
])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_q4(attn, gpu, ctx, new, Hq, Hkv, d, causal):
    cache, table, sl, k, v = _filled(attn, ctx, Hkv, d, 61 + d, gpu)
    T = sum(new)
    q = _randn((T, Hq, d), 62, gpu)
    cu = _i32(np.concatenate([[0], np.cumsum(new)]).tolist(), gpu)
    o, lse = attn.prefill_paged_q4(q, cache, table, cu, sl, max(new), causal=causal)
    # reading back loses nothing: the prefill over a bf16 cache of the same values gives the same bits
    kb, vb = (torch.zeros((len(ctx), table.shape[1] * PAGE, Hkv, d), dtype=torch.bfloat16, device=gpu) for _ in "kv")
    attn.cache_gather_q4(cache, table, sl, k_out=kb, v_out=vb)
    ident = torch.arange(table.numel(), dtype=torch.int32, device=gpu).view_as(table)
    ob, lb = attn.prefill_paged(q, kb.view(-1, PAGE, Hkv, d), vb.view(-1, PAGE, Hkv, d), ident, cu, sl, max(new),
                                causal=causal)
    assert torch.equal(o, ob) and torch.equal(lse, lb)
    want, want_l = oa.prefill_paged(q.cpu(), kb.view(-1, PAGE, Hkv, d).cpu(), vb.view(-1, PAGE, Hkv, d).cpu(),
                                    ident.cpu(), cu.cpu(), sl.cpu(), 1 / math.sqrt(d), causal)
    # probabilities and output are each rounded to bf16: 2^-8 of the value and of the largest |v|
    assert (np.abs(_np(o) - want) <= 2.0 ** -8 * np.abs(want) + 1.1 * 2.0 ** -8 * np.abs(v).max()).all()
    assert np.abs(_np(lse) - want_l).max() <= 1e-3


@pytest.mark.parametrize("fill", [0xFF, 0x7F, 0x00])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,d", [([0, 40, 0, 129], [0, 3, 0, 129], 4, 2, 128), ([17, 0, 200], [1, 0, 70], 3, 1, 64)])
def test_prefill_q4_takes_nothing_from_its_workspace(attn, gpu, ctx, new, Hq, Hkv, d, fill):
    """What a workspace held before (NaN, page numbers out of range) reaches no result; sequences without tokens."""
    cache, table, sl, k, v = _filled(attn, ctx, Hkv, d, 67, gpu)
    wide = torch.full((len(ctx), table.shape[1] + 9), -1, dtype=torch.int32, device=gpu)
    for n, length in enumerate(ctx):
        wide[n, :_pages(length)] = table[n, :_pages(length)]
    q = _randn((sum(new), Hq, d), 68, gpu)
    cu = _i32(np.concatenate([[0], np.cumsum(new)]).tolist(), gpu)
    need = attn.prefill_q4_workspace_bytes(len(ctx), Hkv, d, wide.shape[1])
    ws = torch.full((need,), fill, dtype=torch.uint8, device=gpu)
    o, lse = attn.prefill_paged_q4(q, cache, wide, cu, sl, max(new), workspace=ws)
    at = kat = 0
    for length, rows in zip(ctx, new):
        if rows == 0:
            kat += length
            continue
        want = _attend(_np(q[at:at + rows]), k[kat:kat + length], v[kat:kat + length], 1 / math.sqrt(d))
        err = np.abs(_np(o[at:at + rows]) - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + 1.1 * 2.0 ** -8 * np.abs(v).max()).all()
        at, kat = at + rows, kat + length
    assert torch.isfinite(lse).all()


# ------------------------------------------------------------------------------------------ together
def _attend(q, k, v, scale):
    """q [R, Hq, d] at the last R positions of k, v [L, Hkv, d], causal."""
    R, Hq, d = q.shape
    L, Hkv = k.shape[:2]
    o = np.zeros(q.shape)
    for h in range(Hq):
        s = scale * q[:, h] @ k[:, h // (Hq // Hkv)].T
        s[np.arange(L)[None] > np.arange(L - R, L)[:, None]] = -np.inf
        p = np.exp(s - s.max(-1, keepdims=True))
        o[:, h] = p @ v[:, h // (Hq // Hkv)] / p.sum(-1, keepdims=True)
    return o


@pytest.mark.parametrize("four_bit", [False, True])
def test_a_serving_run(attn, gpu, four_bit):
    """Prompts in chunks, then single tokens, with tables, norm, rotation, cache write and attention of the
    library; each step's output against float64 attention over what the cache holds."""
    N, Hq, Hkv, d, num_blocks, width = 3, 8, 2, 128, 64, 12
    scale = 1 / math.sqrt(d)
    table = attn.rope_table(4096, d, device=gpu)
    w = (1 + 0.1 * torch.randn(2, d, generator=torch.Generator().manual_seed(0))).to(torch.bfloat16).to(gpu)
    cos, sin = (f(os_.rope_angles(np.arange(4096), d, 10000.0)) for f in (np.cos, np.sin))
    free = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(gpu)
    bt = torch.zeros((N, width), dtype=torch.int32, device=gpu)
    cached = torch.zeros(N, dtype=torch.int32, device=gpu)
    kc, vc = (torch.zeros((num_blocks, PAGE, Hkv, d), dtype=torch.bfloat16, device=gpu) for _ in "kv")
    cache = attn.cache_q4_empty(num_blocks, Hkv, d, device=gpu)
    past = [[np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))] for _ in range(N)]
    for step, new in enumerate([[40, 17, 0], [30, 1, 100], [1, 1, 1], [1, 1, 1], [1, 0, 1]]):
        T = sum(new) + 2                                      # two padded rows
        qkv = _randn((T, (Hq + 2 * Hkv) * d), 100 + step, gpu)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        new_t = _i32(new, gpu)
        tb = attn.step_tables(cached, new_t, free, bt, T, num_blocks)
        free = free[int(tb.pages_used):]
        pos = tb.positions.cpu().numpy()
        kn, k_size = os_.norm_rope(_np(k), _np(w[1]), 1e-6, cos[pos], sin[pos], False)
        if four_bit:
            qr, kr = attn.qk_norm_rope(q, k, tb.positions, table, w[0], w[1])
            attn.cache_append_q4(kr, v, tb.slots, cache)
            keep = lambda x: os_.stored(_np(x))  # noqa: E731
        else:
            kr = torch.empty((T, Hkv, d), dtype=torch.bfloat16, device=gpu)
            qr, _ = attn.qk_norm_rope(q, k, tb.positions, table, w[0], w[1], v=v, k_cache=kc, v_cache=vc,
                                      slots=tb.slots, k_out=kr)
            keep = _np
        _check_rope(kr, k, w[1], 1e-6, cos[pos], sin[pos], False, "k")
        cu = tb.cu_seqlens
        if max(new) > 1:
            o = (attn.prefill_paged_q4(qr, cache, bt, cu, tb.seq_lens, max(new)) if four_bit else
                 attn.prefill_paged(qr, kc, vc, bt, cu, tb.seq_lens, max(new)))[0]
            rows = [range(int(cu[n]), int(cu[n + 1])) for n in range(N)]
        else:
            sq = torch.zeros((N, Hq, d), dtype=torch.bfloat16, device=gpu)
            live = [n for n in range(N) if new[n]]
            sq[live] = qr[:len(live)]
            o = (attn.decode_paged_q4(sq, cache, bt, tb.seq_lens) if four_bit else
                 attn.decode_paged(sq, kc, vc, bt, tb.seq_lens, num_splits=0))[0]
            rows = [range(n, n + 1) if new[n] else range(0) for n in range(N)]
        for n in range(N):
            mine = slice(int(cu[n]), int(cu[n + 1]))
            past[n][0] = np.concatenate([past[n][0], keep(kr[mine])])
            past[n][1] = np.concatenate([past[n][1], keep(v[mine])])
            assert int(tb.seq_lens[n]) == len(past[n][0])
            if new[n]:
                want = _attend(_np(qr[mine]), past[n][0], past[n][1], scale)
                got = _np(o)[list(rows[n])]
                # probabilities (2^-8 at most) and output rounded to bf16
                assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1.1 * 2.0 ** -8 * np.abs(past[n][1]).max()).all()
        cached = tb.seq_lens.clone()


@pytest.mark.parametrize("d", [64, 256])
def test_a_step_without_tokens(attn, gpu, d):
    """No request brings a token: every call of the step passes, and nothing changes.  Wrong arguments are
    refused all the same."""
    N, Hq, Hkv, num_blocks = 2, 4, 2, 6
    cached, bt = _i32([20, 5], gpu), _i32([[3, 1, 0], [2, 0, 0]], gpu)
    cache = torch.randint(0, 256, (num_blocks, Hkv, 17 * d), dtype=torch.uint8, device=gpu)
    kc, vc = _randn((num_blocks, PAGE, Hkv, d), 1, gpu), _randn((num_blocks, PAGE, Hkv, d), 2, gpu)
    before = [x.clone() for x in (bt, cache, kc, vc)]
    tb = attn.step_tables(cached, _i32([0, 0], gpu), _i32([4, 5], gpu), bt, 0, num_blocks)
    assert tb.seq_lens.tolist() == [20, 5] and tb.cu_seqlens.tolist() == [0, 0, 0] and int(tb.pages_used) == 0
    q, k, v = (x.unflatten(1, (-1, d)) for x in
               torch.empty((0, (Hq + 2 * Hkv) * d), dtype=torch.bfloat16, device=gpu).split([Hq * d, Hkv * d, Hkv * d], 1))
    table, w = attn.rope_table(32, d, device=gpu), torch.ones(d, dtype=torch.bfloat16, device=gpu)
    qr, kr = attn.qk_norm_rope(q, k, tb.positions, table, w, w)
    assert qr.shape == (0, Hq, d) and kr.shape == (0, Hkv, d)
    qr, none = attn.qk_norm_rope(q, k, tb.positions, table, w, w, v=v, k_cache=kc, v_cache=vc, slots=tb.slots)
    assert qr.shape == (0, Hq, d) and none is None
    attn.cache_append_q4(kr, v, tb.slots, cache)
    o, lse = attn.prefill_paged_q4(qr, cache, bt, tb.cu_seqlens, tb.seq_lens, 0)
    assert o.shape == (0, Hq, d) and lse.shape == (Hq, 0)
    assert all(torch.equal(a, b) for a, b in zip((bt, cache, kc, vc), before))
    with pytest.raises(ValueError):
        attn.qk_norm_rope(q, k, tb.positions, table, w[:16], w)
    with pytest.raises(ValueError):
        attn.cache_append_q4(kr, v[:, :1], tb.slots, cache)
    with pytest.raises(ValueError):
        attn.prefill_paged_q4(qr, cache, bt, tb.cu_seqlens[:2], tb.seq_lens, 0)


def test_captured_steps(attn, gpu):
    """Two captured decode steps (tables, norm + rotation, 4-bit write, attention) replayed over new lengths
    and inputs give what eager calls give; each has a workspace of its own."""
    N, Hq, Hkv, d, num_blocks, width = 4, 8, 2, 128, 100, 8
    table = attn.rope_table(512, d, device=gpu)
    w = torch.ones(d, dtype=torch.bfloat16, device=gpu)

    def world(seed):
        g = torch.Generator().manual_seed(seed)
        cache = torch.randint(0, 256, (num_blocks, Hkv, 17 * d), generator=g, dtype=torch.uint8)
        cache[:, :, 16 * d:] = 0x3C                           # scales of 0.0115
        return dict(cached=torch.randint(0, 60, (N,), generator=g).to(torch.int32).to(gpu),
                    new=torch.ones(N, dtype=torch.int32, device=gpu),
                    free=torch.randperm(num_blocks, generator=g)[:50].to(torch.int32).to(gpu),
                    bt=torch.randint(0, num_blocks, (N, width), generator=g).to(torch.int32).to(gpu),
                    qkv=torch.randn((N, (Hq + 2 * Hkv) * d), generator=g).to(torch.bfloat16).to(gpu),
                    cache=cache.to(gpu))

    def step(s, ws=None):
        q, k, v = (x.unflatten(1, (-1, d)) for x in s["qkv"].split([Hq * d, Hkv * d, Hkv * d], 1))
        tb = attn.step_tables(s["cached"], s["new"], s["free"], s["bt"], N, num_blocks)
        qr, kr = attn.qk_norm_rope(q, k, tb.positions, table, w, w)
        attn.cache_append_q4(kr, v, tb.slots, s["cache"])
        return attn.decode_paged_q4(qr, s["cache"], s["bt"], tb.seq_lens, workspace=ws)

    states = [world(1), world(2)]
    step(world(9))                                            # first calls outside a capture
    torch.cuda.synchronize()
    graphs = []
    for s in states:
        ws = torch.empty(attn.decode_q4_workspace_bytes(d), dtype=torch.uint8, device=gpu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(s, ws)
        graphs.append((graph, out, ws))
    streams = [torch.cuda.Stream() for _ in states]
    for seed in (3, 5):
        fresh = [world(seed), world(seed + 1)]
        for s, f in zip(states, fresh):
            for name in s:
                s[name].copy_(f[name])
        torch.cuda.synchronize()
        for (graph, _, _), stream in zip(graphs, streams):    # side by side
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out, _), f, s in zip(graphs, fresh, states):
            o, lse = step(f)
            assert torch.equal(out[0], o) and torch.equal(out[1], lse) and torch.equal(s["cache"], f["cache"])


def test_calls_on_given_streams(attn, gpu):
    """Calls on side streams with everything allocated inside, two at once."""
    cache, table, sl, k, v = _filled(attn, [2000, 900], 2, 128, 71, gpu)
    q = _randn((2, 8, 128), 72, gpu)
    want, want_l = attn.decode_paged_q4(q, cache, table, sl)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in streams:
            got.append(attn.decode_paged_q4(q, cache, table, sl, stream=s))
            torch.full((1 << 20,), float("nan"), device=gpu)  # would reuse a freed workspace
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(l, want_l) for o, l in got)
