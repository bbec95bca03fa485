"""The 8-bit paged cache, attention over it, block selection and attention over selected blocks, against their
definitions in 64 bits (oracle/f8.py).

Tolerances, fixed before the first run.  The cache's codes, scales, bounds and read-back values, and the selected
blocks, are exact.  An attention output is a sum of p v / sum p: rounded to bf16 (2^-8 of it), each p 2^b rounded to
fp16 (2^-11 of |p v|), each score off by at most DOT = (2 d / 16 + 4) 2^-22 of sum |q k| scale (the products' sums of 16
terms and their additions) and the exponential and the sums' rounding by 2^-16, both relative to |p v| and, through
the normaliser, once more.  Log-sum-exp: the score's error, 2^-16, and 2^-22 of its own size (base 2 to e).
"""
import math

import numpy as np
import pytest
import torch

import oracle.f8 as o8

pytestmark = pytest.mark.gpu
PAGE = 16


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _bf16(rng, shape, size=1.0):
    return torch.from_numpy(np.asarray(rng.standard_normal(shape) * size, np.float32)).to(torch.bfloat16)


class Cache:
    """A cache on the GPU and the oracle's pages beside it."""

    def __init__(self, attn, gpu, blocks, Hkv, d, fill=None):
        self.attn, self.gpu, self.Hkv, self.d, self.blocks = attn, gpu, Hkv, d, blocks
        self.rec = attn.cache_f8_empty(blocks, Hkv, d, device=gpu)
        self.bounds = attn.key_bounds_empty(blocks, Hkv, d, device=gpu)
        if fill is not None:              # what no token was written to is not to be used
            self.rec.fill_(fill)
            self.bounds.fill_(float("nan"))
        self.pages = {}

    def page(self, p, h, v):
        return self.pages.setdefault((p, h, v), o8.Page(self.d))

    def append(self, k, v, slots, **kw):
        self.attn.cache_append_f8(k.to(self.gpu), v.to(self.gpu), torch.tensor(slots, dtype=torch.int32, device=self.gpu),
                                  self.rec, bounds=self.bounds, **kw)
        self.note(k, v, slots)

    def note(self, k, v, slots):
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        i = 0
        while i < len(slots):
            j = i + 1
            while slots[i] >= 0 and j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] % PAGE != 0:
                j += 1
            if 0 <= slots[i] < self.blocks * PAGE:
                for h in range(self.Hkv):
                    for x, is_v in ((k, 0), (v, 1)):
                        self.page(slots[i] // PAGE, h, is_v).write(slots[i] % PAGE, x[i:j, h])
            i = j

    def check(self, rows_of):
        """Every page's live rows (rows_of: page -> rows) bit for bit."""
        rec, bounds = self.rec.cpu().numpy(), self.bounds.double().cpu().numpy()
        for p, rows in rows_of.items():
            for h in range(self.Hkv):
                for is_v, (codes, scale) in enumerate(o8.read_record(rec[p, h], self.d)):
                    page = self.page(p, h, is_v)
                    assert scale == 2.0 ** page.e, (p, h, is_v)
                    assert np.array_equal(codes[:rows], page.codes[:rows], equal_nan=True), (p, h, is_v)
                page = self.page(p, h, 0)
                assert np.array_equal(bounds[p, h], np.stack([page.lo, page.hi]), equal_nan=True), (p, h)

    def context(self, table, length, h):
        """Keys and values [length, d] of a sequence's KV head."""
        out = []
        for is_v in (0, 1):
            x = [self.page(int(table[i]), h, is_v).values() for i in range(_pages(length))]
            out.append(np.concatenate(x)[:length] if x else np.zeros((0, self.d)))
        return out


def _filled(attn, gpu, rng, lens, Hkv, d, extra=3, width=None, k_size=1.0, v_size=1.0, fill=0xFF):
    """(cache, block table) with sequences of the given lengths on shuffled pages, appended as one batch."""
    need = sum(_pages(n) for n in lens)
    order = rng.permutation(need + extra)
    table = np.zeros((len(lens), width or max(_pages(max(lens)), 1) + 1), np.int32)
    slots, at = [], 0
    for n, length in enumerate(lens):
        table[n, :_pages(length)] = order[at:at + _pages(length)]
        slots += [int(table[n, p // PAGE]) * PAGE + p % PAGE for p in range(length)]
        at += _pages(length)
    c = Cache(attn, gpu, need + extra, Hkv, d, fill)
    if slots:
        T = len(slots)
        c.append(_bf16(rng, (T, Hkv, d), k_size), _bf16(rng, (T, Hkv, d), v_size), slots)
    return c, torch.from_numpy(table)


def _near(o, lse, want, d, where=""):
    """One row's output and log-sum-exp against attend()'s."""
    wo, wl, mass, biggest = want
    dot = (2 * d / 16 + 4) * 2.0 ** -22 * biggest
    tol = 2.0 ** -8 * np.abs(wo) + (2.0 ** -11 + 2 * (dot + 2.0 ** -16)) * mass + 2.0 ** -133
    err = np.abs(o - wo)
    assert (err <= tol).all(), (where, (err / tol).max())
    if math.isinf(wl):
        assert lse == wl, where
    else:
        assert abs(lse - wl) <= dot + 2.0 ** -16 + 2.0 ** -22 * abs(wl), (where, lse, wl)


# ---------------------------------------------------------------------------------------------- the cache
@pytest.mark.parametrize("Hkv,d", [(1, 64), (2, 64), (3, 128), (2, 256), (1, 256)])
def test_append_by_steps(attn, gpu, Hkv, d):
    """Prompts, then tokens one at a time and a few at a time, each larger than what the page held before or not."""
    rng = np.random.default_rng(d + Hkv)
    lens, pages = [0, 0, 0, 0], [[5, 0, 9, 3], [1, 7, 2, 12], [4, 11, 6, 13], [8, 10, 14, 15]]
    c = Cache(attn, gpu, 17, Hkv, d, fill=0xA5)
    live = {}
    for step, new in enumerate([[20, 1, 16, 3], [1, 1, 1, 1], [1, 3, 0, 12], [7, 1, 1, 1], [0, 14, 2, 17], [4, 0, 1, 2]]):
        slots = [-1] if step == 2 else []
        for n, m in enumerate(new):
            slots += [pages[n][p // PAGE] * PAGE + p % PAGE for p in range(lens[n], lens[n] + m)]
            lens[n] += m
        slots += [-1] * (step % 3)
        T = len(slots)
        grow = 2.0 ** rng.integers(-6, 3 + 2 * step, (T, Hkv, 1))
        k, v = (torch.from_numpy((rng.standard_normal((T, Hkv, d)) * grow).astype(np.float32)).to(torch.bfloat16) for _ in "kv")
        c.append(k, v, slots)
        for n in range(4):
            for i in range(_pages(lens[n])):
                live[pages[n][i]] = min(PAGE, lens[n] - i * PAGE)
        c.check(live)
    untouched = [p for p in range(17) if p not in live]
    assert untouched and (c.rec[untouched] == 0xA5).all() and torch.isnan(c.bounds[untouched]).all()


def test_append_begins_a_page_anew_and_takes_rows_back(attn, gpu):
    """A run at row 0 forgets the page's scale and bounds; one further down keeps the rows before it alone."""
    rng = np.random.default_rng(1)
    c = Cache(attn, gpu, 3, 2, 128)
    c.append(_bf16(rng, (16, 2, 128), 1e6), _bf16(rng, (16, 2, 128), 1e6), list(range(16, 32)))
    c.append(_bf16(rng, (4, 2, 128)), _bf16(rng, (4, 2, 128)), list(range(20, 24)))
    c.check({1: 8})
    c.append(_bf16(rng, (3, 2, 128)), _bf16(rng, (3, 2, 128)), [16, 17, 18])
    c.check({1: 3})
    assert c.page(1, 0, 0).e < -4


@pytest.mark.parametrize("d,Hkv,T", [(64, 8, 2500), (128, 8, 1100), (256, 4, 1500), (128, 1, 9000)])
def test_append_of_many_tokens(attn, gpu, d, Hkv, T):
    """Past the size from which a warp looks after 16 tokens: prompts that begin and end inside pages, and single
    tokens on pages of their own."""
    assert T * Hkv * d > 1 << 20
    rng = np.random.default_rng(T)
    lens = [T // 2 - 33, 17, 1, T // 4, 40]
    starts = [0, 5, 0, 9, 15]
    slots, live, page = [], {}, 0
    for n, (start, length) in enumerate(zip(starts, lens)):
        for p in range(start, start + length):
            slots.append((page + p // PAGE) * PAGE + p % PAGE)
        for i in range(_pages(start + length)):
            live[page + i] = min(PAGE, start + length - i * PAGE)
        page += _pages(start + length)
    while len(slots) < T:
        slots += [page * PAGE, -1]
        live[page] = 1
        page += 1
    c = Cache(attn, gpu, page, Hkv, d)
    T = len(slots)
    for p in (i for i, s in enumerate(starts) if s):            # rows before a run that begins inside a page
        first = slots[sum(lens[:p])]
        rows = first % PAGE
        c.append(_bf16(rng, (rows, Hkv, d), 3.0), _bf16(rng, (rows, Hkv, d), 0.1), list(range(first - rows, first)))
    c.append(_bf16(rng, (T, Hkv, d)), _bf16(rng, (T, Hkv, d)), slots)
    some = rng.permutation(page)[:60].tolist() + [0, 1, page - 1] + [slots[sum(lens[:i])] // PAGE for i in range(5)]
    c.check({p: live[p] for p in some})


def test_append_keeps_nan_and_odd_sizes(attn, gpu):
    """NaN, infinities, zeros, the largest and the smallest numbers."""
    rng = np.random.default_rng(5)
    T, Hkv, d = 96, 2, 64
    k = _bf16(rng, (T, Hkv, d))
    k[3, 0, 5], k[20, 1, 7], k[21, 0, 0] = float("nan"), float("inf"), -float("inf")
    k[32:48] = 0
    k[48:64] *= 2.0 ** 120
    k[60, 0, 0] = torch.finfo(torch.bfloat16).max
    k[64:80] = (k[64:80].float() * 2.0 ** -128).to(torch.bfloat16)
    k[80:96] = float("nan")
    v = k.flip(0).contiguous()
    c = Cache(attn, gpu, 6, Hkv, d)
    c.append(k, v, list(range(T)))
    c.check({p: 16 for p in range(6)})
    c.append(k[3:4], v[3:4], [15])        # NaN stays NaN where a page's rows move
    c.append((k[4:5] * 2.0 ** 9), v[4:5] * 2.0 ** 9, [31])
    c.check({p: 16 for p in range(6)})
    ko, vo = attn.cache_gather_f8(c.rec, torch.arange(6, dtype=torch.int32, device=gpu)[None],
                                  torch.tensor([T], dtype=torch.int32, device=gpu))
    for x, is_v in ((ko, 0), (vo, 1)):
        for h in range(Hkv):
            want = np.concatenate([c.page(p, h, is_v).values() for p in range(6)])
            want = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
            assert np.array_equal(x[0, :, h].double().cpu().numpy(), want, equal_nan=True)


def test_append_of_views_without_bounds(attn, gpu):
    """K and V as views of one projection's output; no bounds wanted."""
    rng = np.random.default_rng(6)
    T, Hq, Hkv, d = 37, 4, 2, 128
    qkv = _bf16(rng, (T, (Hq + 2 * Hkv) * d)).to(gpu)
    k, v = (qkv[:, at * d:(at + Hkv) * d].view(T, Hkv, d) for at in (Hq, Hq + Hkv))
    c = Cache(attn, gpu, 3, Hkv, d)
    slots = torch.arange(T, dtype=torch.int32, device=gpu)
    attn.cache_append_f8(k, v, slots, c.rec)
    assert not c.bounds.any()
    c.note(k.cpu(), v.cpu(), list(range(T)))
    other = attn.cache_f8_empty(3, Hkv, d, device=gpu)
    attn.cache_append_f8(k.contiguous(), v.contiguous(), slots, other, bounds=c.bounds)
    assert torch.equal(other, c.rec)
    c.check({0: 16, 1: 16, 2: 5})
    attn.cache_append_f8(k[:0], v[:0], slots[:0], c.rec)     # a step without tokens


def test_append_past_the_last_page_is_recorded(attn, gpu):
    rng = np.random.default_rng(7)
    c = Cache(attn, gpu, 2, 1, 64)
    c.append(_bf16(rng, (4, 1, 64)), _bf16(rng, (4, 1, 64)), [32, 33, 3, 2 ** 31 - 1])
    assert attn.device_status(clear=True) == 8
    rec = c.rec.clone()
    c.check({0: 0})
    assert torch.equal(rec[1], torch.zeros_like(rec[1]))


@pytest.mark.parametrize("lens,Hkv,d", [([1, 16, 0, 33], 2, 64), ([100, 250], 3, 128), ([47], 1, 256)])
def test_gather_leaves_what_is_behind(attn, gpu, lens, Hkv, d):
    rng = np.random.default_rng(d)
    c, table = _filled(attn, gpu, rng, lens, Hkv, d)
    shape = (len(lens), table.shape[1] * PAGE, Hkv, d)
    ko, vo = (torch.full(shape, 7.0, dtype=torch.bfloat16, device=gpu) for _ in "kv")
    attn.cache_gather_f8(c.rec, table.to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu), k_out=ko, v_out=vo)
    for n, length in enumerate(lens):
        assert (ko[n, length:] == 7).all() and (vo[n, length:] == 7).all()
        for h in range(Hkv):
            k, v = c.context(table[n], length, h)
            assert np.array_equal(ko[n, :length, h].double().cpu().numpy(), k)
            assert np.array_equal(vo[n, :length, h].double().cpu().numpy(), v)


def test_pages_and_lengths_out_of_range_are_recorded(attn, gpu):
    rng = np.random.default_rng(8)
    c, table = _filled(attn, gpu, rng, [40, 20], 2, 64)
    bad = table.clone()
    bad[0, 1] = c.blocks
    q = _bf16(rng, (2, 4, 64)).to(gpu)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    every = torch.arange(4, dtype=torch.int32, device=gpu).expand(2, 2, 4).contiguous()
    for tab, lens, want in ((bad, [40, 20], 2), (table, [40, 20000], 5), (table, [-1, 20], 5)):
        attn.cache_gather_f8(c.rec, tab.to(gpu), ints(lens))
        assert attn.device_status(clear=True) == want
        o, _ = attn.decode_paged_f8(q, c.rec, tab.to(gpu), ints(lens))
        assert attn.device_status(clear=True) == (2 if want == 2 else 3)
        attn.decode_blocks_f8(q, c.rec, tab.to(gpu), ints(lens), every)
        assert attn.device_status(clear=True) == (2 if want == 2 else 3)
        attn.select_blocks(q, c.bounds, tab.to(gpu), ints(lens), 2, first=0, last=1)
        assert attn.device_status(clear=True) == want
    for cu in ([0, 1, 5], [0, 2, 1], [-1, 1, 2]):
        attn.decode_blocks_f8(q, c.rec, table.to(gpu), ints([40, 20]), every, cu_seqlens_q=ints(cu))
        assert attn.device_status(clear=True) == 5
        attn.select_blocks(q, c.bounds, table.to(gpu), ints([40, 20]), 2, last=1, cu_seqlens_q=ints(cu), max_seqlen_q=2)
        assert attn.device_status(clear=True) == 5


# ---------------------------------------------------------------------------------------------- attention
def _decode_case(attn, gpu, lens, Hq, Hkv, d, seed, **kw):
    rng = np.random.default_rng(seed)
    c, table = _filled(attn, gpu, rng, lens, Hkv, d, **kw)
    q = _bf16(rng, (len(lens), Hq, d))
    return c, table, q


@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ([1], 1, 1, 64), ([16], 4, 1, 128), ([17], 8, 1, 256), ([0, 1, 15, 16, 17, 31, 32, 33], 8, 2, 128),
    ([0, 0], 4, 2, 64), ([300, 5], 5, 1, 64), ([1009], 32, 8, 128), ([700, 0, 33], 16, 2, 256), ([130, 260], 6, 2, 64),
    ([500], 9, 1, 128), ([64, 63, 65], 32, 2, 64), ([200] * 3, 3, 3, 256), ([2000], 8, 2, 128), ([50] * 40, 4, 1, 64),
    ([1500], 20, 1, 256),
])
def test_decode(attn, gpu, lens, Hq, Hkv, d):
    c, table, q = _decode_case(attn, gpu, lens, Hq, Hkv, d, seed=sum(lens) + d)
    sl = torch.tensor(lens, dtype=torch.int32, device=gpu)
    o, lse = attn.decode_paged_f8(q.to(gpu), c.rec, table.to(gpu), sl)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    every = torch.arange(table.shape[1], dtype=torch.int32, device=gpu).expand(len(lens), Hkv, -1).contiguous()
    ob, lb = attn.decode_blocks_f8(q.to(gpu), c.rec, table.to(gpu), sl, every)
    ob, lb = ob.double().cpu().numpy(), lb.double().cpu().numpy()
    for n, length in enumerate(lens):
        for h in range(Hq):
            k, v = c.context(table[n], length, h // (Hq // Hkv))
            want = o8.attend(q[n, h].double().numpy(), k, v, d ** -0.5)
            _near(o[n, h], lse[n, h], want, d, (n, h))
            _near(ob[n, h], lb[n, h], want, d, ("blocks", n, h))


@pytest.mark.parametrize("q_size,k_size,v_size", [
    (1e-30, 1e30, 1.0), (1e30, 1e-30, 1e-30), (2.0 ** -120, 2.0 ** 115, 2.0 ** 110), (2.0 ** 110, 2.0 ** -112, 2.0 ** -126),
    (1.0, 1.0, 1e37), (5.0, 5.0, 1.0),
])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 7), (256, 2)])
def test_decode_over_the_whole_range(attn, gpu, q_size, k_size, v_size, d, G):
    """Queries, keys and values near either end of bf16's range, whose scores are ordinary numbers."""
    rng = np.random.default_rng(11)
    lens = [70, 19]
    c, table = _filled(attn, gpu, rng, lens, 1, d, k_size=k_size, v_size=v_size)
    q = _bf16(rng, (2, G, d), q_size)
    o, lse = attn.decode_paged_f8(q.to(gpu), c.rec, table.to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu))
    for n in range(2):
        for h in range(G):
            k, v = c.context(table[n], lens[n], 0)
            want = o8.attend(q[n, h].double().numpy(), k, v, d ** -0.5)
            _near(o[n, h].double().cpu().numpy(), float(lse[n, h]), want, d, (n, h))


@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (128, 6), (256, 3)])
def test_values_of_very_different_pages(attn, gpu, d, G):
    """Pages whose values differ by up to 2^80 with weights that make up for it, in either order: what counts in the
    output is what p 2^b is largest for."""
    rng = np.random.default_rng(12)
    for order in (1, -1):
        powers = np.arange(-40, 41, 10)[::order]
        L = PAGE * len(powers)
        k = np.zeros((L, 1, d), np.float32)
        k[:, 0, 0] = -np.repeat(powers, PAGE)                    # weight 2^-power, with q = 1 and scale ln 2
        v = rng.standard_normal((L, 1, d)).astype(np.float32) * np.exp2(np.repeat(powers, PAGE))[:, None, None]
        c = Cache(attn, gpu, len(powers), 1, d)
        c.append(torch.from_numpy(k).to(torch.bfloat16), torch.from_numpy(v).to(torch.bfloat16), list(range(L)))
        q = torch.zeros((1, G, d), dtype=torch.bfloat16)
        q[..., 0] = 1
        table = torch.arange(len(powers), dtype=torch.int32)[None]
        o, lse = attn.decode_paged_f8(q.to(gpu), c.rec, table.to(gpu), torch.tensor([L], dtype=torch.int32, device=gpu),
                                      scale=math.log(2))
        kc, vc = c.context(table[0], L, 0)
        want = o8.attend(q[0, 0].double().numpy(), kc, vc, math.log(2))
        for h in range(G):
            _near(o[0, h].double().cpu().numpy(), float(lse[0, h]), want, d, (order, h))


def test_large_scores_move_the_references(attn, gpu):
    """Scores that rise page by page by hundreds, then fall: only the last of them count."""
    for d, G in ((128, 4), (64, 5), (256, 8)):
        rng = np.random.default_rng(13)
        L = 400
        k = np.zeros((L, 1, d), np.float32)
        k[:, 0, 1] = np.concatenate([np.linspace(-120, 120, 200), np.linspace(120, -120, 200)])
        c = Cache(attn, gpu, 25, 1, d)
        c.append(torch.from_numpy(k).to(torch.bfloat16), _bf16(rng, (L, 1, d)), list(range(L)))
        q = torch.zeros((1, G, d), dtype=torch.bfloat16)
        q[..., 1] = torch.tensor([(-1.0) ** h * (1 + h) for h in range(G)])
        table = torch.arange(25, dtype=torch.int32)[None]
        o, lse = attn.decode_paged_f8(q.to(gpu), c.rec, table.to(gpu), torch.tensor([L], dtype=torch.int32, device=gpu),
                                      scale=4.0)
        kc, vc = c.context(table[0], L, 0)
        for h in range(G):
            _near(o[0, h].double().cpu().numpy(), float(lse[0, h]), o8.attend(q[0, h].double().numpy(), kc, vc, 4.0), d, h)


def test_not_numbers_show(attn, gpu):
    """NaN in a key, a value or a query that counts gives NaN; behind the sequence, or in another, it does not."""
    rng = np.random.default_rng(14)
    lens = [40, 40, 40, 33]
    c, table = _filled(attn, gpu, rng, lens, 1, 128)
    q = _bf16(rng, (4, 4, 128))
    one = _bf16(rng, (1, 1, 128))
    bad = one.clone()
    bad[0, 0, 3] = float("inf")
    c.append(bad, one, [int(table[0, 2]) * PAGE + 7])
    c.append(one, bad, [int(table[1, 2]) * PAGE + 7])
    c.append(bad, bad, [int(table[3, 2]) * PAGE + 1])            # behind the last token
    q[2, 1, 0] = float("nan")
    o, lse = attn.decode_paged_f8(q.to(gpu), c.rec, table.to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu))
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(o[0]).all() and np.isnan(lse[0]).all()
    assert np.isnan(o[1, :, 3]).all() and np.isfinite(np.delete(o[1], 3, -1)).all() and np.isfinite(lse[1]).all()
    assert np.isnan(o[2, 1]).all() and np.isfinite(o[2, [0, 2, 3]]).all()
    assert np.isfinite(o[3]).all()


@pytest.mark.parametrize("rows,lens,Hq,Hkv,d,K", [
    ([1, 1, 1], [100, 5, 1000], 8, 2, 128, 7), ([3, 0, 1, 6], [50, 9, 17, 400], 4, 1, 64, 5),
    ([2, 5], [300, 33], 16, 2, 256, 12), ([8], [129], 5, 1, 128, 1), ([4, 4], [64, 700], 10, 2, 64, 40), ([1], [1], 1, 1, 256, 3),
    ([40], [640], 4, 4, 128, 9),
])
def test_decode_blocks(attn, gpu, rows, lens, Hq, Hkv, d, K):
    """Blocks in any order, some absent (-1), some past the row, one named twice; rows without a sequence behind."""
    rng = np.random.default_rng(K + d)
    c, table = _filled(attn, gpu, rng, lens, Hkv, d)
    cu = np.concatenate([[0], np.cumsum(rows)])
    T = int(cu[-1]) + 3
    q = _bf16(rng, (T, Hq, d))
    blocks = rng.integers(-1, table.shape[1] + 2, (T, Hkv, K)).astype(np.int32)
    blocks[0, 0, :] = -1                                          # a row that sees nothing
    o = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device=gpu)
    lse = torch.full((T, Hq), 7.0, device=gpu)
    attn.decode_blocks_f8(q.to(gpu), c.rec, table.to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu),
                          torch.from_numpy(blocks).to(gpu), cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device=gpu),
                          out=o, lse=lse)
    assert (o[T - 3:] == 7).all() and (lse[T - 3:] == 7).all()
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for n in range(len(rows)):
        for r in range(cu[n], cu[n + 1]):
            seen = lens[n] - (cu[n + 1] - 1 - r)
            for h in range(Hq):
                kk, vv = c.context(table[n], lens[n], h // (Hq // Hkv))
                at = [t for b in blocks[r, h // (Hq // Hkv)] for t in range(b * PAGE, b * PAGE + PAGE) if b >= 0 and t < seen]
                _near(o[r, h], lse[r, h], o8.attend(q[r, h].double().numpy(), kk[at], vv[at], d ** -0.5), d, (r, h))


@pytest.mark.parametrize("rows,lens,Hq,Hkv,d,causal", [
    ([5, 40], [100, 40], 8, 2, 128, True), ([130], [300], 4, 1, 64, True), ([17, 3], [17, 64], 4, 2, 256, False),
])
def test_prefill(attn, gpu, rows, lens, Hq, Hkv, d, causal):
    """Against the bf16 prefill over the values read back, which it is, and the definition (its own tolerance)."""
    rng = np.random.default_rng(sum(rows))
    c, table = _filled(attn, gpu, rng, lens, Hkv, d)
    cu = np.concatenate([[0], np.cumsum(rows)])
    q = _bf16(rng, (int(cu[-1]), Hq, d)).to(gpu)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    o, lse = attn.prefill_paged_f8(q, c.rec, table.to(gpu), ints(cu), ints(lens), max(rows), causal=causal)
    k, v = (x.nan_to_num(0) for x in attn.cache_gather_f8(c.rec, table.to(gpu), ints(lens)))
    for n in range(len(lens)):
        k[n, lens[n]:], v[n, lens[n]:] = 0, 0
    pages = torch.arange(table.numel(), dtype=torch.int32, device=gpu).view(table.shape)
    wo, wl = attn.prefill_paged(q, k.view(-1, PAGE, Hkv, d), v.view(-1, PAGE, Hkv, d), pages, ints(cu), ints(lens), max(rows),
                                causal=causal)
    assert torch.equal(o, wo) and torch.equal(lse, wl)
    for n in range(len(rows)):
        for r in (cu[n], cu[n + 1] - 1):
            seen = lens[n] - (cu[n + 1] - 1 - r) if causal else lens[n]
            for h in range(Hq):
                kk, vv = c.context(table[n], lens[n], h // (Hq // Hkv))
                want = o8.attend(q[r, h].double().cpu().numpy(), kk[:seen], vv[:seen], d ** -0.5)
                assert np.abs(o[r, h].double().cpu().numpy() - want[0]).max() <= 2e-2
                assert abs(float(lse[h, r]) - want[1]) <= 1e-3


# ---------------------------------------------------------------------------------------------- selection
def _bounds(rng, blocks, Hkv, d, size=1.0):
    x = np.sort(rng.standard_normal((blocks, Hkv, 2, d)) * size, axis=2)
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def _check_selection(attn, gpu, q, bounds, table, rows, lens, K, first, last, pad=0, cu_given=True, max_q=None):
    T, Hq, d = q.shape
    Hkv = bounds.shape[1]
    cu = np.concatenate([[0], np.cumsum(rows)])
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    out = torch.full((T, Hkv, K), -7, dtype=torch.int32, device=gpu)
    kw = dict(cu_seqlens_q=ints(cu), max_seqlen_q=max_q or max(max(rows), 1)) if cu_given else {}
    attn.select_blocks(q.to(gpu), bounds.to(gpu), table.to(gpu), ints(lens), K, first=first, last=last, out=out, **kw)
    got = out.cpu().numpy()
    assert (got[cu[-1]:] == -7).all()
    b, qd = bounds.double().numpy(), q.double().numpy()
    with np.errstate(invalid="ignore"):
        for n in range(len(rows)):
            for r in range(cu[n], cu[n + 1]):
                nb = max(0, _pages(lens[n] - (cu[n + 1] - 1 - r)))
                for h in range(Hkv):
                    lo, hi = (b[table[n, :nb].numpy(), h, i] for i in (0, 1))
                    G = Hq // Hkv
                    want = o8.select(o8.scores(qd[r, h * G:(h + 1) * G], lo, hi), K, first, last)
                    assert np.array_equal(got[r, h], want), (n, r, h, got[r, h], want)


def _table(rng, lens, spare=0):
    need = [_pages(n) for n in lens]
    order = rng.permutation(sum(need) + 2)
    t = np.zeros((len(lens), max(max(need), 1) + spare), np.int32)
    at = 0
    for n, m in enumerate(need):
        t[n, :m] = order[at:at + m]
        at += m
    return torch.from_numpy(t), sum(need) + 2


@pytest.mark.parametrize("rows,lens,Hq,Hkv,d,K,first,last,spare", [
    ([1] * 4, [1, 100, 1000, 5000], 8, 2, 128, 8, 1, 2, 0), ([1], [40000], 4, 1, 64, 100, 0, 1, 3),
    ([1, 1], [3000, 2999], 16, 2, 256, 33, 2, 3, 1), ([5, 1, 0, 3], [700, 700, 20, 16], 5, 1, 128, 6, 1, 1, 300),
    ([40, 33], [900, 2000], 8, 2, 64, 20, 1, 2, 0), ([70], [1300], 4, 2, 256, 16, 0, 2, 0), ([3], [500], 2, 1, 128, 1, 0, 1, 0),
    ([4], [640], 3, 3, 128, 3, 1, 2, 0), ([1], [160], 1, 1, 64, 9, 0, 1, 0), ([1] * 3, [170, 0, 16], 64, 1, 64, 10, 4, 6, 0),
    ([33], [200000], 4, 1, 64, 512, 1, 2, 0),
])
def test_select(attn, gpu, rows, lens, Hq, Hkv, d, K, first, last, spare):
    rng = np.random.default_rng(sum(lens))
    table, blocks = _table(rng, lens, spare)
    T = sum(rows) + 2
    q, bounds = _bf16(rng, (T, Hq, d)), _bounds(rng, blocks, Hkv, d)
    _check_selection(attn, gpu, q, bounds, table, rows, lens, K, first, last)
    if max(rows) == 1 == min(rows):
        _check_selection(attn, gpu, q[:-2], bounds, table, rows, lens, K, first, last, cu_given=False)


@pytest.mark.parametrize("d,Hkv", [(64, 1), (128, 2), (256, 1)])
def test_select_at_the_border(attn, gpu, d, Hkv):
    """Scores that float32 cannot tell apart, alike and with differences of 2^-28 of their size in one channel; few of
    them, and more than the kernel keeps at hand."""
    for alike in (20, 700):
        rng = np.random.default_rng(alike)
        lens = [16 * 900]
        table, blocks = _table(rng, lens)
        bounds = _bounds(rng, blocks, Hkv, d)
        q = _bf16(rng, (1, 4 * Hkv, d))
        q[..., 0] = 2.0 ** -20
        best = bounds[int(table[0, 450])].clone()
        best[:, 1] += 2                                            # above all others
        which = 100 + rng.permutation(750)[:alike]
        for i, blk in enumerate(which):
            b = best.clone()
            b[:, 1, 0] = 2.0 + (i % 5) * 2.0 ** -6                 # five scores, each many times
            bounds[int(table[0, blk])] = b
        for K in (5, 14, 3 + alike // 2, alike + 2, alike + 40):
            _check_selection(attn, gpu, q, bounds, table, [1], lens, K, 1, 2)


def test_select_where_scores_are_zero_or_tiny(attn, gpu):
    rng = np.random.default_rng(21)
    lens, d = [16 * 800, 16 * 60], 128
    table, blocks = _table(rng, lens)
    bounds = _bounds(rng, blocks, 2, d)
    q = _bf16(rng, (2, 8, d))
    _check_selection(attn, gpu, torch.zeros_like(q), bounds, table, [1, 1], lens, 20, 1, 2)
    _check_selection(attn, gpu, q, torch.zeros_like(bounds), table, [1, 1], lens, 20, 1, 2)
    tiny = (q.float() * 2.0 ** -110).to(torch.bfloat16)
    small = (bounds.float() * 2.0 ** -100).to(torch.bfloat16)
    _check_selection(attn, gpu, tiny, bounds, table, [1, 1], lens, 20, 1, 2)
    _check_selection(attn, gpu, tiny, small, table, [1, 1], lens, 20, 1, 2)
    _check_selection(attn, gpu, q, small, table, [1, 1], lens, 20, 1, 2)
    large = (q.float() * 2.0 ** 100).to(torch.bfloat16)
    wide = (bounds.float() * 2.0 ** 60).to(torch.bfloat16)         # past float32
    _check_selection(attn, gpu, large, wide, table, [1, 1], lens, 20, 1, 2)


def test_select_takes_what_is_not_a_number_first(attn, gpu):
    rng = np.random.default_rng(22)
    lens, d = [16 * 200], 64
    table, blocks = _table(rng, lens)
    bounds = _bounds(rng, blocks, 1, d)
    q = _bf16(rng, (1, 3, d))
    for i, x in ((50, float("nan")), (60, float("inf")), (70, float("nan"))):
        bounds[int(table[0, i]), 0, 1, 5] = x
    for K in (4, 5, 6, 30):
        _check_selection(attn, gpu, q, bounds, table, [1], lens, K, 1, 2)
    q[0, 1, 9] = float("nan")                                      # every score is none: the lowest numbers
    _check_selection(attn, gpu, q, bounds, table, [1], lens, 12, 1, 2)


def test_select_ignores_pages_behind(attn, gpu):
    """Columns of the table behind a sequence's blocks hold anything; pages of other sequences are NaN."""
    rng = np.random.default_rng(23)
    lens, d = [333, 50], 128
    table, blocks = _table(rng, lens, spare=9)
    bounds = _bounds(rng, blocks, 2, d)
    used = {int(x) for n, m in enumerate(lens) for x in table[n, :_pages(m)]}
    for p in range(blocks):
        if p not in used:
            bounds[p] = float("nan")
    table[0, _pages(333):] = 10 ** 6
    table[1, _pages(50):] = -5
    _check_selection(attn, gpu, _bf16(rng, (5, 4, d)), bounds, table, [4, 1], lens, 6, 1, 1, max_q=9)


# ---------------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (5, 1, 64), (4, 2, 256)])
def test_a_serving_run(attn, gpu, Hq, Hkv, d):
    """Prompts, then tokens one at a time: tables, norm and rotation, write with bounds, selection, attention."""
    rng = np.random.default_rng(d)
    N, width, blocks, K = 3, 24, 64, 6
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    free = torch.from_numpy(rng.permutation(blocks).astype(np.int32)).to(gpu)
    table, cached = torch.zeros((N, width), dtype=torch.int32, device=gpu), ints([0] * N)
    rope = attn.rope_table(512, 64 if d == 64 else 128, device=gpu)
    c = Cache(attn, gpu, blocks, Hkv, d, fill=0xFF)
    w = _bf16(rng, (d,)).to(gpu)
    for step, new in enumerate([[200, 37, 16], [1, 1, 1], [1, 0, 1], [3, 1, 12], [1, 1, 1]]):
        T = sum(new)
        st = attn.step_tables(cached, ints(new), free, table, T, blocks)
        free, cached = free[int(st.pages_used):].contiguous(), st.seq_lens
        q, k, v = (_bf16(rng, (T, h, d)).to(gpu) for h in (Hq, Hkv, Hkv))
        q, k = attn.qk_norm_rope(q, k, st.positions, rope, w, w)
        attn.cache_append_f8(k, v, st.slots, c.rec, bounds=c.bounds)
        c.note(k, v, st.slots.tolist())
        lens, cu = st.seq_lens.tolist(), st.cu_seqlens.tolist()
        picked = attn.select_blocks(q, c.bounds, table, st.seq_lens, K, cu_seqlens_q=st.cu_seqlens, max_seqlen_q=max(new))
        o, lse = attn.decode_blocks_f8(q, c.rec, table, st.seq_lens, picked, cu_seqlens_q=st.cu_seqlens)
        full, fl = attn.prefill_paged_f8(q, c.rec, table, st.cu_seqlens, st.seq_lens, max(new))
        if max(new) == 1 and min(new) == 1:
            one, ol = attn.decode_paged_f8(q, c.rec, table, st.seq_lens)
        b, picked, qd = c.bounds.double().cpu().numpy(), picked.cpu().numpy(), q.double().cpu().numpy()
        for n in range(N):
            for r in range(cu[n], cu[n + 1]):
                seen = lens[n] - (cu[n + 1] - 1 - r)
                if step == 0 and seen % 13:
                    continue                                        # some of a prompt's rows
                for h in range(Hq):
                    kvh = h // (Hq // Hkv)
                    pages = table[n, :_pages(seen)].cpu().numpy()
                    sc = o8.scores(qd[r, kvh * (Hq // Hkv):(kvh + 1) * (Hq // Hkv)], b[pages, kvh, 0], b[pages, kvh, 1])
                    assert np.array_equal(picked[r, kvh], o8.select(sc, K, 1, 2)), (step, r, h)
                    kk, vv = c.context(table[n].cpu(), seen, kvh)
                    at = [t for x in picked[r, kvh] if x >= 0 for t in range(x * PAGE, min(seen, x * PAGE + PAGE))]
                    _near(o[r, h].double().cpu().numpy(), float(lse[r, h]), o8.attend(qd[r, h], kk[at], vv[at], d ** -0.5), d, (step, r, h))
                    want = o8.attend(qd[r, h], kk, vv, d ** -0.5)
                    assert np.abs(full[r, h].double().cpu().numpy() - want[0]).max() <= 2e-2
                    if max(new) == 1 and min(new) == 1:
                        _near(one[r, h].double().cpu().numpy(), float(ol[r, h]), want, d, (step, r, h))


def test_a_captured_step_is_replayed(attn, gpu):
    """Write, selection and both decodes in a graph, with lengths that grow between replays; two graphs in turn."""
    rng = np.random.default_rng(31)
    N, Hq, Hkv, d, K, width, blocks = 3, 8, 2, 128, 5, 20, 70
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    lens = [100, 15, 250]
    c, table = _filled(attn, gpu, rng, lens, Hkv, d, extra=blocks - sum(_pages(x) for x in lens), width=width)
    table = table.to(gpu)
    free = ints([p for p in range(c.blocks) if p not in {int(x) for n, m in enumerate(lens) for x in table[n, :_pages(m)]}])
    cached, one = ints(lens), ints([1] * N)
    k, v, q = (torch.zeros((N, h, d), dtype=torch.bfloat16, device=gpu) for h in (Hkv, Hkv, Hq))

    def step():
        st = attn.step_tables(cached, one, free, table, N, c.blocks)
        attn.cache_append_f8(k, v, st.slots, c.rec, bounds=c.bounds)
        picked = attn.select_blocks(q, c.bounds, table, st.seq_lens, K)
        return st, picked, attn.decode_blocks_f8(q, c.rec, table, st.seq_lens, picked), attn.decode_paged_f8(
            q, c.rec, table, st.seq_lens)

    attn.decode_f8_workspace_bytes(d, gpu)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(6):
        k.copy_(_bf16(rng, k.shape, 1 + i))
        v.copy_(_bf16(rng, v.shape, 1 + i))
        q.copy_(_bf16(rng, q.shape))
        graphs[i % 2].replay()
        st, picked, (ob, lb), (o, lse) = outs[i % 2]
        slots = st.slots.tolist()
        c.note(k, v, slots)
        b = c.bounds.double().cpu().numpy()
        for n in range(N):
            seen = int(st.seq_lens[n])
            for h in range(Hq):
                kvh = h // 4
                pages = table[n, :_pages(seen)].cpu().numpy()
                sc = o8.scores(q[n, 4 * kvh:4 * kvh + 4].double().cpu().numpy(), b[pages, kvh, 0], b[pages, kvh, 1])
                assert np.array_equal(picked[n, kvh].cpu().numpy(), o8.select(sc, K, 1, 2)), (i, n, h)
                kk, vv = c.context(table[n].cpu(), seen, kvh)
                at = [t for x in picked[n, kvh].tolist() if x >= 0 for t in range(x * PAGE, min(seen, x * PAGE + PAGE))]
                qh = q[n, h].double().cpu().numpy()
                _near(o[n, h].double().cpu().numpy(), float(lse[n, h]), o8.attend(qh, kk, vv, d ** -0.5), d, (i, n, h))
                _near(ob[n, h].double().cpu().numpy(), float(lb[n, h]), o8.attend(qh, kk[at], vv[at], d ** -0.5), d, (i, n, h))
        used = int(st.pages_used)
        free.copy_(free.roll(-used))
        cached.copy_(st.seq_lens)


def test_calls_repeat_bit_for_bit(attn, gpu):
    """No result depends on which CTA comes first."""
    rng = np.random.default_rng(33)
    lens = [3000, 77, 0, 1234]
    c, table = _filled(attn, gpu, rng, lens, 2, 128)
    q = _bf16(rng, (4, 8, 128)).to(gpu)
    sl = torch.tensor(lens, dtype=torch.int32, device=gpu)
    first = None
    for _ in range(5):
        picked = attn.select_blocks(q, c.bounds, table.to(gpu), sl, 9)
        out = (picked, *attn.decode_blocks_f8(q, c.rec, table.to(gpu), sl, picked), *attn.decode_paged_f8(q, c.rec, table.to(gpu), sl))
        first = first or [x.clone() for x in out]
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_refusals_on_the_gpu(attn, gpu):
    c = Cache(attn, gpu, 4, 2, 64)
    i32 = dict(dtype=torch.int32, device=gpu)
    q, bt, sl = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=gpu), torch.zeros((2, 2), **i32), torch.ones(2, **i32)
    blocks = torch.zeros((2, 2, 3), **i32)
    for call in (
        lambda: attn.decode_paged_f8(q.float(), c.rec, bt, sl), lambda: attn.decode_paged_f8(q, c.rec[:, :, :-16], bt, sl),
        lambda: attn.decode_paged_f8(q, c.rec, bt[:1], sl), lambda: attn.decode_paged_f8(q, c.rec, bt.long(), sl),
        lambda: attn.decode_blocks_f8(q, c.rec, bt, sl, blocks[:, :1]), lambda: attn.decode_blocks_f8(q, c.rec, bt, sl, blocks[0]),
        lambda: attn.decode_blocks_f8(q[:1], c.rec, bt, sl, blocks[:1]),
        lambda: attn.decode_blocks_f8(q, c.rec, bt, sl, blocks, cu_seqlens_q=sl),
        lambda: attn.select_blocks(q, c.bounds[:, :, :1], bt, sl, 4), lambda: attn.select_blocks(q, c.bounds.float(), bt, sl, 4),
        lambda: attn.select_blocks(q[:1], c.bounds, bt, sl, 4),
        lambda: attn.select_blocks(q, c.bounds, bt, sl, 4, out=blocks),
        lambda: attn.cache_append_f8(q[:, :2], q[:, :2], sl, c.rec, bounds=c.bounds[:3]),
        lambda: attn.cache_append_f8(q[:, :2], q[:, :2], sl, c.rec[:, :1]),
        lambda: attn.cache_gather_f8(c.rec, bt, sl, k_out=q),
        lambda: attn.prefill_paged_f8(q, c.rec, bt, None, sl, 1),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: attn.select_blocks(q, c.bounds, bt, sl, 2), lambda: attn.select_blocks(q, c.bounds, bt, sl, 4, last=0),
                 lambda: attn.select_blocks(q, c.bounds, bt, sl, 4, max_seqlen_q=2),
                 lambda: attn.decode_blocks_f8(q, c.rec, bt, sl, blocks[..., :0].contiguous()),
                 lambda: attn.decode_paged_f8(q, c.rec, bt, sl, scale=0.0),
                 lambda: attn.decode_paged_f8(q, c.rec, bt, sl, workspace=torch.zeros(64, dtype=torch.uint8, device=gpu))):
        with pytest.raises(attn.AttnError):
            call()
