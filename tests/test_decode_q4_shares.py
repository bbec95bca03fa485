"""Every page of a sequence counts once in the 4-bit decode, wherever its shares are cut and merged.

Each page of 16 tokens puts its values into one channel of its KV head, the next page into the next channel, and so
on round the head dim: an output channel is the weighted mean over one page in d, so that a page that is dropped,
counted twice or put elsewhere moves a channel by far more than a rounding, also in a context of 40000 tokens.  The
values are positive; nothing cancels but the zero point's part.

Weights: all 1 (queries of zero), or 2^-j and 2^-2j with j = 0 .. 6 in every page (keys of -j in one channel, scale
ln 2), which the kernel's p s holds exactly as fp16.

Tolerance, fixed before the first run.  The output is rounded to bf16 (2^-8 relative).  p is off by 2^-20 relative (the
product with scale, ex2), the merges of up to 700 partials by 2^-14: less than 2^-13 of the output in all.  A
sum of x (c - 8) and of x (z - 8), x = p s, takes at most 4 products of 16 tokens a warp with a share of 152 SMs'
work, 17 additions each with up to 2^-23 of the sum of |terms|, 8 x: under 2^-16 of 8 mean(x).
"""
import math

import numpy as np
import pytest
import torch

import oracle.step as os_

PAGE = 16
CASES = [
    ([1009], 32, 8, 128), ([4100], 8, 1, 256), ([20000], 4, 1, 128), ([20000], 8, 4, 256), ([9000, 1, 250], 6, 2, 64),
    ([700, 20], 32, 2, 128), ([1000, 3], 5, 1, 128), ([30000, 20001], 8, 2, 128), ([40000, 100, 30000], 16, 4, 64),
    ([9000] * 9, 8, 1, 128), ([2500] * 7, 16, 1, 64), ([333] * 40, 4, 2, 256), ([5] * 700, 2, 1, 64),
    ([(i * 271) % 199 for i in range(90)], 16, 2, 128), ([(i * 1543) % 4999 for i in range(9)], 18, 2, 128),
    ([122863, 6335], 16, 2, 256),
]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _ids(case):
    lens, Hq, Hkv, d = case
    return f"{len(lens)}x{max(lens)}-{Hq}/{Hkv}-{d}"


class Case:
    """Where each token's value is, what it is, and what comes out."""

    def __init__(self, lens, Hq, Hkv, d, uniform):
        self.lens, self.Hq, self.Hkv, self.d, self.uniform = lens, Hq, Hkv, d, uniform
        self.wanted = {}
        one = np.zeros((16, 64))
        one[:, 0] = np.arange(16)
        self.kept = os_.stored(one)[:, 0]                     # what storage keeps of 0 .. 15 alone in its group
        self.scale_of = os_.quantise(one)[1][:, 0]

    def token(self, n, g):
        """(channel, value 1 .. 15, j) of each token of sequence n, KV head g."""
        t = np.arange(self.lens[n])
        page = t // PAGE
        return (page + 7 * g + 3 * n) % self.d, 1 + (5 * t + g) % 15, (3 * t + page) % 7

    def weights(self, h, j):
        return np.ones(len(j)) if self.uniform else 2.0 ** -((1 + h % 2) * j)

    def parts(self, n, h):
        """Per page: its channel and what it adds to it; the sum of weights; mean(x) of each channel's group."""
        ch, v, j = self.token(n, h // (self.Hq // self.Hkv))
        p = self.weights(h, j)
        at = np.arange(0, len(ch), PAGE)
        x = np.bincount(ch // 64, p * self.scale_of[v], self.d // 64) / p.sum()
        return ch[at], np.add.reduceat(p * self.kept[v], at), p.sum(), np.repeat(x, 64)

    def want(self, n, h):
        if (n, h) not in self.wanted:
            ch, add, total, x = self.parts(n, h)
            o = np.bincount(ch, add, self.d) / total
            self.wanted[n, h] = o, math.log(total), (2.0 ** -8 + 2.0 ** -13) * o + 2.0 ** -16 * 8 * x
        return self.wanted[n, h]

    def check(self, o, lse):
        """o [N, Hq, d], lse [N, Hq]"""
        for n, length in enumerate(self.lens):
            if length == 0:
                assert (o[n] == 0).all() and np.isneginf(lse[n]).all()
                continue
            for h in range(self.Hq):
                self.check_head(o[n, h], lse[n, h], n, h)

    def check_head(self, o, lse, n, h):
        want, want_l, tol = self.want(n, h)
        err = np.abs(o - want)
        assert (err <= tol).all(), f"n={n} h={h} channel {(err - tol).argmax()}: {o[(err - tol).argmax()]}"
        assert abs(lse - want_l) <= 2.0 ** -18 * (1 + abs(want_l)), (n, h, lse, want_l)


def _bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("uniform", [True, False])
@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_the_check_sees_every_page(case, uniform):
    """On the CPU: what the definition gives passes; zeros, and any page that is dropped, doubled or one channel
    off, do not."""
    c = Case(*case, uniform)
    rng = np.random.default_rng(0)
    for n in {0, len(c.lens) - 1, int(np.argmax(c.lens))}:
        if c.lens[n] == 0:
            continue
        for h in {0, c.Hq // 2, c.Hq - 1}:
            ch, add, total, _ = c.parts(n, h)
            o, lse, tol = c.want(n, h)
            c.check_head(_bf16(o), lse, n, h)
            with pytest.raises(AssertionError):
                c.check_head(np.zeros(c.d), lse, n, h)
            with pytest.raises(AssertionError):
                c.check_head(_bf16(o), lse + 2.0 ** -10, n, h)
            # every page moves its channel by more than the tolerance and another rounding
            assert (add / total > tol[ch] + 2.0 ** -8 * (o[ch] + add / total)).all()
            for page in rng.integers(0, len(ch), 20):
                for times, off in ((-1, 0), (1, 0), (-1, 1)):
                    bad = o.copy()
                    bad[ch[page]] += times * add[page] / total
                    if off:
                        bad[(ch[page] + off) % c.d] += add[page] / total
                    with pytest.raises(AssertionError):
                        c.check_head(_bf16(bad), lse, n, h)


@pytest.mark.gpu
@pytest.mark.parametrize("uniform", [True, False])
@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_every_page_counts_once(attn, gpu, case, uniform):
    c = Case(*case, uniform)
    lens, Hq, Hkv, d = case
    T, num_blocks = sum(lens), sum(_pages(n) for n in lens) + 3
    k, v = (torch.zeros((T, Hkv, d), dtype=torch.bfloat16) for _ in "kv")
    perm = np.random.default_rng(1).permutation(num_blocks)
    table = np.full((len(lens), max(1, max(_pages(n) for n in lens))), -1, np.int64)
    slots, at, page = np.zeros(T, np.int64), 0, 0
    for n, length in enumerate(lens):
        mine = perm[page:page + _pages(length)]
        table[n, :len(mine)] = mine
        t = np.arange(length)
        slots[at:at + length] = mine[t // PAGE] * PAGE + t % PAGE if length else 0
        for g in range(Hkv):
            ch, val, j = c.token(n, g)
            v[at + torch.from_numpy(t), g, torch.from_numpy(ch)] = torch.from_numpy(val).to(torch.bfloat16)
            k[at:at + length, g, 0] = torch.from_numpy(-j).to(torch.bfloat16)
        at, page = at + length, page + len(mine)
    k[:, :, 1] = -15.0                                        # the scale of K is 1 and its zero point 15
    q = torch.zeros((len(lens), Hq, d), dtype=torch.bfloat16)
    if not uniform:
        q[:, 0::2, 0], q[:, 1::2, 0] = 1.0, 2.0
    # rows behind a sequence's end, and pages of no sequence, hold NaN scales
    cache = torch.full((num_blocks, Hkv, 17 * d), 0xFF, dtype=torch.uint8, device=gpu)
    attn.cache_append_q4(k.to(gpu), v.to(gpu), torch.from_numpy(slots).to(torch.int32).to(gpu), cache)
    bt, sl = (torch.tensor(x, dtype=torch.int32, device=gpu) for x in (table.tolist(), lens))
    o, lse = attn.decode_paged_q4(q.to(gpu), cache, bt, sl, scale=math.log(2.0))
    c.check(o.double().cpu().numpy(), lse.double().cpu().numpy())
