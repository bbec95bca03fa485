"""Float64 definitions of the 8-bit paged cache, of block scores and of attention over listed blocks.  Plain loops and
formulas; shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
LEAST = -124


def exponent(most):
    """The smallest e >= -124 with most <= 448 2^e."""
    if most == 0:
        return LEAST
    e = max(LEAST, math.floor(math.log2(most)) - 12)
    while 448.0 * 2.0 ** e < most:
        e += 1
    return e


def e4m3(x):
    """x (|x| <= 448) to the nearest number of 4 significant bits, a multiple of 2^-9 below 2^-6; ties to even."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    grid = np.exp2(np.maximum(e - 4.0, -9.0))
    return np.rint(x / grid) * grid


class Page:
    """One page of one KV head's keys, or of its values: codes as numbers [16, d], the scale's exponent, the bounds."""

    def __init__(self, d):
        self.codes = np.zeros((PAGE, d))
        self.e = None                     # a cache of zeros
        self.lo = self.hi = np.zeros(d)

    def write(self, row, x):
        """Rows row .. of the page take x [rows, d]."""
        x = np.asarray(x, np.float64)
        finite = np.abs(x[np.isfinite(x)])
        need = exponent(finite.max() if finite.size else 0.0)
        if row == 0 or self.e is None:
            if row > 0:
                self.codes[:row] = 0.0
            e = need
        else:
            e = max(need, self.e)
            self.codes[:row] = e4m3(self.codes[:row] * 2.0 ** (self.e - e))
        with np.errstate(invalid="ignore"):
            self.codes[row:row + len(x)] = np.where(np.isfinite(x), e4m3(np.where(np.isfinite(x), x, 0) * 2.0 ** -e), np.nan)
        self.e = e
        lo, hi = x.min(0), x.max(0)
        self.lo = lo if row == 0 else np.minimum(self.lo, lo)
        self.hi = hi if row == 0 else np.maximum(self.hi, hi)

    def values(self):
        return self.codes * (0.0 if self.e is None else 2.0 ** self.e)


def k_byte(k, c, d):
    return ((k // 8 * (d // 64) + c // 64) * 32 + 4 * (k % 8) + c % 64 // 16) * 16 + c % 16


def v_byte(k, c, d):
    B = min(16, d // 8)
    return 16 * d + (((k // 8 * 2 + k % 2) * (d // (8 * B)) + c // (8 * B)) * 32 + c % (8 * B) // B * 4 + k % 8 // 2) * B + c % B


def code_numbers():
    """What each of the 256 codes stands for."""
    b = np.arange(256)
    e, m = b >> 3 & 15, b & 7
    x = np.where(e > 0, (8 + m) * np.exp2(e - 10.0), m * 2.0 ** -9)
    x = np.where((b & 127) == 127, np.nan, x)
    return np.where(b > 127, -x, x)


def read_record(rec, d):
    """((codes, scale) of the keys, (codes, scale) of the values) of one record (32 d + 16 bytes)."""
    rec = np.asarray(rec, np.uint8)
    number = code_numbers()
    k, c = np.meshgrid(np.arange(PAGE), np.arange(d), indexing="ij")
    scales = rec[32 * d:32 * d + 8].copy().view(np.float32)
    return ((number[rec[k_byte(k, c, d)]], float(scales[0])), (number[rec[v_byte(k, c, d)]], float(scales[1])))


def scores(q, lo, hi):
    """Scores [blocks] of query heads q [G, d] against bounds [blocks, d]."""
    neg, pos = np.minimum(q, 0).sum(0), np.maximum(q, 0).sum(0)
    return (neg * lo + pos * hi).sum(-1)


def select(score, chosen, first, last):
    """The blocks chosen of len(score): ascending, -1 behind."""
    nb = len(score)
    if nb <= chosen:
        return np.array(list(range(nb)) + [-1] * (chosen - nb))
    rank = np.where(np.isnan(score), np.inf, score)
    kept = set(range(first)) | set(range(nb - last, nb))
    # NaN before every number, infinity among them
    order = sorted((b for b in range(nb) if b not in kept), key=lambda b: (not np.isnan(score[b]), -rank[b], b))
    return np.array(sorted(kept | set(order[:chosen - len(kept)])))


def attend(q, k, v, scale):
    """(o [d], lse, mean |p v| [d], largest sum of |q k| scale) of one query over keys and values [L, d]."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -math.inf, np.zeros(v.shape[1]), 0.0
    s = k @ q * scale
    p = np.exp(s - s.max())
    return p @ v / p.sum(), s.max() + math.log(p.sum()), p @ np.abs(v) / p.sum(), float((np.abs(k) @ np.abs(q)).max() * scale)
