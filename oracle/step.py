"""Float64 definitions of the serving step's operators: tables from request lengths, query/key norm
with rotation, and the 4-bit paged cache.  Plain loops and formulas; shares no code with the library.
"""
from __future__ import annotations

import numpy as np

PAGE = 16
GROUP = 64


def step_tables(cached, new, free, table, num_tokens):
    """(seq_lens, cu_seqlens, positions, slots, pages_used, table) of a step whose lengths all fit."""
    table = np.array(table)
    cu, positions, slots, used = [0], [], [], 0
    for n, (c, w) in enumerate(zip(cached, new)):
        for p in range(c, c + w):
            if p % PAGE == 0:
                table[n, p // PAGE] = free[used]
                used += 1
            positions.append(p)
            slots.append(int(table[n, p // PAGE]) * PAGE + p % PAGE)
        cu.append(cu[-1] + w)
    pad = num_tokens - len(slots)
    return ([c + w for c, w in zip(cached, new)], cu, positions + [0] * pad, slots + [-1] * pad, used, table)


def rope_angles(positions, rot, theta):
    i = np.arange(rot // 2, dtype=np.float64)
    return np.asarray(positions, np.float64)[:, None] * theta ** (-2.0 * i / rot)[None, :]


def norm_rope(x, weight, eps, cos, sin, interleaved):
    """x [T, H, d]; cos, sin [T, rot / 2].  Returns (y, size): size bounds the terms a value is the sum of."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, size = x.copy(), np.abs(x)
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


def _scale(step):
    """The smallest number of 4 significant bits that is at least `step` (a multiple of 2^-129 below 2^-126)."""
    m, e = np.frexp(step)
    grid = np.ldexp(1.0, np.maximum(e - 4, -129))
    return np.ceil(step / grid) * grid


def quantise(x):
    """bf16 values x [..., d] -> (codes [..., d] int, scales [..., d / 64], zero points [..., d / 64])."""
    g = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], np.shape(x)[-1] // GROUP, GROUP)
    hi, lo = np.maximum(g.max(-1), 0), np.minimum(g.min(-1), 0)
    scale = _scale((hi - lo) / 15)
    safe = np.where(scale > 0, scale, 1.0)
    zero = np.rint(-lo / safe)
    codes = np.clip(np.rint(g / safe[..., None]) + zero[..., None], 0, 15)
    return codes.astype(np.int64).reshape(np.shape(x)), scale, zero.astype(np.int64)


def stored(x):
    """The values that 4-bit storage keeps of x [..., d]."""
    codes, scale, zero = quantise(x)
    c = codes.reshape(*scale.shape, GROUP)
    return (scale[..., None] * (c - zero[..., None])).reshape(np.shape(x))


def read_record(rec, d):
    """Keys and values [16, d] that one record (17 d bytes) stands for, value by value."""
    rec = np.asarray(rec, np.uint8).astype(np.int64)
    per = min(2, d // GROUP)
    out = []
    for is_v in (0, 1):
        vals = np.zeros((PAGE, d))
        for k in range(PAGE):
            for ch in range(d):
                e, t, h, j = ch // 64, ch % 64 // 16, ch % 16 // 8, ch % 8
                if is_v:
                    p = ch // 2
                    byte = (p // 32 * 32 + p % 8 * 4 + k % 8 // 2) * 16 + p // 8 % 4 * 4 + k // 8 + 2 * (k % 2)
                    code = rec[8 * d + byte] >> (4 * (ch % 2)) & 15
                else:
                    word = e // per * (8 * per) + t * (2 * per) + e % per * 2 + h
                    at = k * (d // 2) + 4 * word
                    w = int(rec[at]) | int(rec[at + 1]) << 8 | int(rec[at + 2]) << 16 | int(rec[at + 3]) << 24
                    w = (w >> 3) | (w & 7) << 29
                    code = w >> (4 * j) & 15
                at = (16 * d + d // 2 if is_v else 16 * d) + 2 * (k * (d // GROUP) + e)
                par = int(rec[at] | rec[at + 1] << 8)
                scale = np.array([(par & 0xFFF0) << 16], np.uint32).view(np.float32)[0]
                vals[k, ch] = float(scale) * (int(code) - (par & 15))
        out.append(vals)
    return out
