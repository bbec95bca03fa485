"""Cases of the serving-step operators: tables from request lengths, query/key norm with rotation, the 4-bit paged
cache, and attention over it.

``run`` makes one pass.  With ``own`` false it computes an operator in its plain form, elementary torch operations
in 32 bits; with ``own`` true it calls the library.  Head counts and lengths follow the library's own workloads:
32 query / 8 KV heads at d = 128 and 16 / 2 at d = 256, 16-token pages.
"""
import math
import random

import torch

own = False

PAGE = 16
GROUP = 64  # channels that share a scale and a zero point in the 4-bit cache


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's bookkeeping: 64 running requests, one new token each
        dict(name="tables_step", op="tables", N=64, cached_lo=512, cached_hi=8192, new_lo=1, new_hi=1),
        # a large mixed batch: running requests beside chunks of new prompts
        dict(name="tables_mixed", op="tables", N=512, cached_lo=0, cached_hi=4096, new_lo=1, new_hi=1024),
        # one decode step's projections: 64 tokens, K and V go to the paged cache
        dict(name="rope_step", op="rope", T=64, Hq=32, Hkv=8, d=128, rot=128, interleaved=False, norm=True, paged=True),
        # a 2048-token prompt
        dict(name="rope_prompt", op="rope", T=2048, Hq=32, Hkv=8, d=128, rot=128, interleaved=False, norm=True, paged=True),
        # a packed batch of long prompts, a quarter of each head rotated, adjacent pairs, K kept dense
        dict(name="rope_long", op="rope", T=32749, Hq=16, Hkv=2, d=256, rot=64, interleaved=True, norm=True, paged=False),
        # a 4-bit cache of short conversations takes one token of each and is read back
        dict(name="cache_step", op="cache", N=64, len_lo=17, len_hi=250, new=1, Hkv=8, d=128),
        # four prompts are written into the 4-bit cache and read back
        dict(name="cache_prompts", op="cache", N=4, len_lo=6000, len_hi=10001, new=0, Hkv=8, d=128),
        # one user, one short conversation: latency
        dict(name="decode_one", op="decode", N=1, len_lo=1009, len_hi=1009, Hq=32, Hkv=8, d=128),
        # the paged decode mix of the library's benchmark
        dict(name="decode_paged", op="decode", N=64, len_lo=512, len_hi=8192, Hq=32, Hkv=8, d=128),
        # its long-context mix
        dict(name="decode_long", op="decode", N=8, len_lo=6335, len_hi=122863, Hq=16, Hkv=2, d=256),
        # chunks of four prompts against what is cached of them
        dict(name="prefill_chunks", op="prefill", N=4, q_lo=129, q_hi=512, len_lo=4001, len_hi=8192, Hq=32, Hkv=8, d=128),
        # one long prompt's chunk
        dict(name="prefill_long", op="prefill", N=1, q_lo=2048, q_hi=2048, len_lo=32768, len_hi=32768, Hq=16, Hkv=2, d=256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "cache", "decode", "prefill"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128, 128, 256])
    if op == "tables":
        N = _log(rng, 1, 512)
        cached_hi = _log(rng, 16, 8192)
        new_lo = rng.choice([0, 1])
        return dict(op=op, N=N, cached_lo=rng.randint(0, cached_hi), cached_hi=cached_hi, new_lo=new_lo,
                    new_hi=_log(rng, 1, 1024))
    if op == "rope":
        rot = rng.choice([d, d, d // 2, d // 4])
        most = 32749 * 18 * 256 // ((Hq + 2 * Hkv) * d)
        return dict(op=op, T=_log(rng, 1, min(most, 32749)), Hq=Hq, Hkv=Hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.75, paged=rng.random() < 0.5)
    if op == "cache":
        N = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 32000 * 8 * 128 // (N * Hkv * d)))
        return dict(op=op, N=N, len_lo=rng.randint(1, hi), len_hi=hi, new=rng.choice([0, 1, 1, 7]), Hkv=Hkv, d=d)
    if op == "decode":
        N = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, min(122863, 270000 * 8 * 128 // (N * Hkv * d))))
        return dict(op=op, N=N, len_lo=rng.randint(0, hi), len_hi=hi, Hq=Hq, Hkv=Hkv, d=d)
    N = _log(rng, 1, 8)
    hi = _log(rng, 32, 16384 // N)
    q_hi = _log(rng, 1, min(hi, 1024))
    return dict(op=op, N=N, q_lo=rng.randint(1, q_hi), q_hi=q_hi, len_lo=rng.randint(q_hi, hi), len_hi=hi, Hq=Hq,
                Hkv=Hkv, d=d)


def _spread(n, lo, hi):
    """n lengths from hi down to lo, the same for every seed (work depends on their sum)."""
    return [hi] if n == 1 else [hi - (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case, seed, key="len"):
    lens = _spread(case["N"], case[key + "_lo"], case[key + "_hi"])
    random.Random(seed * 7 + 3).shuffle(lens)
    return lens


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _table_lens(case):
    """(cached, new) of each request: most requests run on with one token (or none), each eighth takes a chunk."""
    cached = _spread(case["N"], case["cached_lo"], case["cached_hi"])
    chunks = _spread(case["N"], case["new_lo"], case["new_hi"])
    new = [chunks[i] if i % 8 == 0 else min(1, chunks[i]) for i in range(case["N"])]
    return cached, new


# ---------------------------------------------------------------------------------------------- inputs
def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _keys(shape, gen):
    """Keys with a few strong channels, as models have them."""
    gain = 1.0 + 3.0 * (torch.rand(shape[-2:], generator=gen, device="cuda") < 0.05)
    return (torch.randn(shape, generator=gen, device="cuda") * gain).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _block_table(lens, width, gen):
    """Shuffled physical pages for sequences of the given lengths: (table [N, width], pages in all, the unused ids)."""
    need = torch.tensor([_pages(n) for n in lens], device="cuda")
    total = int(sum(_pages(n) for n in lens))
    num_blocks = total + 3
    perm = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(need, 0) - need)[:, None] + col[None, :]
    table = torch.where(col[None, :] < need[:, None], perm[at.clamp(max=num_blocks - 1)], 0)
    return table.to(torch.int32).contiguous(), num_blocks, perm[total:].contiguous()


def _slots_of(table, lens, new):
    """Slots of the last `new` tokens of each sequence (all of them where new is 0), packed in sequence order."""
    out = []
    for n, length in enumerate(lens):
        first = 0 if new == 0 else max(0, length - new)
        p = torch.arange(first, length, device="cuda")
        out.append(table[n].long()[p // PAGE] * PAGE + p % PAGE)
    return torch.cat(out).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "tables":
        cached, new = _table_lens(case)
        order = list(range(case["N"]))
        random.Random(seed).shuffle(order)
        cached, new = [cached[i] for i in order], [new[i] for i in order]
        width = _pages(max(c + w for c, w in zip(cached, new)) or 1) + 2
        need = sum(_pages(c + w) - _pages(c) for c, w in zip(cached, new))
        held = sum(_pages(c) for c in cached)
        num_blocks = held + need + 64
        perm = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
        pages = torch.tensor([_pages(c) for c in cached], device="cuda")
        col = torch.arange(width, device="cuda")
        at = (torch.cumsum(pages, 0) - pages)[:, None] + col[None, :]
        table = torch.where(col[None, :] < pages[:, None], perm[at.clamp(max=num_blocks - 1)], 0).to(torch.int32)
        # the batch is padded to a multiple of 64 tokens, as for a captured graph
        s.update(cached=_ints(cached), new=_ints(new), table=table.contiguous(), free=perm[held:].contiguous(),
                 num_tokens=max(64, (sum(new) + 63) // 64 * 64), num_blocks=num_blocks)
        return s
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "rope":
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        qkv = _randn((T, (Hq + 2 * Hkv) * d), gen)  # one projection's output; q, k and v are views of it
        s["q"] = qkv[:, :Hq * d].view(T, Hq, d)
        s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
        s["v"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        max_pos = 40960
        s["positions"] = torch.randint(0, max_pos, (T,), generator=gen, device="cuda").to(torch.int32)
        angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * (
            500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))[None, :]
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        if case["paged"]:
            num_blocks = _pages(T) + 5
            s["slots"] = torch.randperm(num_blocks * PAGE, generator=gen, device="cuda")[:T].to(torch.int32)
            s["k_cache"] = _randn((num_blocks, PAGE, Hkv, d), gen)
            s["v_cache"] = _randn((num_blocks, PAGE, Hkv, d), gen)
        return s
    lens = _lens(case, seed)
    table, num_blocks, _ = _block_table(lens, _pages(max(max(lens), 1)) + 1, gen)
    k = _keys((num_blocks, PAGE, Hkv, d), gen)
    v = _randn((num_blocks, PAGE, Hkv, d), gen)
    s.update(block_table=table, seq_lens=_ints(lens), cache=_pack(*_codes(k), *_codes(v)))
    del k, v
    if case["op"] == "cache":
        s["slots"] = _slots_of(table, lens, case["new"])
        s["k"] = _keys((s["slots"].numel(), Hkv, d), gen)
        s["v"] = _randn((s["slots"].numel(), Hkv, d), gen)
        s["out_k"] = torch.zeros((case["N"], table.shape[1] * PAGE, Hkv, d), dtype=torch.bfloat16, device="cuda")
        s["out_v"] = torch.zeros_like(s["out_k"])
    elif case["op"] == "decode":
        s["q"] = _randn((case["N"], case["Hq"], d), gen)
    else:
        q_lens = _lens(case, seed + 1, "q")
        cu = [0]
        for n in q_lens:
            cu.append(cu[-1] + n)
        s.update(q=_randn((cu[-1], case["Hq"], d), gen), cu=_ints(cu), max_q=max(q_lens))
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _codes(x):
    """4-bit codes of bf16 rows [..., d], in groups of 64 channels: (codes int32, parameters int32: scale | zero point)."""
    g = x.float().reshape(*x.shape[:-1], -1, GROUP)
    hi, lo = g.amax(-1).clamp(min=0), g.amin(-1).clamp(max=0)
    span = hi.double() - lo.double()  # in 64 bits: a step that is just one of the 4-bit numbers stays it
    step = span / torch.full_like(span, 15)
    scale = ((step.view(torch.int64) + ((1 << 49) - 1)) >> 49 << 49).view(torch.float64).float()
    bits = scale.view(torch.int32)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    zero = torch.round(-lo / safe)
    codes = (torch.round(g / safe[..., None]) + zero[..., None]).clamp(0, 15)
    return codes.to(torch.int32).reshape(x.shape), (bits >> 16) | zero.to(torch.int32)


def _le_bytes(w):
    """int32 words [..., n] as little-endian bytes [..., 4 n]."""
    return w.contiguous().view(torch.uint8)


def _pack(kc, kp, vc, vp):
    """Records [pages, Hkv, 17 d] of codes [pages, 16, Hkv, d] and parameters [pages, 16, Hkv, d / 64]."""
    P, _, H, d = kc.shape
    pair = min(2, d // GROUP)
    # K: channel = ((pairs, 2), t 4, half 2, nibble 8); a row's words are ordered (pair, t, group of the pair, half)
    w = kc.view(P, PAGE, H, -1, pair, 4, 2, 8)
    word = sum(w[..., n] << (4 * n) for n in range(8))
    word = (word << 3) | ((word >> 29) & 7)
    k_bytes = _le_bytes(word.permute(0, 2, 1, 3, 5, 4, 6).reshape(P, H, -1))
    # V: token = (byte bit 0: 2, t: 4, byte bit 1: 2), channel = (chunk, word 4, g 8, nibble 2)
    w = vc.view(P, 2, 4, 2, H, -1, 4, 8, 2)
    byte = w[..., 0] | (w[..., 1] << 4)                     # P, b0, t, b1, H, chunk, word, g
    v_bytes = byte.permute(0, 4, 5, 7, 2, 6, 3, 1).reshape(P, H, -1).to(torch.uint8)  # chunk, g, t, word, b1, b0
    par = [_le_bytes(p.permute(0, 2, 1, 3).reshape(P, H, -1).to(torch.int16)) for p in (kp, vp)]
    return torch.cat([k_bytes, v_bytes] + par, -1).contiguous()


def _unpack(rec, d):
    """Records [..., 17 d] uint8 to the values they stand for: k and v [..., 16, d] in 32 bits."""
    lead = rec.shape[:-1]
    pair = min(2, d // GROUP)
    nib = torch.arange(0, 32, 4, device=rec.device, dtype=torch.int32)
    w = rec[..., :8 * d].contiguous().view(torch.int32)
    w = ((w >> 3) & 0x1FFFFFFF) | (w << 29)
    kc = ((w[..., None] >> nib) & 15).view(*lead, PAGE, -1, 4, pair, 2, 8)
    kc = kc.transpose(-4, -3).reshape(*lead, PAGE, d)
    b = rec[..., 8 * d:16 * d].contiguous().view(*lead, -1, 8, 4, 4, 2, 2)       # chunk, g, t, word, b1, b0
    vc = torch.stack([b & 15, b >> 4], -1)
    n = len(lead)
    vc = vc.permute(*range(n), n + 5, n + 2, n + 4, n, n + 3, n + 1, n + 6).reshape(*lead, PAGE, d)
    out = []
    for codes, at in ((kc, 16 * d), (vc, 16 * d + d // 2)):
        par = rec[..., at:at + d // 2].contiguous().view(torch.int16).to(torch.int32).view(*lead, PAGE, -1)
        scale = ((par & 0xFFF0) << 16).view(torch.float32)
        value = (codes.view(*lead, PAGE, -1, GROUP).float() - (par & 15).float()[..., None]) * scale[..., None]
        out.append(value.reshape(*lead, PAGE, d))
    return out


def _context(s):
    """Keys and values of every sequence, padded: [N, Hkv, L, d] in 32 bits, zero past a sequence's end."""
    rec = s["cache"][s["block_table"].long()]                                    # N, blocks, Hkv, 17 d
    N, nb, H, _ = rec.shape
    live = torch.arange(nb * PAGE, device="cuda")[None, :] < s["seq_lens"].long()[:, None]
    k, v = (x.transpose(1, 2).reshape(N, H, nb * PAGE, s["d"]) for x in _unpack(rec, s["d"]))
    return torch.where(live[:, None, :, None], k, 0), torch.where(live[:, None, :, None], v, 0), live


def _attend(q, k, v, seen):
    """q [N, H, R, d], k and v [N, H, L, d], seen [N, 1, R, L] -> (o, lse), a row that sees nothing gives 0 and -inf."""
    score = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    score = score.masked_fill(~seen, -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(score - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o, (m + torch.log(l))[..., 0]


def _plain_tables(s):
    c, w = s["cached"].long(), s["new"].long()
    N, T = c.numel(), s["num_tokens"]
    cu = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(w, 0)
    first = (c + PAGE - 1) // PAGE
    need = (c + w + PAGE - 1) // PAGE - first
    before = torch.cumsum(need, 0) - need
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    fresh = (col >= first[:, None]) & (col < (first + need)[:, None])
    take = (before[:, None] + col - first[:, None]).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][take], s["table"]))
    t = torch.arange(T, device="cuda")
    n = torch.searchsorted(cu[1:], t, right=True).clamp(max=N - 1)
    live = t < cu[-1]
    pos = torch.where(live, c[n] + t - cu[n], 0)
    slot = s["table"][n, pos // PAGE].long() * PAGE + pos % PAGE
    return dict(seq_lens=(c + w).to(torch.int32), cu_seqlens=cu.to(torch.int32), positions=pos.to(torch.int32),
                slots=torch.where(live, slot, -1).to(torch.int32), table=s["table"],
                pages_used=need.sum(0, keepdim=True).to(torch.int32))


def _plain_rope(s):
    cos, sin = s["table"][s["positions"].long()].chunk(2, -1)

    def head(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = x[..., :s["rot"]], x[..., s["rot"]:]
        c, si = cos[:, None, :], sin[:, None, :]
        if s["interleaved"]:
            e, o = a[..., 0::2], a[..., 1::2]
            a = torch.stack([e * c - o * si, o * c + e * si], -1).reshape(a.shape)
        else:
            e, o = a.chunk(2, -1)
            a = torch.cat([e * c - o * si, o * c + e * si], -1)
        return torch.cat([a, b], -1).to(torch.bfloat16)

    q, k = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"])
    if not s["paged"]:
        return dict(q=q, k=k)
    at = s["slots"].long()
    s["k_cache"].view(-1, *k.shape[1:])[at] = k
    s["v_cache"].view(-1, *k.shape[1:])[at] = s["v"]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_cache(s):
    """The new rows' bytes are set one code at a time in the records, which are then read back."""
    d, H = s["d"], s["Hkv"]
    page, tok = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    kc, kp = _codes(s["k"])
    vc, vp = _codes(s["v"])
    pair = min(2, d // GROUP)
    T = page.numel()
    head = torch.arange(H, device="cuda")[None, :, None]
    row = lambda x: x[:, None, None]  # noqa: E731
    w = kc.view(T, H, -1, pair, 4, 2, 8)
    w = (w << torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)).sum(-1).to(torch.int32)
    w = (w << 3) | ((w >> 29) & 7)
    b = w.permute(0, 1, 2, 4, 3, 5).reshape(T, H, -1).contiguous().view(torch.uint8)
    cache = s["cache"]
    cache[row(page), head, row(tok) * (d // 2) + torch.arange(d // 2, device="cuda")] = b
    j = torch.arange(d // 2, device="cuda")
    at = ((j // 32) * 32 + (j % 8) * 4) * 16 + (j // 8 % 4) * 4
    at = at + row(tok % 8 // 2 * 16 + tok // 8 + 2 * (tok % 2)) + 8 * d
    cache[row(page), head, at] = (vc[..., 0::2] | (vc[..., 1::2] << 4)).to(torch.uint8)
    ng = d // GROUP
    for par, base in ((kp, 16 * d), (vp, 16 * d + d // 2)):
        b = par.to(torch.int16).contiguous().view(torch.uint8)
        cache[row(page), head, base + row(tok) * 2 * ng + torch.arange(2 * ng, device="cuda")] = b
    k, v, live = _context(s)
    keep = live[:, :, None, None]
    s["out_k"].copy_(torch.where(keep, k.transpose(1, 2).to(torch.bfloat16), s["out_k"]))
    s["out_v"].copy_(torch.where(keep, v.transpose(1, 2).to(torch.bfloat16), s["out_v"]))
    return dict(k=s["out_k"], v=s["out_v"])


def _plain_decode(s):
    N, Hq, d = s["q"].shape
    k, v, live = _context(s)
    o, lse = _attend(s["q"].float().view(N, s["Hkv"], -1, d), k, v, live[:, None, None, :])
    return dict(o=o.reshape(N, Hq, d).to(torch.bfloat16), lse=lse.reshape(N, Hq))


def _plain_prefill(s):
    T, Hq, d = s["q"].shape
    N, H, M = s["seq_lens"].numel(), s["Hkv"], s["max_q"]
    k, v, live = _context(s)
    cu = s["cu"].long()
    i = torch.arange(M, device="cuda")
    own_row = i[None, :] < (cu[1:] - cu[:-1])[:, None]                           # N, M
    q = s["q"].float()[(cu[:-1, None] + i).clamp(max=T - 1)]                     # N, M, Hq, d
    q = q.view(N, M, H, -1, d).permute(0, 2, 3, 1, 4).reshape(N, H, -1, d)       # rows (head of the group, token)
    pos = s["seq_lens"].long()[:, None] - (cu[1:] - cu[:-1])[:, None] + i        # N, M
    seen = torch.arange(k.shape[2], device="cuda")[None, None, :] <= pos[..., None]
    seen = (seen & live[:, None, :] & own_row[..., None])[:, None, None].expand(-1, 1, Hq // H, -1, -1)
    o, lse = _attend(q, k, v, seen.reshape(N, 1, -1, k.shape[2]))
    o = o.view(N, H, -1, M, d).permute(0, 3, 1, 2, 4).reshape(N, M, Hq, d)
    lse = lse.view(N, Hq, M).transpose(1, 2)
    return dict(o=o[own_row].to(torch.bfloat16), lse=lse[own_row].t().contiguous())


def run(state):
    s = state
    if not own:
        return dict(tables=_plain_tables, rope=_plain_rope, cache=_plain_cache, decode=_plain_decode,
                    prefill=_plain_prefill)[s["op"]](s)
    import attention_attn_prefill_gb300 as attn

    if s["op"] == "tables":
        t = attn.step_tables(s["cached"], s["new"], s["free"], s["table"], s["num_tokens"], s["num_blocks"])
        return dict(seq_lens=t.seq_lens, cu_seqlens=t.cu_seqlens, positions=t.positions, slots=t.slots,
                    table=s["table"], pages_used=t.pages_used)
    if s["op"] == "rope":
        paged = dict(v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"]) if s["paged"] else {}
        q, k = attn.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], q_weight=s["q_weight"],
                                 k_weight=s["k_weight"], eps=1e-6, interleaved=s["interleaved"], **paged)
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"]) if s["paged"] else dict(q=q, k=k)
    if s["op"] == "cache":
        attn.cache_append_q4(s["k"], s["v"], s["slots"], s["cache"])
        k, v = attn.cache_gather_q4(s["cache"], s["block_table"], s["seq_lens"], k_out=s["out_k"], v_out=s["out_v"])
        return dict(k=k, v=v)
    if s["op"] == "decode":
        o, lse = attn.decode_paged_q4(s["q"], s["cache"], s["block_table"], s["seq_lens"])
    else:
        o, lse = attn.prefill_paged_q4(s["q"], s["cache"], s["block_table"], s["cu"], s["seq_lens"], s["max_q"])
    return dict(o=o, lse=lse)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "tables":
        cached, new = _table_lens(case)
        T = max(64, (sum(new) + 63) // 64 * 64)
        need = sum(_pages(c + w) - _pages(c) for c, w in zip(cached, new))
        return dict(bytes=16 * case["N"] + 8 * T + 8 * need, flops=0)
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "rope":
        T, Hq = case["T"], case["Hq"]
        values = T * (Hq + Hkv * (2 if case["paged"] else 1)) * d
        table = min(T, 40960) * case["rot"] * 4
        return dict(bytes=4 * values + table + 8 * T, flops=8 * T * (Hq + Hkv) * d)
    tokens = _spread(case["N"], case["len_lo"], case["len_hi"])
    held = sum(tokens) * Hkv * 17 * d // 16 + 4 * sum(_pages(n) for n in tokens)  # one read of the 4-bit cache
    if case["op"] == "cache":
        fresh = sum(n if case["new"] == 0 else min(n, case["new"]) for n in tokens)
        return dict(bytes=fresh * Hkv * d * 4 + fresh * Hkv * 17 * d // 16 + held + sum(tokens) * Hkv * d * 4, flops=0)
    Hq = case["Hq"]
    if case["op"] == "decode":
        return dict(bytes=held + 4 * case["N"] * Hq * d, flops=4 * sum(tokens) * Hq * d)
    q = _spread(case["N"], case["q_lo"], case["q_hi"])
    # which chunk meets which context depends on the seed: the mean over their pairings
    pairs = sum(q) * sum(tokens) / case["N"] - sum(n * n / 2 for n in q)
    return dict(bytes=held + 4 * sum(q) * Hq * d, flops=4 * pairs * Hq * d)


# ---------------------------------------------------------------------------------------------- 64 bits
def _exact_values(rec, d):
    """Values [..., 16, d] in 64 bits of records [..., 17 d], each code fetched from its byte by the layout's formula."""
    tok = torch.arange(PAGE, device="cuda")[:, None]
    ch = torch.arange(d, device="cuda")[None, :]
    rec = rec.long()
    grp, within = ch // GROUP, ch % GROUP
    per = 2 * min(2, d // GROUP)                                                 # words a thread holds of a pair
    word = grp // 2 * (4 * per) + within // 16 * per + grp % 2 * 2 + within % 16 // 8
    bit = (4 * (within % 8) + 3) % 32                                            # words are stored turned left by 3
    lo = tok * (d // 2) + word * 4 + bit // 8
    nxt = tok * (d // 2) + word * 4 + (bit // 8 + 1) % 4
    kc = ((rec[..., lo] | (rec[..., nxt] << 8)) >> (bit % 8)) & 15
    j = ch // 2
    at = 8 * d + (j // 32 * 32 + j % 8 * 4 + tok % 8 // 2) * 16 + j // 8 % 4 * 4 + tok // 8 + 2 * (tok % 2)
    vc = (rec[..., at] >> (4 * (ch % 2))) & 15
    out = []
    for codes, base in ((kc, 16 * d), (vc, 16 * d + d // 2)):
        at = base + 2 * (tok * (d // GROUP) + grp)
        low, high = rec[..., at], rec[..., at + 1]
        exponent = ((high & 127) << 1) | (low >> 7)
        mantissa = 8 + ((low >> 4) & 7)
        scale = torch.where(exponent > 0, mantissa * torch.exp2(exponent.double() - 130), (mantissa - 8) * 2.0 ** -129)
        out.append(scale * (codes - (low & 15)).double())
    return out


def _exact_codes(x):
    """What 4-bit storage keeps of rows [..., d], by the definition in 64 bits."""
    g = x.double().reshape(*x.shape[:-1], -1, GROUP)
    hi, lo = g.amax(-1, keepdim=True).clamp(min=0), g.amin(-1, keepdim=True).clamp(max=0)
    m, e = torch.frexp((hi - lo) / torch.full_like(hi, 15))
    scale = torch.ldexp(torch.ceil(m * 16) / 16, e)
    inv = torch.where(scale > 0, scale, 1)
    z = torch.round(-lo / inv)
    return (scale * (torch.clamp(torch.round(g / inv) + z, 0, 15) - z)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "rope":
        half = case["rot"] // 2
        cs = s["table"].double()[s["positions"].long()]

        def head(x, w):
            x = x.double()
            if w is not None:
                x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6)
            out = x.clone()
            i = torch.arange(half, device="cuda")
            at, to = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            turn = torch.complex(cs[:, None, :half], cs[:, None, half:]) * torch.complex(x[..., at], x[..., to])
            out[..., at], out[..., to] = turn.real, turn.imag
            return out

        q, k = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"])
        if not case["paged"]:
            return dict(q=q, k=k)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc.view(-1, Hkv, d).index_copy_(0, s["slots"].long(), k)
        vc.view(-1, Hkv, d).index_copy_(0, s["slots"].long(), s["v"].double())
        return dict(q=q, k_cache=kc, v_cache=vc)
    lens = s["seq_lens"].tolist()
    if case["op"] == "cache":
        k, v = s["out_k"].double(), s["out_v"].double()
        new_k, new_v = _exact_codes(s["k"]), _exact_codes(s["v"])
        at = 0
        for n, length in enumerate(lens):
            fresh = length if case["new"] == 0 else min(length, case["new"])
            rows = s["block_table"][n, :_pages(length)].long()
            for out, old, new in zip((k, v), _exact_values(s["cache"][rows], d), (new_k, new_v)):
                out[n, :length] = old.transpose(1, 2).reshape(-1, Hkv, d)[:length]
                out[n, length - fresh:length] = new[at:at + fresh]
            at += fresh
        return dict(k=k, v=v)
    Hq = case["Hq"]
    G = Hq // Hkv
    q = s["q"].double()
    cu = list(range(case["N"] + 1)) if case["op"] == "decode" else s["cu"].tolist()
    o = torch.zeros_like(q)
    lse = torch.full((q.shape[0], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for n, length in enumerate(lens):
        if length == 0:
            continue
        k, v = (x.transpose(0, 1).reshape(Hkv, -1, d)[:, :length]
                for x in _exact_values(s["cache"][s["block_table"][n, :_pages(length)].long()], d))
        rows = cu[n + 1] - cu[n]
        hidden = torch.arange(length, device="cuda")[None, :] > torch.arange(length - rows, length, device="cuda")[:, None]
        for h in range(Hq):
            x = q[cu[n]:cu[n + 1], h] @ k[h // G].T / math.sqrt(d)
            x[hidden] = -math.inf
            lse[cu[n]:cu[n + 1], h] = torch.logsumexp(x, -1)
            o[cu[n]:cu[n + 1], h] = torch.softmax(x, -1) @ v[h // G]
    return dict(o=o, lse=lse if case["op"] == "decode" else lse.t().contiguous())
