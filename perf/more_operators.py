"""Cases of the 8-bit paged cache and of attention over selected blocks: write and read-back of the cache, attention
over all of it, the choice of a query's blocks by key bounds, and attention over chosen blocks.

``run`` makes one pass.  With ``own`` false it computes an operator in its plain form, elementary torch operations
in 32 bits (block scores in 64: they decide borders); with ``own`` true it calls the library.  Head counts and
lengths follow the library's own workloads: 32 query / 8 KV heads at d = 128 and 16 / 2 at d = 256, 16-token pages.
"""
import math
import random

import torch

own = False

PAGE = 16      # tokens of a page, which is also the block that is chosen or left
LEAST = -124   # the smallest exponent of a scale: every stored value is a bf16 number


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step: 64 short conversations take a token each, are written with their bounds and read back
        dict(name="cache_step", op="cache", N=64, len_lo=17, len_hi=250, new=1, Hkv=8, d=128),
        # four prompts are written and read back
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
        # one decode step over selected blocks: 64 of up to 512 for each request and KV head
        dict(name="select_step", op="select", N=64, q_lo=1, q_hi=1, len_lo=512, len_hi=8192, Hq=32, Hkv=8, d=128, chosen=64,
             first=1, last=2),
        # long contexts: 256 of up to 7679 blocks
        dict(name="select_long", op="select", N=8, q_lo=1, q_hi=1, len_lo=6335, len_hi=122863, Hq=16, Hkv=2, d=256,
             chosen=256, first=1, last=2),
        # every token of a prompt's chunk chooses its own 64 of up to 2048 blocks
        dict(name="select_chunk", op="select", N=1, q_lo=512, q_hi=512, len_lo=32768, len_hi=32768, Hq=32, Hkv=8, d=128,
             chosen=64, first=1, last=2),
        # attention of the decode step over its chosen blocks
        dict(name="blocks_step", op="blocks", N=64, q_lo=1, q_hi=1, len_lo=512, len_hi=8192, Hq=32, Hkv=8, d=128, chosen=64),
        # and of the long contexts
        dict(name="blocks_long", op="blocks", N=8, q_lo=1, q_hi=1, len_lo=6335, len_hi=122863, Hq=16, Hkv=2, d=256,
             chosen=256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cache", "decode", "prefill", "select", "blocks"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128, 128, 256])
    if op == "cache":
        N = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 32000 * 8 * 128 // (N * Hkv * d)))
        return dict(op=op, N=N, len_lo=rng.randint(1, hi), len_hi=hi, new=rng.choice([0, 1, 1, 7]), Hkv=Hkv, d=d)
    if op == "decode":
        N = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, min(122863, 270000 * 8 * 128 // (N * Hkv * d))))
        return dict(op=op, N=N, len_lo=rng.randint(0, hi), len_hi=hi, Hq=Hq, Hkv=Hkv, d=d)
    if op == "prefill":
        N = _log(rng, 1, 8)
        hi = _log(rng, 32, 16384 // N)
        q_hi = _log(rng, 1, min(hi, 1024))
        return dict(op=op, N=N, q_lo=rng.randint(1, q_hi), q_hi=q_hi, len_lo=rng.randint(q_hi, hi), len_hi=hi, Hq=Hq,
                    Hkv=Hkv, d=d)
    N = _log(rng, 1, 64)
    hi = _log(rng, 256, max(256, min(122863, 270000 * 8 * 128 // (N * Hkv * d))))
    if op == "select":
        # rows x blocks x heads x channels within the largest listed case
        most = 512 * 2048 * 8 * 128 // (N * ((hi + PAGE - 1) // PAGE) * Hkv * d)
        q_hi = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, min(hi, 512, most)))
        first, last = rng.randint(0, 3), rng.randint(1, 3)
        chosen = _log(rng, first + last + 1, min(512, max(first + last + 1, _pages(hi) // 2)))
        return dict(op=op, N=N, q_lo=rng.randint(1, q_hi), q_hi=q_hi, len_lo=rng.randint(q_hi, hi), len_hi=hi, Hq=Hq,
                    Hkv=Hkv, d=d, chosen=chosen, first=first, last=last)
    q_hi = 1 if rng.random() < 0.75 else rng.randint(1, min(hi, 8))
    chosen = _log(rng, 1, max(1, min(512, 64 * 8 * 64 * 128 // (N * q_hi * Hkv * d))))
    return dict(op=op, N=N, q_lo=rng.randint(1, q_hi), q_hi=q_hi, len_lo=rng.randint(q_hi, hi), len_hi=hi, Hq=Hq,
                Hkv=Hkv, d=d, chosen=chosen)


def _spread(n, lo, hi):
    """n lengths from hi down to lo, the same for every seed (work depends on their sum)."""
    return [hi] if n == 1 else [hi - (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case, seed, key="len"):
    lens = _spread(case["N"], case[key + "_lo"], case[key + "_hi"])
    random.Random(seed * 7 + 3).shuffle(lens)
    return lens


def _pages(n):
    return (n + PAGE - 1) // PAGE


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
    """Shuffled physical pages for sequences of the given lengths: (table [N, width], pages in all)."""
    need = torch.tensor([_pages(n) for n in lens], device="cuda")
    num_blocks = int(sum(_pages(n) for n in lens)) + 3
    perm = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(need, 0) - need)[:, None] + col[None, :]
    table = torch.where(col[None, :] < need[:, None], perm[at.clamp(max=num_blocks - 1)], 0)
    return table.to(torch.int32).contiguous(), num_blocks


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
    Hkv, d, N = case["Hkv"], case["d"], case["N"]
    lens = _lens(case, seed)
    table, num_blocks = _block_table(lens, _pages(max(max(lens), 1)) + 1, gen)
    k = _keys((num_blocks, PAGE, Hkv, d), gen)
    if case["op"] in ("cache", "select"):
        # neighbouring keys resemble each other: each page has a mean of its own
        k = (k + 0.7 * torch.randn((num_blocks, 1, Hkv, d), generator=gen, device="cuda")).to(torch.bfloat16)
        s["bounds"] = torch.stack([k.amin(1), k.amax(1)], 2).contiguous()        # [blocks, Hkv, 2, d]
    s.update(block_table=table, seq_lens=_ints(lens))
    if case["op"] != "select":
        v = _randn((num_blocks, PAGE, Hkv, d), gen)
        s["cache"] = _pack(*_codes(k), *_codes(v))
        del v
    del k
    if case["op"] == "cache":
        s["slots"] = _slots_of(table, lens, case["new"])
        s["k"] = _keys((s["slots"].numel(), Hkv, d), gen)
        s["v"] = _randn((s["slots"].numel(), Hkv, d), gen)
        s["out_k"] = torch.zeros((N, table.shape[1] * PAGE, Hkv, d), dtype=torch.bfloat16, device="cuda")
        s["out_v"] = torch.zeros_like(s["out_k"])
        return s
    if case["op"] == "decode":
        s["q"] = _randn((N, case["Hq"], d), gen)
        return s
    q_lens = _lens(case, seed + 1, "q")
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s.update(q=_randn((cu[-1], case["Hq"], d), gen), cu=_ints(cu), max_q=max(q_lens))
    if case["op"] == "blocks":
        # distinct blocks of those each token sees, its own among them, in ascending order
        vis = _visible(s)[1]
        nb = (vis + PAGE - 1) // PAGE
        col = torch.arange(table.shape[1], device="cuda")
        luck = torch.rand((cu[-1], Hkv, table.shape[1]), generator=gen, device="cuda")
        luck = torch.where(col < nb[:, None, None] - 1, luck, 2.0 * (col < nb[:, None, None]).float() - 0.5)
        top, at = luck.topk(min(case["chosen"], table.shape[1]), -1)
        at = torch.where(top >= 0, at, 1 << 30).sort(-1).values
        at = torch.where(at < 1 << 30, at, -1).to(torch.int32)
        s["blocks"] = torch.nn.functional.pad(at, (0, case["chosen"] - at.shape[-1]), value=-1).contiguous()
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _exponent(amax):
    """The smallest e (at least LEAST) with amax <= 448 2^e."""
    m, e = torch.frexp(amax)
    return (e - 9 + (m > 0.875).to(torch.int32)).clamp(min=LEAST)


def _e4m3(x):
    """x rounded to 8 bits, as the number that they stand for."""
    return x.to(torch.float8_e4m3fn).float()


def _codes(x):
    """Rows [pages, 16, H, d] in 8 bits with a scale a page and head: (numbers of 8 bits in float32, scales [pages, H])."""
    e = _exponent(x.float().abs().amax((1, 3)))
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return _e4m3(x.float() / scale[:, None, :, None]), scale


def _pack(kc, ks, vc, vs):
    """Records [pages, Hkv, 32 d + 16] of codes [pages, 16, Hkv, d] and scales [pages, Hkv]."""
    P, _, H, d = kc.shape
    B = min(16, d // 8)
    kb, vb = (c.to(torch.float8_e4m3fn).view(torch.uint8) for c in (kc, vc))
    # K: (token / 8, channel / 64, token % 8, the 64 channels); V: (token / 8, token % 2, channel / 8 B, g 8,
    # token / 2 % 4, B channels)
    kb = kb.view(P, 2, 8, H, d // 64, 64).permute(0, 3, 1, 4, 2, 5).reshape(P, H, -1)
    vb = vb.view(P, 2, 4, 2, H, d // (8 * B), 8, B).permute(0, 4, 1, 3, 5, 6, 2, 7).reshape(P, H, -1)
    tail = torch.stack([ks, vs, torch.zeros_like(ks), torch.zeros_like(ks)], -1).contiguous().view(torch.uint8)
    return torch.cat([kb, vb, tail], -1).contiguous()


def _unpack(rec, d):
    """Records [..., 32 d + 16] uint8: codes of k and v [..., 16, d] as numbers in 32 bits, and their scales [...]."""
    lead, n = rec.shape[:-1], rec.dim() - 1
    B = min(16, d // 8)
    k = rec[..., :16 * d].reshape(*lead, 2, d // 64, 8, 64).transpose(-3, -2).reshape(*lead, PAGE, d)
    v = rec[..., 16 * d:32 * d].reshape(*lead, 2, 2, d // (8 * B), 8, 4, B)
    v = v.permute(*range(n), n, n + 4, n + 1, n + 2, n + 3, n + 5).reshape(*lead, PAGE, d)
    scale = rec[..., 32 * d:].contiguous().view(torch.float32)
    return (k.contiguous().view(torch.float8_e4m3fn).float(), scale[..., 0],
            v.contiguous().view(torch.float8_e4m3fn).float(), scale[..., 1])


def _values(rec, d):
    kc, ks, vc, vs = _unpack(rec, d)
    return kc * ks[..., None, None], vc * vs[..., None, None]


def _context(s):
    """Keys and values of every sequence, padded: [N, Hkv, L, d] in 32 bits, zero past a sequence's end."""
    rec = s["cache"][s["block_table"].long()]                                    # N, blocks, Hkv, record
    N, nb, H, _ = rec.shape
    live = torch.arange(nb * PAGE, device="cuda")[None, :] < s["seq_lens"].long()[:, None]
    k, v = (x.transpose(1, 2).reshape(N, H, nb * PAGE, s["d"]) for x in _values(rec, s["d"]))
    return torch.where(live[:, None, :, None], k, 0), torch.where(live[:, None, :, None], v, 0), live


def _visible(s):
    """Of each packed query token: its sequence, and the tokens it sees (itself the last)."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    n = torch.searchsorted(cu[1:], t, right=True)
    return n, s["seq_lens"].long()[n] - (cu[n + 1] - t) + 1


def _attend(q, k, v, seen):
    """q [N, H, R, d], k and v [N, H, L, d], seen [N, 1 or H, R, L] -> (o, lse); a row that sees nothing gives 0 and -inf."""
    score = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    score = score.masked_fill(~seen, -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(score - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o, (m + torch.log(l))[..., 0]


def _plain_cache(s):
    """The pages that take new rows are taken out, rescaled where their scale grows, filled and put back."""
    d = s["d"]
    cache, bounds = s["cache"], s["bounds"]
    page, inv = torch.unique(s["slots"].long() // PAGE, return_inverse=True)
    row = s["slots"].long() % PAGE
    U, H = page.numel(), s["Hkv"]
    first = torch.full((U,), PAGE, device="cuda").scatter_reduce(0, inv, row, "amin")
    old = torch.arange(PAGE, device="cuda")[None, :] < first[:, None]
    out = []
    for x, (codes, scale) in zip((s["k"].float(), s["v"].float()), zip(*[iter(_unpack(cache[page], d))] * 2)):
        most = torch.zeros((U, H), device="cuda").index_reduce(0, inv, x.abs().amax(-1), "amax")
        need = torch.ldexp(torch.ones_like(most), _exponent(most))
        now = torch.where(first[:, None] > 0, torch.maximum(scale, need), need)
        moved = _e4m3(codes * (scale / now)[..., None, None])                    # U, H, 16, d
        codes = torch.where(old[:, None, :, None], moved, codes)
        codes[inv, :, row] = _e4m3(x / now[inv][..., None])
        out += [codes.transpose(1, 2), now]
    cache[page] = _pack(*out)
    x = s["k"].float()
    lo = torch.full((U, H, d), math.inf, device="cuda").index_reduce(0, inv, x, "amin")
    hi = torch.full((U, H, d), -math.inf, device="cuda").index_reduce(0, inv, x, "amax")
    was = bounds[page].float()
    lo = torch.where(first[:, None, None] > 0, torch.minimum(was[:, :, 0], lo), lo)
    hi = torch.where(first[:, None, None] > 0, torch.maximum(was[:, :, 1], hi), hi)
    bounds[page] = torch.stack([lo, hi], 2).to(torch.bfloat16)
    k, v, live = _context(s)
    keep = live[:, :, None, None]
    s["out_k"].copy_(torch.where(keep, k.transpose(1, 2).to(torch.bfloat16), s["out_k"]))
    s["out_v"].copy_(torch.where(keep, v.transpose(1, 2).to(torch.bfloat16), s["out_v"]))
    return dict(k=s["out_k"], v=s["out_v"], bounds=bounds)


def _plain_decode(s):
    N, Hq, d = s["q"].shape
    k, v, live = _context(s)
    o, lse = _attend(s["q"].float().view(N, s["Hkv"], -1, d), k, v, live[:, None, None, :])
    return dict(o=o.reshape(N, Hq, d).to(torch.bfloat16), lse=lse.reshape(N, Hq))


def _padded(s):
    """(own [N, M]: which of M rows a sequence has, their packed places [N, M])."""
    cu = s["cu"].long()
    i = torch.arange(s["max_q"], device="cuda")
    return i[None, :] < (cu[1:] - cu[:-1])[:, None], (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)


def _plain_prefill(s):
    T, Hq, d = s["q"].shape
    N, H, M = s["seq_lens"].numel(), s["Hkv"], s["max_q"]
    k, v, live = _context(s)
    own_row, at = _padded(s)
    q = s["q"].float()[at].view(N, M, H, -1, d).permute(0, 2, 3, 1, 4).reshape(N, H, -1, d)
    pos = _visible(s)[1][at] - 1                                                 # N, M
    seen = torch.arange(k.shape[2], device="cuda")[None, None, :] <= pos[..., None]
    seen = (seen & live[:, None, :] & own_row[..., None])[:, None, None].expand(-1, 1, Hq // H, -1, -1)
    o, lse = _attend(q, k, v, seen.reshape(N, 1, -1, k.shape[2]))
    o = o.view(N, H, -1, M, d).permute(0, 3, 1, 2, 4).reshape(N, M, Hq, d)
    lse = lse.view(N, Hq, M).transpose(1, 2)
    return dict(o=o[own_row].to(torch.bfloat16), lse=lse[own_row].t().contiguous())


def _plain_select(s):
    """A block's score is the largest that a key within its bounds could have, summed over the heads of a KV head."""
    T, Hq, d = s["q"].shape
    H, K = s["Hkv"], s["chosen"]
    nb = (_visible(s)[1] + PAGE - 1) // PAGE                                     # T
    own_row, at = _padded(s)
    q = s["q"].double().view(T, H, -1, d)
    both = torch.cat([q.clamp(max=0).sum(2), q.clamp(min=0).sum(2)], -1)[at]     # N, M, H, 2 d: times minimum, maximum
    b = s["bounds"][s["block_table"].long()].double().flatten(3)                 # N, blocks, H, 2 d
    score = torch.matmul(both.transpose(1, 2), b.permute(0, 2, 3, 1)).transpose(1, 2)[own_row]   # T, H, blocks
    col = torch.arange(b.shape[1], device="cuda")
    there = (col < nb[:, None])[:, None]
    kept = ((col < s["first"]) | (col >= nb[:, None] - s["last"]))[:, None] & there
    score = torch.where(kept, math.inf, torch.where(there, score, -math.inf))
    at = score.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    at = torch.where(at < nb[:, None, None], at, 1 << 30).sort(-1).values
    at = torch.where(at < 1 << 30, at, -1).to(torch.int32)
    return torch.nn.functional.pad(at, (0, K - at.shape[-1]), value=-1)


def _plain_blocks(s):
    T, Hq, d = s["q"].shape
    H, K = s["Hkv"], s["chosen"]
    n, vis = _visible(s)
    blk = s["blocks"].long()                                                     # T, H, K
    page = s["block_table"].long()[n[:, None, None], blk.clamp(min=0)]
    k, v = (x.reshape(T, H, K * PAGE, d) for x in
            _values(s["cache"][page, torch.arange(H, device="cuda")[None, :, None]], d))
    token = blk[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    seen = ((blk >= 0)[..., None] & (token < vis[:, None, None, None])).reshape(T, H, 1, K * PAGE)
    o, lse = _attend(s["q"].float().view(T, H, -1, d), k, torch.where(seen.transpose(-1, -2), v, 0), seen)
    return dict(o=o.reshape(T, Hq, d).to(torch.bfloat16), lse=lse.reshape(T, Hq))


def run(state):
    s = state
    if not own:
        return dict(cache=_plain_cache, decode=_plain_decode, prefill=_plain_prefill, select=_plain_select,
                    blocks=_plain_blocks)[s["op"]](s)
    import attention_attn_prefill_gb300 as attn

    if s["op"] == "cache":
        attn.cache_append_f8(s["k"], s["v"], s["slots"], s["cache"], bounds=s["bounds"])
        k, v = attn.cache_gather_f8(s["cache"], s["block_table"], s["seq_lens"], k_out=s["out_k"], v_out=s["out_v"])
        return dict(k=k, v=v, bounds=s["bounds"])
    if s["op"] == "select":
        return attn.select_blocks(s["q"], s["bounds"], s["block_table"], s["seq_lens"], s["chosen"], first=s["first"],
                                  last=s["last"], cu_seqlens_q=s["cu"], max_seqlen_q=s["max_q"])
    if s["op"] == "decode":
        o, lse = attn.decode_paged_f8(s["q"], s["cache"], s["block_table"], s["seq_lens"])
    elif s["op"] == "prefill":
        o, lse = attn.prefill_paged_f8(s["q"], s["cache"], s["block_table"], s["cu"], s["seq_lens"], s["max_q"])
    else:
        o, lse = attn.decode_blocks_f8(s["q"], s["cache"], s["block_table"], s["seq_lens"], s["blocks"],
                                       cu_seqlens_q=s["cu"])
    return dict(o=o, lse=lse)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    Hkv, d, N = case["Hkv"], case["d"], case["N"]
    tokens = _spread(N, case["len_lo"], case["len_hi"])
    held = sum(tokens) * Hkv * (2 * d + 1) + 4 * sum(_pages(n) for n in tokens)  # one read of the 8-bit cache
    if case["op"] == "cache":
        fresh = sum(n if case["new"] == 0 else min(n, case["new"]) for n in tokens)
        pages = sum(_pages(n) if case["new"] == 0 else _pages(min(n, case["new"])) for n in tokens)
        return dict(bytes=fresh * Hkv * d * 6 + pages * Hkv * 4 * d + held + sum(tokens) * Hkv * d * 4, flops=0)
    Hq = case["Hq"]
    if case["op"] == "decode":
        return dict(bytes=held + 4 * N * Hq * d, flops=4 * sum(tokens) * Hq * d)
    q = _spread(N, case["q_lo"], case["q_hi"])
    if case["op"] == "prefill":
        # which chunk meets which context depends on the seed: the mean over their pairings
        pairs = sum(q) * sum(tokens) / N - sum(n * n / 2 for n in q)
        return dict(bytes=held + 4 * sum(q) * Hq * d, flops=4 * pairs * Hq * d)
    blocks = sum(_pages(n) for n in tokens)
    if case["op"] == "select":
        return dict(bytes=blocks * Hkv * 4 * d + 4 * blocks + 2 * sum(q) * Hq * d + 4 * sum(q) * Hkv * case["chosen"],
                    flops=4 * sum(q) * blocks // N * Hkv * d)
    # tokens that share blocks may share their reads: at most every page of a sequence once
    seen = sum(q) / N * sum(min(case["chosen"], _pages(n)) for n in tokens)
    once = min(seen, blocks)
    return dict(bytes=int(once * PAGE * Hkv * (2 * d + 1)) + 4 * sum(q) * Hq * d + 4 * sum(q) * Hkv * case["chosen"],
                flops=int(4 * seen * PAGE * Hq * d))


# ---------------------------------------------------------------------------------------------- 64 bits
def _exact_round(x):
    """x rounded to the nearest number of 4 significant bits (a multiple of 2^-9 below 2^-6), ties to even."""
    grid = torch.exp2(torch.frexp(x).exponent.double() - 4).clamp(min=2.0 ** -9)
    return torch.round(x / grid) * grid


def _exact_parts(rec, d):
    """Codes [..., 16, d] and scales of records in 64 bits, each code fetched from its byte by the layout's formula."""
    B = min(16, d // 8)
    tok = torch.arange(PAGE, device="cuda")[:, None]
    ch = torch.arange(d, device="cuda")[None, :]
    k_at = ((tok // 8 * (d // 64) + ch // 64) * 32 + tok % 8 * 4 + ch % 64 // 16) * 16 + ch % 16
    plane = (tok // 8 * 2 + tok % 2) * (d // (8 * B)) + ch // (8 * B)
    v_at = 16 * d + (plane * 32 + ch % (8 * B) // B * 4 + tok % 8 // 2) * B + ch % B
    out = []
    for at, word in ((k_at, 0), (v_at, 1)):
        b = rec[..., at].long()
        exponent, mantissa = b >> 3 & 15, b & 7
        x = torch.where(exponent > 0, (8 + mantissa) * torch.exp2(exponent.double() - 10), mantissa * 2.0 ** -9)
        tail = rec[..., 32 * d + 4 * word:32 * d + 4 * word + 4].long()
        scale = torch.exp2((((tail[..., 3] & 127) << 1) | (tail[..., 2] >> 7)).double() - 127)
        out += [torch.where(b > 127, -x, x), scale]
    return out


def _exact_values(rec, d):
    kc, ks, vc, vs = _exact_parts(rec, d)
    return kc * ks[..., None, None], vc * vs[..., None, None]


def _exact_cache(s, case):
    """Sequence by sequence, page by page of those that take new rows."""
    d = case["d"]
    out = [s["out_k"].double(), s["out_v"].double()]
    bounds, at = s["bounds"].double(), 0
    for n, length in enumerate(s["seq_lens"].tolist()):
        fresh = length if case["new"] == 0 else min(length, case["new"])
        start = length - fresh
        p0, rows = start // PAGE, s["block_table"][n, :_pages(length)].long()
        parts = _exact_parts(s["cache"][rows], d)
        touched = torch.arange(p0, _pages(length), device="cuda")
        tok = touched[:, None] * PAGE + torch.arange(PAGE, device="cuda")        # U, 16
        new, old = (tok >= start) & (tok < length), tok < start
        for i, x in enumerate((s["k"], s["v"])):
            codes, scale = parts[2 * i], parts[2 * i + 1]                        # pages, H, 16, d; pages, H
            y = x[at + (tok - start).clamp(0, fresh - 1)].double()               # U, 16, H, d
            y = torch.where(new[..., None, None], y, 0).transpose(1, 2)          # U, H, 16, d
            most = y.abs().amax((-1, -2))
            e = torch.ceil(torch.log2(most.clamp(min=1e-300) / 448)).clamp(min=LEAST)
            e = torch.where(448 * torch.exp2(e - 1) >= most, e - 1, e).clamp(min=LEAST)
            need = torch.exp2(torch.where(448 * torch.exp2(e) < most, e + 1, e))
            was = torch.where(old.any(1)[:, None], scale[p0:], 0)
            now = torch.maximum(need, was)[..., None, None]
            mine = _exact_round(y / now) * now
            kept = _exact_round(codes[p0:] * (scale[p0:][..., None, None] / now)) * now
            value = codes * scale[..., None, None]
            value[p0:] = torch.where(new[:, None, :, None], mine, torch.where(old[:, None, :, None], kept, value[p0:]))
            out[i][n, :length] = value.transpose(1, 2).reshape(-1, case["Hkv"], d)[:length]
            if i == 0:
                lo = torch.where(new[:, None, :, None], y, math.inf).amin(2)
                hi = torch.where(new[:, None, :, None], y, -math.inf).amax(2)
                had = old.any(1)[:, None, None]
                b = bounds[rows[p0:]]
                bounds[rows[p0:]] = torch.stack([torch.where(had, torch.minimum(b[:, :, 0], lo), lo),
                                                 torch.where(had, torch.maximum(b[:, :, 1], hi), hi)], 2)
        at += fresh
    return dict(k=out[0], v=out[1], bounds=bounds)


def _exact_select(s, case):
    """Row by row: the sum over heads and channels of the larger of q times either bound."""
    n_of, vis = (x.tolist() for x in _visible(s))
    H, K, d = case["Hkv"], case["chosen"], case["d"]
    out = torch.full((len(vis), H, K), -1, dtype=torch.int32, device="cuda")
    held = None
    for t, (n, seen) in enumerate(zip(n_of, vis)):
        nb = _pages(seen)
        if nb <= K:
            out[t, :, :nb] = torch.arange(nb, device="cuda")
            continue
        if held != n:
            b, held = s["bounds"][s["block_table"][n].long()].double(), n        # blocks, H, 2, d
        q = s["q"][t].double().view(1, H, -1, d)
        lo, hi = b[:nb, :, 0], b[:nb, :, 1]
        score = sum(torch.maximum(q[:, :, g] * lo, q[:, :, g] * hi).sum(-1) for g in range(q.shape[2]))   # nb, H
        score[:case["first"]] = math.inf
        score[nb - case["last"]:] = math.inf
        for h in range(H):
            order = torch.argsort(score[:, h], descending=True, stable=True)[:K]
            out[t, h] = order.sort().values.to(torch.int32)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "cache":
        return _exact_cache(s, case)
    if case["op"] == "select":
        return _exact_select(s, case)
    Hq = case["Hq"]
    G = Hq // Hkv
    q = s["q"].double()
    o = torch.zeros_like(q)
    lse = torch.full((q.shape[0], Hq), -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "blocks":
        n_of, vis = (x.tolist() for x in _visible(s))
        for t, (n, seen) in enumerate(zip(n_of, vis)):
            for h in range(Hkv):
                blk = s["blocks"][t, h]
                blk = blk[blk >= 0].long()
                k, v = (x.reshape(-1, d) for x in _exact_values(s["cache"][s["block_table"][n][blk].long(), h], d))
                gone = (blk[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten() >= seen
                x = (q[t, h * G:(h + 1) * G] @ k.T / math.sqrt(d)).masked_fill(gone, -math.inf)
                lse[t, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                o[t, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
        return dict(o=o, lse=lse)
    cu = list(range(case["N"] + 1)) if case["op"] == "decode" else s["cu"].tolist()
    for n, length in enumerate(s["seq_lens"].tolist()):
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
