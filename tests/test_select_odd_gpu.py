"""Block selection beside a few pages whose bounds are no finite numbers, or too large for float32 scores.

Such a page once made every page of the row be scored in 64 bits, again for each digit of the border: 126 ms for 512 rows
of 2048 pages and 8 heads that take 0.04 ms.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE = 16
# name: sequences, rows each, columns of the block table, KV heads, head dim, chosen.  Every kernel that scores, and every one that
# picks: in one launch (256 and 128 threads); 128 and 1024 threads a row; scores that shared memory does not hold; a warp a row
SHAPES = {
    "one launch": (3, 1, 150, 2, 128, 20), "one launch, many": (80, 1, 120, 4, 64, 11), "few rows": (40, 3, 300, 3, 256, 30),
    "long": (1, 1, 3000, 2, 128, 100), "past shared memory": (1, 2, 13000, 1, 64, 40), "a warp a row": (2, 300, 500, 2, 128, 33),
    "a warp a row, wide": (1, 600, 2300, 2, 64, 64), "chunk": (3, 70, 700, 3, 256, 25), "chunk, few rows a CTA": (60, 20, 800, 1, 128, 9),
}


def _case(name, dev):
    N, rows, width, H, d, K = SHAPES[name]
    gen = torch.Generator(device=dev).manual_seed(len(name))
    pages = width + 40
    b = torch.randn((pages, H, 2, d), generator=gen, device=dev).sort(2).values.to(torch.bfloat16)
    table = torch.stack([torch.randperm(pages, generator=gen, device=dev)[:width] for _ in range(N)]).to(torch.int32)
    q = torch.randn((N * rows, 2 * H, d), generator=gen, device=dev).to(torch.bfloat16)
    lens = torch.tensor([PAGE * (width - n % 5) - n % 16 for n in range(N)], dtype=torch.int32, device=dev)
    cu = torch.arange(0, N * rows + 1, rows, dtype=torch.int32, device=dev)
    return q, b, table, lens, cu, rows, K


def _call(attn, case):
    q, b, table, lens, cu, rows, K = case
    return attn.select_blocks(q, b, table, lens, K, cu_seqlens_q=cu, max_seqlen_q=rows)


def _wanted(case, row, first=1, last=2):
    """A row's selection by 64-bit scores: what is no number first, then the highest, the lower block where they are equal."""
    q, b, table, lens, cu, rows, K = case
    n = row // rows
    nb = (int(lens[n]) - (rows - 1 - row % rows) + PAGE - 1) // PAGE
    x, y = q[row].double().view(b.shape[1], -1, q.shape[2]), b[table[n, :nb].long()].double()
    s = (x.clamp(max=0).sum(1) * y[:, :, 0]).sum(-1) + (x.clamp(min=0).sum(1) * y[:, :, 1]).sum(-1)
    out = []
    for col in s.T.tolist():
        kept = [i < first or i >= nb - last for i in range(nb)]
        order = sorted(range(nb), key=lambda i: (not kept[i], not math.isnan(col[i]), 0.0 if math.isnan(col[i]) else -col[i], i))
        out.append(sorted(order[:K]))
    return torch.tensor(out, dtype=torch.int32, device=q.device)


def _spoil(case, kind, odd):
    """odd pages of the first sequence's table, and of others by chance, get bounds of a kind."""
    q, b, table, lens, cu, rows, K = case
    at = table[0, odd].long()
    if kind == "nan":
        b[at, :, 1, 3] = math.nan
    elif kind == "infinite":
        b[at, :, 1, 3], b[at[::2], :, 0, 5] = math.inf, -math.inf
    elif kind == "large":                          # scores of 10^30 and their order, some below all others
        size = 10.0 ** (25 + 5 * torch.rand(len(odd), device=b.device))
        b[at] = (b[at].float() * size[:, None, None, None]).to(torch.bfloat16)
        b[at[::3], :, 1] = b[at[::3], :, 0].abs().neg()
        b[at[::3], :, 0] = b[at[::3], :, 1]
    elif kind == "alike":                          # equal ones, more than there are places
        b[at] = (b[at[:1]].float() * 1e28).to(torch.bfloat16)
    elif kind == "zero queries":                   # 0 times infinity beside scores of 0
        q[:, :, :] = 0
        b[at, :, 1, 3] = math.inf


@pytest.mark.parametrize("kind", ["nan", "infinite", "large", "alike", "zero queries"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_select_beside_odd_pages(attn, gpu, name, kind):
    """A few such pages, the first and the last one among them; and so many that they alone fill the places, or are all."""
    _, _, width, _, _, K = SHAPES[name]
    for odd in ([width // 3], [0, 1, 5, width // 2, width // 2 + 7, width - 1], list(range(3, width, 2)), list(range(width))):
        case = _case(name, gpu)
        _spoil(case, kind, odd)
        got = _call(attn, case)
        rows = case[5]
        total = got.shape[0]
        for r in sorted({0, rows // 2, rows - 1, total // 2, total - 1}):
            assert torch.equal(got[r], _wanted(case, r)), (len(odd), r)
    assert attn.device_status() == 0


@pytest.mark.parametrize("kind", ["one large", "two kinds", "close", "nan queries", "infinite queries"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_select_where_many_are_close_to_the_border(attn, gpu, name, kind):
    """More pages than a warp settles lie within the error of the border: a page so large, though no score passes its range,
    that all are unsure; two kinds of pages, each many times; pages that differ in a part of 10^11 to 10^13 of their scores; queries whose sums
    are no numbers, or infinite."""
    q, b, table, lens, cu, rows, K = case = _case(name, gpu)
    width = table.shape[1]
    gen = torch.Generator(device=gpu).manual_seed(3)
    if kind == "one large":
        b[table[:, width // 3].long()] *= 2.0 ** 14
    elif kind == "two kinds":
        b[0::2], b[1::2] = b[0].clone(), b[1].clone()
    elif kind == "close":
        b[:] = b[0].clone()
        b[:, :, :, 7] = torch.randn((b.shape[0], b.shape[1], 1), generator=gen, device=gpu).to(torch.bfloat16)
        q[:, :, 7] = q[:, :, 7].abs().clamp(min=0.1) * 1e-10
    elif kind == "nan queries":
        q[::2, 0, 5] = math.nan
    else:
        q[::2, 0, 5], q[1::2, 1, 6] = math.inf, -math.inf
    got = _call(attn, case)
    for r in sorted({0, 1 % got.shape[0], rows // 2, rows - 1, got.shape[0] // 2, got.shape[0] - 1}):
        assert torch.equal(got[r], _wanted(case, r)), r
    assert attn.device_status() == 0


def _micros(call):
    for _ in range(3):
        call()
    best = math.inf
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("name", list(SHAPES))
def test_an_odd_page_does_not_hold_up_the_others(attn, gpu, name):
    """It costs its tile of 16 pages a product in 64 bits: more than the plain case, but not what all pages cost.  The bound is
    wide: one such page once took 50 to 3000 times as long."""
    case = _case(name, gpu)
    plain = _micros(lambda: _call(attn, case))
    width = SHAPES[name][2]
    for where in ([width // 3], [0]):              # one that competes; the first one, which is chosen anyway
        for kind in ("nan", "large"):
            case = _case(name, gpu)
            _spoil(case, kind, where)
            taken = _micros(lambda: _call(attn, case))
            assert taken < 6 * plain + 60, (where, kind, taken, plain)


@pytest.mark.parametrize("name", [n for n in SHAPES if "one launch" not in n])
def test_a_large_page_does_not_hold_up_the_others(attn, gpu, name):
    """A page, and a few, with bounds 2^14 times the others': they take part with exact scores."""
    case = _case(name, gpu)
    plain = _micros(lambda: _call(attn, case))
    q, b, table, lens, cu, rows, K = case
    width = table.shape[1]
    for odd in ([width // 3], list(range(40, width, max(600, width // 4)))):
        case = _case(name, gpu)
        for n in range(table.shape[0]):
            at = case[2][n, odd].long()
            case[1][at] = (b[at].float() * 2.0 ** 14).to(torch.bfloat16)
        got = _call(attn, case)
        for r in sorted({0, rows - 1, got.shape[0] // 2, got.shape[0] - 1}):
            assert torch.equal(got[r], _wanted(case, r)), (len(odd), r)
        if len(odd) * table.shape[0] * 16 * 16 < width:  # (pages lie in several sequences' tables)
            taken = _micros(lambda: _call(attn, case))
            assert taken < 8 * plain + 100, (taken, plain)


@pytest.mark.parametrize("name", ["a warp a row, wide", "chunk"])
def test_exact_scores_are_computed_once(attn, gpu, name):
    """Two kinds of pages whose scores tie, but not their bounds: exact scores in 64 bits of all, upper halves and lower ones, take
    4 ns a row, head and page of a full GPU; 15 where each of eight digits took them again."""
    case = _case(name, gpu)
    N, rows, width, H, _, _ = SHAPES[name]
    b = case[1]
    b[0::2], b[1::2] = b[0].clone(), b[0].clone()
    b[1::2, :, :, 5] = 0
    case[0][:, :, 5] = 0
    taken = _micros(lambda: _call(attn, case))
    assert taken * 1e3 / (N * rows * H * width) < 7
    got = _call(attn, case)
    assert torch.equal(got[0], _wanted(case, 0))
