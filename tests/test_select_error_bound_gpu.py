"""How far the tensor cores' block scores may be off, against the bound that block selection takes them by.

The scores of a call with more than one row a sequence lie at the start of its workspace, a row for each query token and KV
head.  The bound, relative to ||Q|| ||b|| for a row's sums Q over heads and a block's bounds b, counts
- Q as two bf16 numbers, 2^-18, and its sums over G heads, 2^-24 each;
- for each matrix product of 16 terms with an accumulator the terms' alignment, which drops what lies below 2^-25 of the largest
  one's power of two, and the rounding of the sum towards zero, 2^-23: (16 + 4) 2^-25, or where the instruction takes 8 terms at
  a time (16 + 2 x 4) 2^-25; and one more for the products of Q's second parts, which are 2^-8 of the first at most.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE = 16
# name: query rows, columns of the block table, rows' upper bound, terms that an instruction adds at a time
FORMS = {"few": (4, 4000, 4, 8), "many": (64, 2048, 64, 16), "many, small tiles": (64, 20000, 64, 16)}


def _eps(d, G, terms):
    if terms == 8:  # two accumulators share the products, and three additions join their parts
        return 2.0 ** -18 + (G + 3) * 2.0 ** -24 + d // 16 * 25 * 2.0 ** -25
    return 2.0 ** -18 + G * 2.0 ** -24 + d // 8 * 21 * 2.0 ** -25


def _scores(attn, q, bounds, width, max_q):
    """Scores [T, H, blocks] of a sequence whose blocks are the pages in order, and the selection."""
    dev, (T, _, d), (nb, H) = q.device, q.shape, bounds.shape[:2]
    i32 = dict(dtype=torch.int32, device=dev)
    table = torch.zeros((1, width), **i32)
    table[0, :nb] = torch.arange(nb, **i32)
    ws = torch.zeros(attn.select_blocks_workspace_bytes(T, 1, max_q, H, d, width), dtype=torch.uint8, device=dev)
    # the last token of every row's view is in the last page: each sees all blocks
    lens, cu = torch.full((1,), PAGE * nb, **i32), torch.tensor([0, T], **i32)
    picked = attn.select_blocks(q, bounds, table, lens, 5, cu_seqlens_q=cu, max_seqlen_q=max_q, workspace=ws)
    stride = (width + 7) // 8 * 8
    seen = (PAGE * nb - (T - 1) + PAGE - 1) // PAGE           # blocks that every row sees
    return ws[:4 * T * H * stride].view(torch.float32).view(T, H, stride)[:, :, :seen].double(), picked


def _sums(q, bounds):
    """(Q [T, H, 2 d], b [blocks, H, 2 d]) in 64 bits."""
    x = q.double().view(q.shape[0], bounds.shape[1], -1, q.shape[2])
    return torch.cat([x.clamp(max=0).sum(2), x.clamp(min=0).sum(2)], -1), bounds.double().flatten(2)


def _large(terms):
    """Channels of size 1, first in each accumulator: instructions of 8 terms have two, of every other four channels."""
    return (0, 4) if terms == 8 else (0,)


def _rough(nb, T, d, terms, dev):
    """Terms that lose all that they can: next to one of size 1 each of the others is a whole number of 2^-25 and 127 / 128 of
    one, for the first part of Q as for the second.  Four heads: first and second part of the negative and of the positive sums."""
    q = torch.zeros((T, 4, d), device=dev)
    first, second = 129 / 128 * 2.0 ** -9, 255 / 128 * 2.0 ** -18
    q[:, 0], q[:, 1], q[:, 2], q[:, 3] = -first, -second, first, second
    b = torch.empty((nb, 1, 2, d), device=dev)
    b[:, :, 0], b[:, :, 1] = -255 / 128 * 2.0 ** -9, 255 / 128 * 2.0 ** -9
    for c in _large(terms):
        q[:, :, c] = 0
        q[:, 0, c] = -1
        b[:, :, 0, c], b[:, :, 1, c] = -1, 0
    return q.to(torch.bfloat16), b.to(torch.bfloat16)


def _inputs(kind, nb, T, G, d, terms, dev):
    gen = torch.Generator(device=dev).manual_seed(d + G)
    rand = lambda *shape: torch.rand(shape, generator=gen, device=dev)  # noqa: E731
    if kind == "rough":
        return _rough(nb, T, d, terms, dev)
    if kind == "random":
        q = torch.randn((T, G, d), generator=gen, device=dev)
        return q.to(torch.bfloat16), torch.randn((nb, 1, 2, d), generator=gen, device=dev).sort(2).values.to(torch.bfloat16)
    # one channel, the first, above all others by 2^kind, and all terms of one sign
    q, b = (1 + rand(T, G, d)) * 2.0 ** -(kind // 2), (1 + rand(nb, 1, 2, d)) * 2.0 ** -(kind - kind // 2)
    q[:, :, 0], b[..., 0] = 1 + rand(T, G), 1 + rand(nb, 1, 2)
    b[:, :, 0] = 0
    return q.to(torch.bfloat16), b.to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("form", list(FORMS))
def test_scores_are_within_their_bound(attn, gpu, form, d):
    if form == "many, small tiles" and d != 128:
        return                                                # only d = 128 has them
    T, width, max_q, terms = FORMS[form]
    for kind in ["rough", "random"] + list(range(4, 31, 2)):
        for G in (1, 4):
            q, b = _inputs(kind, 600, T, G, d, terms, gpu)
            got = _scores(attn, q, b, width, max_q)[0]
            Q, bb = _sums(q, b)
            want = torch.einsum("thc,bhc->thb", Q, bb[:got.shape[2]])
            size = Q.norm(dim=-1)[:, :, None] * bb[:got.shape[2]].norm(dim=-1).T[None]
            worst = float(((got - want).abs() / size).max()) / _eps(d, q.shape[1], terms)
            assert worst <= 1, (kind, G, worst)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_rough_score_next_to_an_exact_one(attn, gpu, form, d):
    """A block whose score loses all that it can, and one that scores 10^-6 less and loses nothing."""
    T, width, max_q, terms = FORMS[form]
    nb, A, B = 600, 100, 200
    q, b = _rough(nb, T, d, terms, gpu)
    fine = (1, 2, 3)
    for c in fine:                                            # channels for the second block's score
        q[:, :, c] = 0
        q[:, 2, c] = 2.0 ** -4
        b[:, :, :, c] = 0
    b[torch.arange(nb, device=gpu) != A] = 0
    Q, bb = _sums(q, b)
    rest = float((Q[0, 0] * bb[A, 0]).sum()) - len(_large(terms)) - 1e-6     # of its score, beside the channels of size 1
    for c in _large(terms):
        b[B, 0, 0, c] = -1
    for c in fine:
        b[B, 0, 1, c] = rest * 16
        rest -= float(b[B, 0, 1, c]) / 16
    Q, bb = _sums(q, b)
    gap = float((Q[0, 0] * (bb[A, 0] - bb[B, 0])).sum())
    assert 0.9e-6 < gap < 1.1e-6
    dev = dict(dtype=torch.int32, device=gpu)
    table = torch.zeros((1, width), **dev)
    table[0, :nb] = torch.arange(nb, **dev)
    got = attn.select_blocks(q, b, table, torch.full((1,), PAGE * nb, **dev), 2, first=0, last=1,
                             cu_seqlens_q=torch.tensor([0, T], **dev), max_seqlen_q=max_q)
    assert (got[:, :, 0] == A).all()
