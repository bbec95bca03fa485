"""Attention over listed blocks with query rows that belong to no sequence."""
import pytest
import torch

from test_f8_more_gpu import PAGE, _check_rows, _i32, _pages, _randn, _setup, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,rows,spare,length,Hq,Hkv,d,K", [
    # few rows and units, long lists: a descriptor a pair
    (2, 1, 2, 9000, 8, 2, 128, 500), (1, 1, 1, 30000, 3, 1, 256, 700), (3, 2, 3, 6000, 4, 1, 64, 371),
    # more of them, past the sizes that take a row whole: a descriptor a share
    (3, 15, 5, 9000, 8, 2, 128, 500), (5, 12, 30, 4000, 5, 1, 64, 200), (4, 50, 9, 3000, 4, 2, 256, 180),
])
def test_rows_of_no_sequence_in_shares(attn, gpu, N, rows, spare, length, Hq, Hkv, d, K):
    """Rows before the first sequence's and behind the last one's, where shares cut the list: left as they were."""
    gen, cache, bounds, table = _setup(attn, gpu, [length] * N, Hkv, d, seed=K)
    cu = [spare + n * rows for n in range(N + 1)]
    T = cu[-1] + spare
    q = _randn((T, Hq, d), gen, gpu)
    nb = _pages(length)
    blocks = torch.rand((T, Hkv, nb), generator=gen, device=gpu).argsort(-1)[..., :K].to(torch.int32).contiguous()
    o = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device=gpu)
    lse = torch.full((T, Hq), 7.0, device=gpu)
    for _ in range(2):
        attn.decode_blocks_f8(q, cache, table, _i32([length] * N, gpu), blocks, cu_seqlens_q=_i32(cu, gpu), out=o, lse=lse)
        for x in (o, lse):
            assert (x[:spare] == 7).all() and (x[cu[-1]:] == 7).all() and not (x[spare:cu[-1]] == 7).flatten(1).all(1).any()
    G = Hq // Hkv
    for r in sorted({spare, cu[-1] - 1, cu[N // 2], (spare + cu[-1]) // 2}):
        n = (r - spare) // rows
        seen = length - (cu[n + 1] - 1 - r)
        k, v = (x[0].double() for x in _values(attn, cache, table[n:n + 1], [length], gpu))
        for h in range(Hkv):
            at = (blocks[r, h].long()[:, None] * PAGE + torch.arange(PAGE, device=gpu)).flatten()
            at = at[at < seen]
            sl = slice(h * G, (h + 1) * G)
            _check_rows(o[r, sl], lse[r, sl], q[r, sl], k[at, h], v[at, h], d ** -0.5, d)
    assert attn.device_status() == 0
