"""Block selection called from several host threads at once.

A kernel's limit of shared memory is one number for all calls on a device: a call that set it to its own need could have
it lowered by another before its launch, which then failed.
"""
import threading

import pytest
import torch

from attention_attn_prefill_gb300._lib import _SIGNATURES

pytestmark = pytest.mark.gpu
CALLS = 6000


def _call(attn, dev, N, width, rows, Hkv, d, stream):
    """A call of the C entry point alone on short sequences, whose work is small next to the call itself; and its output."""
    gen = torch.Generator(device=dev).manual_seed(N + width + rows)
    i32 = dict(dtype=torch.int32, device=dev)
    K, length = 5, 16 * 40
    bounds = torch.randn((64, Hkv, 2, d), generator=gen, device=dev).sort(2).values.to(torch.bfloat16)
    table = torch.randint(0, 64, (N, width), generator=gen, **i32)
    q = torch.randn((N * rows, Hkv, d), generator=gen, device=dev).to(torch.bfloat16)
    lens, cu = torch.full((N,), length, **i32), torch.arange(0, N * rows + 1, rows, **i32)
    out = torch.full((N * rows, Hkv, K), -7, **i32)
    need = attn.select_blocks_workspace_bytes(N * rows, N, rows, Hkv, d, width)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    held = (q, bounds, table, cu, lens, out, ws)
    args = (q.data_ptr(), bounds.data_ptr(), table.data_ptr(), cu.data_ptr(), lens.data_ptr(), out.data_ptr(), K, 1, 2,
            N * rows, N, rows, Hkv, Hkv, d, 16, width, 64, ws.data_ptr(), need, stream.cuda_stream)
    fn = attn.lib().attn_select_blocks
    assert fn.argtypes == _SIGNATURES["attn_select_blocks"][1]
    return (lambda: fn(*args)), held, lambda: attn.select_blocks(q, bounds, table, lens, K, cu_seqlens_q=cu, max_seqlen_q=rows)


# wide beside narrow tables, and one row beside four: the largest and the smallest need of each kernel
@pytest.mark.parametrize("one,other", [
    ((4, 12000, 1, 80, 64), (4, 300, 1, 80, 64)),          # select_kernel<128, cached>
    ((1, 12000, 1, 2, 128), (1, 1300, 1, 2, 128)),         # select_kernel<1024, cached>
    ((1, 200000, 2, 1, 64), (1, 13000, 2, 1, 64)),         # select_kernel<1024, not cached>
    ((40, 300, 1, 9, 128), (40, 300, 4, 9, 128)),          # score_few_kernel, one and four rows
    ((40, 300, 2, 9, 256), (40, 300, 3, 9, 256)),
    ((8, 300, 1, 38, 128), (8, 50, 1, 38, 128)),           # select_one_kernel
])
def test_select_from_two_host_threads(attn, gpu, one, other):
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [_call(attn, gpu, *shape, stream) for shape, stream in zip((one, other), streams)]
    torch.cuda.synchronize()
    failed = [0, 0]
    ready = threading.Barrier(2)

    def work(i):
        torch.cuda.set_device(gpu)
        ready.wait()
        for _ in range(CALLS):
            failed[i] += calls[i][0]() != 0

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for _, held, alone in calls:
        assert torch.equal(held[5], alone())
