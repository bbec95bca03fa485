"""Calls on another stream than the current one, with everything that they need allocated inside, while the
current stream is busy.

Memory that a program has freed on the current stream may be handed out again at once there, although work that
uses it is still to run.  A call on another stream must not get such memory: its results and that work would
overwrite each other.  And what a call returns may be used and freed on the current stream.  Equal means equal bits:
every call is compared with itself on the current stream.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 16
BUSY = 500_000_000   # cycles: a quarter of a second
BLOCKS = [1 << 9, 1 << 12, 1 << 16, 1 << 19, 1 << 20, 1 << 21, 1 << 22, 3 << 21, 1 << 23, 1 << 24]


def _randn(shape, seed, dev):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(dev)


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _calls(attn, dev):
    """(name, call that takes a stream) of every function of the package that allocates."""
    N, Hq, Hkv, d, blocks = 2, 8, 2, 128, 40
    lens = [300, 150]
    q1, q = _randn((N, Hq, d), 1, dev), _randn((64, Hq, d), 2, dev)
    kc, vc = _randn((blocks, PAGE, Hkv, d), 3, dev), _randn((blocks, PAGE, Hkv, d), 4, dev)
    bt = torch.randperm(blocks, generator=torch.Generator().manual_seed(5))[:N * 20].view(N, 20).to(torch.int32).to(dev)
    sl, cu = _i32(lens, dev), _i32([0, 40, 64], dev)
    k, v = _randn((64, Hkv, d), 6, dev), _randn((64, Hkv, d), 7, dev)
    cache = attn.cache_q4_empty(blocks, Hkv, d, device=dev)
    attn.cache_append_q4(kc.view(-1, Hkv, d), vc.view(-1, Hkv, d), torch.arange(blocks * PAGE, dtype=torch.int32, device=dev),
                         cache)
    table, pos = attn.rope_table(512, d, device=dev), torch.arange(64, dtype=torch.int32, device=dev)
    cached, new, free = _i32([16, 32], dev), _i32([40, 24], dev), torch.arange(blocks, dtype=torch.int32, device=dev)
    part_o = torch.randn((32, 4, d), generator=torch.Generator().manual_seed(8)).to(dev)
    part_m, part_l = torch.zeros((32, 4), device=dev), torch.ones((32, 4), device=dev)
    own_bt = bt.clone()                                       # extended in place, by the same pages every time
    paged = (kc, vc, bt, sl)
    host = [x.cpu().pin_memory() for x in (q, k, v)]
    return [
        ("decode_paged_q4", lambda **s: attn.decode_paged_q4(q1, cache, bt, sl, **s)),
        ("prefill_paged_q4", lambda **s: attn.prefill_paged_q4(q, cache, bt, cu, sl, 40, **s)),
        # the rows behind a sequence's end are not written: compared where they are
        ("cache_gather_q4", lambda **s: [x[n, :lens[n]] for x in attn.cache_gather_q4(cache, bt, sl, **s)
                                         for n in range(N)]),
        ("qk_norm_rope", lambda **s: attn.qk_norm_rope(q, k, pos, table, **s)),
        ("step_tables", lambda **s: attn.step_tables(cached, new, free, own_bt, 64, blocks, **s)),
        ("rope_table", lambda **s: [attn.rope_table(512, d, device=dev, **s)]),
        ("prefill", lambda **s: attn.prefill(q[None], k[None], v[None], **s)),
        ("prefill_varlen", lambda **s: attn.prefill_varlen(q, k, v, cu, 40, **s)),
        ("prefill_paged", lambda **s: attn.prefill_paged(q, kc, vc, bt, cu, sl, 40, **s)),
        ("decode_paged", lambda **s: attn.decode_paged(q1, *paged, num_splits=4, **s)),
        ("decode_paged balanced", lambda **s: attn.decode_paged(q1, *paged, num_splits=0, **s)),
        ("decode_paged_noalloc", lambda **s: attn.decode_paged_noalloc(q1, *paged, num_splits=2, **s)),
        ("decode_paged_emulated", lambda **s: attn.decode_paged_emulated(q1, *paged, numerics="trt", **s)[:2]),
        ("combine", lambda **s: attn.combine(part_o, part_m, part_l, **s)),
        ("merge_emulated", lambda **s: attn.merge_emulated("triton", part_o, part_m, part_l, **s)),
        ("prefill_host", lambda **s: attn.prefill_host(*host, chunks=2, **s)),
    ]


NAMES = ["decode_paged_q4", "prefill_paged_q4", "cache_gather_q4", "qk_norm_rope", "step_tables", "rope_table", "prefill",
         "prefill_varlen", "prefill_paged", "decode_paged", "decode_paged balanced", "decode_paged_noalloc",
         "decode_paged_emulated", "combine", "merge_emulated", "prefill_host"]


def _busy_with_freed_blocks(dev):
    """Work on the current stream that is still to write and read blocks which are free again for it."""
    torch.cuda._sleep(BUSY)
    seen = []
    for size in BLOCKS:
        for _ in range(2):
            b = torch.empty(size, dtype=torch.uint8, device=dev)
            b.fill_(0xFF)
            seen.append(b.clone())
            del b
    return seen


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_a_side_stream_has_memory_of_its_own(attn, gpu, name, handle):
    calls = dict(_calls(attn, gpu))
    assert list(calls) == NAMES
    call = calls[name]
    side = torch.cuda.Stream()
    given = dict(stream=side.cuda_stream if handle else side)
    want = call()
    torch.cuda.synchronize()
    want = [x.clone() for x in want]
    first = call(**given)                                     # the side stream's pool gets its memory
    del first
    torch.cuda.synchronize()
    for _ in range(2):
        seen = _busy_with_freed_blocks(gpu)
        busy = torch.cuda.Event()
        busy.record()
        got = call(**given)
        side.synchronize()
        assert not busy.query()                               # the call did not wait for the current stream
        # the results are used on the current stream, and freed there before that use has run
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(BUSY // 4)
        kept = [x.clone() if x.is_cuda else x for x in got]
        sizes = [(x.shape, x.dtype) for x in got if x.is_cuda]
        del got
        with torch.cuda.stream(side):
            for shape, dtype in sizes * 2:
                torch.full(shape, 99, dtype=dtype, device=gpu)
        torch.cuda.synchronize()
        assert all((b == 0xFF).all() for b in seen)
        assert len(kept) == len(want)
        for a, b in zip(kept, want):
            assert torch.equal(a, b) or np.array_equal(a.cpu().float().numpy(), b.cpu().float().numpy(), equal_nan=True)


def test_a_captured_call_on_a_forked_stream(attn, gpu):
    """Inside a capture, on a stream forked from the capturing one, everything allocated there."""
    calls = dict(_calls(attn, gpu))
    names = ["decode_paged_q4", "prefill_paged_q4", "qk_norm_rope", "decode_paged"]
    want = [[x.clone() for x in calls[n]()] for n in names]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [calls[n](stream=side) for n in names]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for outs in got:
            for x in outs:
                x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_default_stream_by_its_handle(attn, gpu):
    """Handle 0 is the default stream, from another current stream too."""
    x = _randn((64, 8, 128), 1, gpu)
    want = attn.qk_norm_rope(x, x, None, None, stream=0)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = attn.qk_norm_rope(x, x, None, None, stream=0)
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, x) for a, b in zip(got, want))
