"""Waits of the 4-bit decode that run out: the call ends soon, with a status, and the GPU stays usable.

The kernel's computing warps wait for copies and for their merge buffer, its loading warp for free slots and for
the warps' states.  Each wait gives up after ATTN_WAIT_LIMIT_NS and records device status 1; a warp whose wait ran
out makes no other, so that a call is over after a few limits however many sequences its shares hold.  A test-only
build with a limit of 2 ms and ATTN_TEST_DROP_COPY makes the waits of one CTA run out: its first copy is left out,
or its loading warp leaves at once.  Nothing faults, traps or hangs.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.step as os_
from attention_attn_prefill_gb300._lib import _SIGNATURES

pytestmark = pytest.mark.gpu

WAIT_LIMIT_NS = 2_000_000
PAGE = 16


@pytest.fixture(scope="module")
def lib():
    from attention_attn_prefill_gb300.build import build
    path = build(variant="waittest", extra_flags=["-DATTN_TEST_DROP_COPY", f"-DATTN_WAIT_LIMIT_NS={WAIT_LIMIT_NS}ull"])
    handle = ctypes.CDLL(path)
    for name in ("attn_decode_paged_q4", "attn_decode_q4_workspace_bytes", "attn_device_status"):
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = _SIGNATURES[name]
    handle.attn_test_drop_copy_q4.restype = ctypes.c_int
    handle.attn_test_drop_copy_q4.argtypes = [ctypes.c_int]
    return handle


def _status(lib):
    code = ctypes.c_uint32(0)
    assert lib.attn_device_status(ctypes.byref(code), 1) == 0
    return int(code.value)


def _decode(lib, q, cache, bt, sl):
    """(o, ms) of a call whose output holds NaN before."""
    N, Hq, d = q.shape
    o = torch.full_like(q, float("nan"))
    need = lib.attn_decode_q4_workspace_bytes(d)
    ws = torch.zeros(need, dtype=torch.uint8, device=q.device)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    torch.cuda.synchronize()
    start.record()
    st = lib.attn_decode_paged_q4(q.data_ptr(), cache.data_ptr(), bt.data_ptr(), sl.data_ptr(), o.data_ptr(), 0, N, Hq,
                                  cache.shape[1], d, PAGE, bt.shape[1], cache.shape[0], d ** -0.5, ws.data_ptr(), need,
                                  torch.cuda.current_stream().cuda_stream)
    end.record()
    torch.cuda.synchronize()
    assert st == 0                      # the launch itself is fine; the error is recorded on the device
    return o, start.elapsed_time(end)


@pytest.mark.parametrize("drop", [1, 2])
@pytest.mark.parametrize("N,length,Hq,Hkv,d", [
    (3, 700, 8, 2, 128),                # one or two segments a share, a descriptor a pair
    (20000, 16, 4, 2, 64),              # 66 segments a share and more
    (20000, 16, 5, 1, 128), (20000, 16, 2, 1, 256),
])
def test_waits_that_run_out_end_with_a_status(attn, gpu, lib, drop, N, length, Hq, Hkv, d):
    pages = (length + PAGE - 1) // PAGE
    blocks = 3 * pages                  # three sequences' pages, shared by all
    gen = torch.Generator().manual_seed(N + d)
    k, v = (torch.randn((blocks * PAGE, Hkv, d), generator=gen).to(torch.bfloat16) for _ in "kv")
    q = torch.randn((N, Hq, d), generator=gen).to(torch.bfloat16).to(gpu)
    cache = attn.cache_q4_empty(blocks, Hkv, d, device=gpu)
    attn.cache_append_q4(k.to(gpu), v.to(gpu), torch.arange(blocks * PAGE, dtype=torch.int32, device=gpu), cache)
    which = torch.arange(N) % 3
    bt = (which[:, None] * pages + torch.arange(pages)).to(torch.int32).to(gpu)
    sl = torch.full((N,), length, dtype=torch.int32, device=gpu)
    assert _status(lib) == 0
    want, quick = _decode(lib, q, cache, bt, sl)
    assert _status(lib) == 0 and torch.isfinite(want).all()

    assert lib.attn_test_drop_copy_q4(drop) == 0
    o, ms = _decode(lib, q, cache, bt, sl)
    assert lib.attn_test_drop_copy_q4(0) == 0
    assert _status(lib) == 1            # kDevWaitTimeout
    # a warp's own wait, one for each of the others' and the loading warp's, the drain of three slots: 6 limits
    assert ms < 8 * WAIT_LIMIT_NS * 1e-6 + quick, ms
    # what the CTA at fault had no part in is there: all but its share of the sequences, and those cut at its ends
    same = (o == want).all(-1).all(-1)
    if N > 3:
        assert int(same.sum()) > N - N // 100 - 3 and same[N // 2:].all()

    again, _ = _decode(lib, q, cache, bt, sl)
    assert _status(lib) == 0 and torch.equal(again, want)
    # and right: a sequence of each kind against the definition
    ks, vs = (os_.stored(x.double().numpy()).reshape(3, pages * PAGE, Hkv, d)[:, :length] for x in (k, v))
    for n in (0, N // 2, N - 1):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = ks[n % 3, :, g] @ q[n, h].double().cpu().numpy() / math.sqrt(d)
            p = np.exp(s - s.max())
            assert np.abs(again[n, h].double().cpu().numpy() - p @ vs[n % 3, :, g] / p.sum()).max() <= 2e-2
