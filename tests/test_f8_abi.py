"""Refusals of the 8-bit cache's and of block selection's entry points: every host check returns before any CUDA call,
so they run without a GPU.  And the oracle's number format and layout, checked by what they promise."""
import numpy as np
import pytest
import torch

import oracle.f8 as o8

FAKE = 0x10000  # an aligned non-null address; never dereferenced by the host checks


def _call(attn, fn, base, over):
    assert set(over) <= set(base)
    return getattr(attn.lib(), fn)(*dict(base, **over).values())


APPEND = dict(k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, cache=FAKE, bounds=FAKE, T=4, Hkv=2, d=128, page=16, nblocks=4,
              stream=None)
GATHER = dict(cache=FAKE, bt=FAKE, sl=FAKE, ko=FAKE, vo=FAKE, N=2, Hkv=2, d=128, page=16, maxb=4, nblocks=4,
              stream=None)
DECODE = dict(q=FAKE, cache=FAKE, bt=FAKE, sl=FAKE, o=FAKE, lse=None, N=2, Hq=8, Hkv=2, d=128, page=16, maxb=4,
              nblocks=4, scale=0.1, ws=FAKE, wsb=1 << 30, stream=None)
BLOCKS = dict(q=FAKE, cache=FAKE, bt=FAKE, cu=FAKE, sl=FAKE, blocks=FAKE, K=3, o=FAKE, lse=None, T=5, N=2, Hq=8, Hkv=2,
              d=128, page=16, maxb=4, nblocks=4, scale=0.1, ws=FAKE, wsb=1 << 30, stream=None)
PREFILL = dict(q=FAKE, cache=FAKE, bt=FAKE, cu=FAKE, sl=FAKE, o=FAKE, lse=None, N=2, maxq=8, T=10, Hq=8, Hkv=2,
               d=128, page=16, maxb=4, nblocks=4, scale=0.1, causal=1, ws=FAKE, wsb=1 << 30, stream=None)
SELECT = dict(q=FAKE, bounds=FAKE, bt=FAKE, cu=FAKE, sl=FAKE, blocks=FAKE, K=4, first=1, last=2, T=5, N=2, maxq=4, Hq=8,
              Hkv=2, d=128, page=16, maxb=4, nblocks=4, ws=FAKE, wsb=1 << 30, stream=None)
TABLES = [(dict(bt=FAKE + 2), 1), (dict(bt=None), 1), (dict(sl=None), 1), (dict(N=0), 1), (dict(Hkv=0), 1),
          (dict(d=96), 2), (dict(page=32), 2), (dict(maxb=0), 1), (dict(nblocks=0), 1), (dict(N=65536), 1),
          (dict(nblocks=1 << 27), 1), (dict(maxb=1 << 27), 1)]
CACHE = TABLES + [(dict(cache=None), 1), (dict(cache=FAKE + 8), 1)]
ATTEND = CACHE + [(dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(o=FAKE + 2), 1), (dict(lse=FAKE + 2), 1),
                  (dict(Hq=7), 1), (dict(Hq=0), 1), (dict(Hq=65536), 1), (dict(scale=0.0), 1),
                  (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ws=None), 3), (dict(ws=FAKE + 4), 3)]


@pytest.mark.parametrize("over,want", [
    (dict(k=None), 1), (dict(v=FAKE + 4), 1), (dict(slots=None), 1), (dict(slots=FAKE + 2), 1), (dict(cache=FAKE + 8), 1),
    (dict(cache=None), 1), (dict(bounds=FAKE + 2), 1), (dict(T=0), 1), (dict(T=(1 << 30) + 1), 1), (dict(Hkv=0), 1),
    (dict(Hkv=65536), 1), (dict(nblocks=0), 1), (dict(nblocks=1 << 27), 1), (dict(page=32), 2), (dict(d=32), 2),
    (dict(ks=252), 1), (dict(vs=128), 1), (dict(ks=(1 << 32) + 8), 1),
])
def test_append_refusals(attn, over, want):
    assert _call(attn, "attn_cache_append_f8", APPEND, over) == want


@pytest.mark.parametrize("over,want", CACHE + [(dict(ko=None), 1), (dict(vo=FAKE + 8), 1),
                                               (dict(maxb=1 << 26, Hkv=64), 1)])
def test_gather_refusals(attn, over, want):
    assert _call(attn, "attn_cache_gather_f8", GATHER, over) == want


@pytest.mark.parametrize("over,want", ATTEND)
def test_decode_refusals(attn, over, want):
    assert _call(attn, "attn_decode_paged_f8", DECODE, over) == want


@pytest.mark.parametrize("over,want", ATTEND + [
    (dict(blocks=None), 1), (dict(blocks=FAKE + 1), 1), (dict(K=0), 1), (dict(K=(1 << 18) + 1), 1), (dict(T=0), 1),
    (dict(T=(1 << 30) + 1), 1), (dict(cu=None), 1), (dict(cu=FAKE + 2), 1)])
def test_decode_blocks_refusals(attn, over, want):
    assert _call(attn, "attn_decode_blocks_f8", BLOCKS, over) == want


@pytest.mark.parametrize("over,want", CACHE + [
    (dict(q=None), 1), (dict(o=None), 1), (dict(cu=None), 1), (dict(maxq=0), 1), (dict(T=0), 1), (dict(Hq=7), 1),
    (dict(scale=-1.0), 1), (dict(ws=None), 3), (dict(ws=FAKE + 16), 3), (dict(wsb=1000), 3),
    (dict(maxq=128 * 65536), 1),
])
def test_prefill_refusals(attn, over, want):
    assert _call(attn, "attn_prefill_paged_f8", PREFILL, over) == want


@pytest.mark.parametrize("over,want", TABLES + [
    (dict(q=None), 1), (dict(bounds=None), 1), (dict(bounds=FAKE + 8), 1), (dict(blocks=None), 1),
    (dict(cu=FAKE + 2), 1), (dict(cu=None), 1), (dict(cu=None, T=2, maxq=2), 1), (dict(Hq=7), 1), (dict(Hq=0), 1),
    (dict(K=0), 1), (dict(first=-1), 1), (dict(last=0), 1), (dict(first=3), 1), (dict(last=4), 1),
    (dict(first=1 << 30, last=1 << 30), 1), (dict(K=(1 << 18) + 1), 1), (dict(T=0), 1), (dict(maxq=0), 1),
    (dict(maxb=(1 << 18) + 1), 2), (dict(T=1 << 29, N=65535, maxq=1 << 29), 1), (dict(T=1 << 30), 1), (dict(ws=None), 3), (dict(ws=FAKE + 128), 3),
    (dict(wsb=100), 3),
])
def test_select_refusals(attn, over, want):
    assert _call(attn, "attn_select_blocks", SELECT, over) == want


def test_sizes(attn):
    L = attn.lib()
    assert [L.attn_cache_f8_record_bytes(d) for d in (64, 96, 128, 256)] == [2064, 0, 4112, 8208]
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert L.attn_prefill_f8_workspace_bytes(3, 2, 64, 5) == 2 * up(15 * 16 * 2 * 64 * 2) + up(60)
    assert L.attn_prefill_f8_workspace_bytes(3, 2, 96, 5) == 0
    assert L.attn_decode_f8_workspace_bytes(96) == 0
    few = up(10 * 104 * 4) + up(40) + up(6 * 7 * 4)
    assert L.attn_select_blocks_workspace_bytes(5, 3, 1, 2, 128, 100) == few
    assert L.attn_select_blocks_workspace_bytes(5, 3, 4, 2, 128, 100) == few
    # a row tile of 64 rows (32 at d = 256) for each sequence, and one for each 64 rows
    assert L.attn_select_blocks_workspace_bytes(5, 3, 5, 2, 128, 100) == few + 4 * 2 * 64 * 8 * 128
    assert L.attn_select_blocks_workspace_bytes(5, 3, 5, 2, 256, 100) == few + 4 * 2 * 32 * 8 * 256
    for bad in ((0, 3, 1, 2, 128, 100), (5, 3, 0, 2, 128, 100), (5, 3, 1, 2, 96, 100), (5, 3, 1, 2, 128, (1 << 18) + 1),
                (65535, 65535, 1, 1024, 128, 1000)):
        assert L.attn_select_blocks_workspace_bytes(*bad) == 0


def test_wrappers_refuse(attn):
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros((1, 2, 32 * 64 + 16), dtype=torch.uint8)
    bounds = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: attn.cache_append_f8(x, x, i, cache), lambda: attn.cache_gather_f8(cache, i.view(2, 1), i),
                 lambda: attn.decode_paged_f8(x, cache, i.view(2, 1), i),
                 lambda: attn.decode_blocks_f8(x, cache, i.view(2, 1), i, i.view(2, 1, 1)),
                 lambda: attn.prefill_paged_f8(x, cache, i.view(2, 1), i, i, 1),
                 lambda: attn.select_blocks(x, bounds, i.view(2, 1), i, 4),
                 lambda: attn.cache_f8_empty(4, 2, 96), lambda: attn.key_bounds_empty(4, 2, 96),
                 lambda: attn.decode_f8_workspace_bytes(64, device="cpu")):
        with pytest.raises(ValueError):
            call()


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("make", [
    lambda r: r.standard_normal((16, 128)),
    lambda r: r.standard_normal((16, 128)) * 10.0 ** r.uniform(-36, 36),
    lambda r: np.where(r.random((16, 128)) < 0.02, 400.0, 1.0) * r.standard_normal((16, 128)),
    lambda r: (r.integers(16, 33, (16, 128)) + 0.5) * 2.0 ** r.integers(-12, 4, (16, 1)),   # ties
    lambda r: np.full((16, 64), 448.0), lambda r: np.full((16, 64), 450.0), lambda r: np.zeros((16, 64)),
])
def test_stored_values_are_bf16_and_near(make):
    x = _bf16(make(np.random.default_rng(3)))
    page = o8.Page(x.shape[1])
    page.write(0, x)
    y = page.values()
    assert np.array_equal(y, _bf16(y))                            # exactly bf16 numbers
    assert np.abs(page.codes).max() <= 448
    unit = 2.0 ** page.e
    assert (np.abs(x - y) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * unit)).all()
    # the numbers are those of torch's type, rounded its way
    t = torch.from_numpy(x / unit).to(torch.float8_e4m3fn)
    assert np.array_equal(t.double().numpy(), page.codes)
    assert set(np.unique(np.abs(page.codes))) <= set(o8.code_numbers()[:127])
    # a larger scale keeps the numbers that it can
    before = page.values().copy()
    page.write(15, np.full((1, x.shape[1]), 16 * max(np.abs(x).max(), 1e-30)))
    grid = 2.0 ** (page.e - 9)
    moved = page.values()[:15]
    assert (np.abs(moved - before[:15]) <= grid / 2).all()
    assert np.array_equal(moved[np.abs(moved) >= 16 * grid], before[:15][np.abs(moved) >= 16 * grid])


def test_code_numbers_are_e4m3():
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o8.code_numbers(), want, equal_nan=True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_record_layout_is_a_bijection(d):
    at = [f(k, c, d) for f in (o8.k_byte, o8.v_byte) for k in range(16) for c in range(d)]
    assert sorted(at) == list(range(32 * d))
