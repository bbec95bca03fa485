"""Refusals of the serving-step entry points: every host check returns before any CUDA call, so they run
without a GPU.  And the oracle's number format, checked by what it promises."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.step as os_

FAKE = 0x10000  # an aligned non-null address; never dereferenced by the host checks


def _call(attn, fn, base, over):
    a = dict(base, **over)
    assert set(over) <= set(base)
    return getattr(attn.lib(), fn)(*a.values())


TABLES = dict(cached=FAKE, new=FAKE, free=FAKE, bt=FAKE, sl=FAKE, cu=FAKE, pos=FAKE, slots=FAKE, used=FAKE, N=2, T=8,
              nf=4, page=16, maxb=4, nblocks=8, stream=None)


@pytest.mark.parametrize("over,want", [
    (dict(cached=None), 1), (dict(new=None), 1), (dict(bt=FAKE + 2), 1), (dict(sl=None), 1), (dict(cu=None), 1),
    (dict(used=None), 1), (dict(pos=None), 1), (dict(slots=None), 1), (dict(free=None), 1), (dict(N=0), 1),
    (dict(T=-1), 1), (dict(nf=-1), 1), (dict(maxb=0), 1), (dict(nblocks=0), 1), (dict(page=32), 2),
    (dict(nblocks=1 << 27), 1), (dict(maxb=1 << 27), 1), (dict(N=(1 << 24) + 1), 1),
])
def test_step_tables_refusals(attn, over, want):
    assert _call(attn, "attn_step_tables", TABLES, over) == want


def _apart():
    """TABLES with a megabyte between the tensors."""
    names = ["cached", "new", "free", "bt", "sl", "cu", "pos", "slots", "used"]
    return dict(TABLES, **{n: FAKE + (i << 20) for i, n in enumerate(names)})


@pytest.mark.parametrize("out,other,by", [
    ("sl", "cached", 0), ("sl", "new", 0), ("cu", "cached", 0), ("cu", "cached", -8), ("sl", "cached", 4),
    ("pos", "new", 4), ("slots", "free", 12), ("used", "free", 0), ("used", "cached", 4), ("pos", "slots", -28),
    ("cu", "sl", 4), ("bt", "free", -28), ("bt", "cached", 0), ("used", "bt", 28), ("sl", "bt", -4), ("slots", "cu", 8),
])
def test_step_tables_refuses_outputs_in_other_tensors(attn, out, other, by):
    """Whole or by one element, at either end: N = 2, T = 8, 4 free pages, a table of 2 x 4."""
    a = _apart()
    assert getattr(attn.lib(), "attn_step_tables")(*dict(a, **{out: a[other] + by}).values()) == 1


@pytest.mark.parametrize("args,want", [
    ((None, 10, 32, 1e4, None), 1), ((FAKE + 4, 10, 32, 1e4, None), 1), ((FAKE, 0, 32, 1e4, None), 1),
    ((FAKE, 10, 0, 1e4, None), 1), ((FAKE, 10, 32, 0.0, None), 1), ((FAKE, 10, 32, float("inf"), None), 1),
    ((FAKE, 10, 24, 1e4, None), 2), ((FAKE, 10, 272, 1e4, None), 2),
])
def test_rope_table_refusals(attn, args, want):
    assert attn.lib().attn_rope_table(*args) == want


ROPE = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, table=FAKE,
            maxp=100, rot=128, inter=0, qo=FAKE, qos=1024, ko=FAKE, kos=256, kc=FAKE, vc=FAKE, slots=FAKE, T=4, Hq=8,
            Hkv=2, d=128, page=16, nblocks=4, stream=None)


@pytest.mark.parametrize("over,want", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(q=FAKE + 8), 1), (dict(qw=FAKE + 2), 1),
    (dict(T=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(d=96), 2), (dict(qs=1020), 1), (dict(qs=1016), 1),
    (dict(ks=128), 1), (dict(qos=1000), 1), (dict(kos=255), 1), (dict(vs=8), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(rot=-16), 1), (dict(rot=144), 1), (dict(rot=24), 2), (dict(pos=None), 1),
    (dict(table=None), 1), (dict(maxp=0), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(v=None), 1),
    (dict(slots=None), 1), (dict(nblocks=0), 1), (dict(page=8), 2),
    (dict(kc=None, vc=None, ko=None), 1),                    # nowhere to put K
    (dict(T=1 << 27), 1),
])
def test_qk_norm_rope_refusals(attn, over, want):
    assert _call(attn, "attn_qk_norm_rope", ROPE, over) == want


APPEND = dict(k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, cache=FAKE, T=4, Hkv=2, d=128, page=16, nblocks=4,
              stream=None)


@pytest.mark.parametrize("over,want", [
    (dict(k=None), 1), (dict(v=FAKE + 4), 1), (dict(slots=None), 1), (dict(cache=FAKE + 8), 1), (dict(T=0), 1),
    (dict(Hkv=0), 1), (dict(nblocks=0), 1), (dict(page=32), 2), (dict(d=32), 2), (dict(ks=252), 1), (dict(vs=128), 1),
])
def test_cache_append_refusals(attn, over, want):
    assert _call(attn, "attn_cache_append_q4", APPEND, over) == want


GATHER = dict(cache=FAKE, bt=FAKE, sl=FAKE, ko=FAKE, vo=FAKE, N=2, Hkv=2, d=128, page=16, maxb=4, nblocks=4,
              stream=None)
DECODE = dict(q=FAKE, cache=FAKE, bt=FAKE, sl=FAKE, o=FAKE, lse=None, N=2, Hq=8, Hkv=2, d=128, page=16, maxb=4,
              nblocks=4, scale=0.1, ws=FAKE, wsb=1 << 30, stream=None)
PREFILL = dict(q=FAKE, cache=FAKE, bt=FAKE, cu=FAKE, sl=FAKE, o=FAKE, lse=None, N=2, maxq=8, T=10, Hq=8, Hkv=2,
               d=128, page=16, maxb=4, nblocks=4, scale=0.1, causal=1, ws=FAKE, wsb=1 << 30, stream=None)
SHARED = [(dict(cache=None), 1), (dict(bt=FAKE + 2), 1), (dict(sl=None), 1), (dict(N=0), 1), (dict(Hkv=0), 1),
          (dict(d=96), 2), (dict(page=32), 2), (dict(maxb=0), 1), (dict(nblocks=0), 1), (dict(N=65536), 1),
          (dict(nblocks=1 << 27), 1)]


@pytest.mark.parametrize("over,want", SHARED + [(dict(ko=None), 1), (dict(vo=FAKE + 8), 1)])
def test_cache_gather_refusals(attn, over, want):
    assert _call(attn, "attn_cache_gather_q4", GATHER, over) == want


@pytest.mark.parametrize("over,want", SHARED + [
    (dict(q=None), 1), (dict(o=FAKE + 2), 1), (dict(lse=FAKE + 2), 1), (dict(Hq=7), 1), (dict(Hq=0), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(ws=None), 3), (dict(ws=FAKE + 4), 3),
])
def test_decode_q4_refusals(attn, over, want):
    assert _call(attn, "attn_decode_paged_q4", DECODE, over) == want


@pytest.mark.parametrize("over,want", SHARED + [
    (dict(q=None), 1), (dict(o=None), 1), (dict(cu=None), 1), (dict(maxq=0), 1), (dict(T=0), 1), (dict(Hq=7), 1),
    (dict(scale=-1.0), 1), (dict(ws=None), 3), (dict(ws=FAKE + 16), 3), (dict(wsb=1000), 3),
    (dict(maxq=128 * 65536), 1),
])
def test_prefill_q4_refusals(attn, over, want):
    assert _call(attn, "attn_prefill_paged_q4", PREFILL, over) == want


def test_sizes(attn):
    L = attn.lib()
    assert [L.attn_cache_q4_record_bytes(d) for d in (64, 96, 128, 256)] == [1088, 0, 2176, 4352]
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert L.attn_prefill_q4_workspace_bytes(3, 2, 64, 5) == 2 * up(15 * 16 * 2 * 64 * 2) + up(60)
    assert L.attn_prefill_q4_workspace_bytes(3, 2, 96, 5) == 0
    assert L.attn_prefill_q4_workspace_bytes(1 << 10, 2, 64, 1 << 20) == 0
    assert L.attn_decode_q4_workspace_bytes(96) == 0


def test_wrappers_refuse_host_tensors(attn):
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.qk_norm_rope(x, x, None, None)
    with pytest.raises(ValueError):
        attn.cache_append_q4(x, x, i, torch.zeros((1, 2, 17 * 64), dtype=torch.uint8))
    with pytest.raises(ValueError):
        attn.decode_paged_q4(x, torch.zeros((1, 2, 17 * 64), dtype=torch.uint8), i.view(2, 1), i)
    with pytest.raises(ValueError):
        attn.step_tables(i, i, i, i.view(2, 1), 4, 4)
    with pytest.raises(ValueError):
        attn.cache_q4_empty(4, 2, 96)


@pytest.mark.parametrize("device", ["cpu", "cpu:0", torch.device("cpu")])
def test_wrappers_refuse_other_devices_by_name(attn, device):
    with pytest.raises(ValueError):
        attn.rope_table(16, 16, device=device)
    with pytest.raises(ValueError):
        attn.decode_q4_workspace_bytes(64, device=device)


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("make", [
    lambda r: r.standard_normal((40, 128)),
    lambda r: r.standard_normal((40, 128)) * 10.0 ** r.uniform(-20, 20, (40, 1)),
    lambda r: np.abs(r.standard_normal((40, 128))) + 3,           # one sign: the range still holds 0
    lambda r: np.where(r.random((40, 128)) < 0.02, 100.0, 1.0) * r.standard_normal((40, 128)),
    lambda r: r.integers(-15, 16, (40, 128)) * 2.0 ** r.integers(-5, 5, (40, 1)),  # ties and exact grids
    lambda r: np.zeros((4, 64)),
])
def test_stored_values_are_bf16_and_near(make):
    x = _bf16(make(np.random.default_rng(3)))
    codes, scale, zero = os_.quantise(x)
    y = os_.stored(x)
    assert codes.min() >= 0 and codes.max() <= 15 and zero.min() >= 0 and zero.max() <= 15
    assert np.array_equal(y, _bf16(y))                            # exactly bf16 numbers
    step = np.repeat(scale, 64, -1)
    assert (np.abs(x - y) <= step / 2).all()
    again, scale2, _ = os_.quantise(y)                            # storing them again never widens the step
    assert (scale2 <= scale).all()


def test_record_layout_is_a_bijection():
    """Each nibble of a record's code bytes belongs to one (token, channel)."""
    for d in (64, 128, 256):
        per = min(2, d // 64)
        k_at, v_at = set(), set()
        for k in range(16):
            for ch in range(d):
                e, t, h, j = ch // 64, ch % 64 // 16, ch % 16 // 8, ch % 8
                word = e // per * (8 * per) + t * (2 * per) + e % per * 2 + h
                k_at.add((k * (d // 2) + 4 * word) * 2 + j)
                p = ch // 2
                byte = (p // 32 * 32 + p % 8 * 4 + k % 8 // 2) * 16 + p // 8 % 4 * 4 + k // 8 + 2 * (k % 2)
                v_at.add(byte * 2 + ch % 2)
        assert k_at == set(range(16 * d)) and v_at == set(range(16 * d))
