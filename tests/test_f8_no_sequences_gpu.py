"""Steps without sequences over the 8-bit cache: every call checks its arguments and returns without a launch."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_step_without_sequences(attn, gpu):
    Hq, Hkv, d, width = 4, 2, 64, 5
    cache, bounds = attn.cache_f8_empty(3, Hkv, d, device=gpu), attn.key_bounds_empty(3, Hkv, d, device=gpu)
    i32 = dict(dtype=torch.int32, device=gpu)
    table, lens, cu = torch.zeros((0, width), **i32), torch.zeros((0,), **i32), torch.zeros((1,), **i32)
    q, k = (torch.zeros((0, H, d), dtype=torch.bfloat16, device=gpu) for H in (Hq, Hkv))
    attn.cache_append_f8(k, k, lens, cache, bounds=bounds)
    o, lse = attn.decode_paged_f8(q, cache, table, lens)
    assert o.shape == (0, Hq, d) and lse.shape == (0, Hq)
    assert attn.select_blocks(q, bounds, table, lens, 4).shape == (0, Hkv, 4)
    blocks = torch.zeros((0, Hkv, 4), **i32)
    assert attn.decode_blocks_f8(q, cache, table, lens, blocks)[0].shape == (0, Hq, d)
    assert attn.prefill_paged_f8(q, cache, table, cu, lens, 1)[0].shape == (0, Hq, d)
    k_out, v_out = attn.cache_gather_f8(cache, table, lens)
    assert k_out.shape == v_out.shape == (0, 16 * width, Hkv, d)
    with pytest.raises(ValueError):
        attn.decode_paged_f8(q.float(), cache, table, lens)
    assert attn.device_status() == 0
