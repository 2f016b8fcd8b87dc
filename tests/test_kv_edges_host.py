"""Refusals of the key/value cache's calls that test_kv_host.py does not reach, on the host."""
import pytest
import torch

import nvfp4_adaptive_block_amd as fos


@pytest.mark.parametrize("name", ["budget", "sinks", "recent"])
@pytest.mark.parametrize("far", [2 ** 31, 2 ** 32, 2 ** 32 + 4, 2 ** 63, -2 ** 31 - 1, 4 - 2 ** 32])
def test_shares_past_32_bits_are_refused(name, far):
    """Cut to 32 bits they would be shares to evict by: a budget of 2^32 one of 0."""
    k, v = (fos.fos_kv_cache(3, 2, 16, 64, device="cpu") for _ in range(2))
    table, lens, acc = torch.zeros(2, 3).int(), torch.zeros(2).int(), torch.zeros(2, 2, 48)
    shares = dict(budget=4, sinks=0, recent=0)
    shares[name] = far
    with pytest.raises(ValueError, match=name):
        fos.fos_kv_evict(acc, k, v, table, lens, shares.pop("budget"), **shares)
    if name != "sinks":
        with pytest.raises(ValueError, match=name):
            fos.fos_kv_evict_workspace(2, 2, far if name == "budget" else 4, far if name == "recent" else 0)


@pytest.mark.parametrize("i", [1, 4, 5, 6])
def test_sizes_past_32_bits_have_no_workspace(i):
    sizes = [1, 8, 1, 4, 2, 64, 128]
    assert fos.fos_kv_attention_workspace(*sizes) >= 0
    sizes[i] += 2 ** 32
    with pytest.raises(ValueError):
        fos.fos_kv_attention_workspace(*sizes)
    with pytest.raises(ValueError):
        fos.fos_kv_evict_workspace(2, 2 ** 32 + 2, 10)
