"""The 4-bit cache's binding without a GPU: what it refuses before it calls the library."""
import pytest
import torch

from mixed_bit_kv_gb300 import rdkv


def _cache(batch=2, h_kv=3, head_dim=64):
    cache = rdkv.Q4Cache.__new__(rdkv.Q4Cache)       # the checks alone, on CPU tensors
    cache.batch, cache.h_kv, cache.head_dim, cache.device, cache._seen = batch, h_kv, head_dim, torch.device("cpu"), {}
    return cache


def test_selections_need_their_own_shape_and_a_page():
    cache = _cache()
    sel = torch.zeros(2, 4, 3, 5, dtype=torch.int32)
    assert rdkv._q4_selection(cache, None, 4) == (0, None)
    assert rdkv._q4_selection(cache, sel, 4) == (5, sel.data_ptr())
    one = sel[:, :1].contiguous()
    assert rdkv._q4_selection(cache, one, 1) == rdkv._q4_selection(cache, one.view(2, 3, 5), 1) == (5, one.data_ptr())
    # no page at all (its pointer would be NULL: every position), and as many numbers in another order
    for bad, n_q in ((sel[..., :0], 4), (sel[..., :0].contiguous(), 4), (torch.empty(2, 3, 0, dtype=torch.int32), 1),
                     (sel.transpose(1, 2).contiguous(), 4), (sel.view(4, 2, 3, 5), 4), (sel.view(2, 12, 5), 4), (sel.view(-1), 4),
                     (one.view(2, 3, 5), 2), (sel[:, :2], 4), (sel[:1], 4), (sel.long(), 4), (sel.transpose(2, 3), 4),
                     (sel[..., ::2], 4), (torch.tensor(1, dtype=torch.int32), 1)):
        with pytest.raises(rdkv.RDKVError):
            rdkv._q4_selection(cache, bad, n_q)
