"""The 4-bit cache's binding without a GPU: what it refuses before it calls the library."""
import ctypes
import os
import subprocess
import sys
import types

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


def test_the_timeout_selftest_refuses_limits_that_are_not_positive():
    import __graft_entry__
    __graft_entry__.build()
    L = rdkv.lib()
    c = rdkv.Q4CacheStruct(2, 2, 64, 8, 4, 4096, 8192, 256, 512, 1024)
    before = L.rdkv_launch_count()
    for withhold, cycles, h_q, ws, code in ((0, 1000, 4, 1 << 40, rdkv.RDKV_ERR_INVALID_ARG), (-1, 1000, 4, 1 << 40, rdkv.RDKV_ERR_INVALID_ARG),
                                            (1, 0, 4, 1 << 40, rdkv.RDKV_ERR_INVALID_ARG), (1, -5, 4, 1 << 40, rdkv.RDKV_ERR_INVALID_ARG),
                                            (1, 1000, 3, 1 << 40, rdkv.RDKV_ERR_INVALID_ARG), (1, 1000, 4, 16, rdkv.RDKV_ERR_WORKSPACE)):
        assert L.rdkv_q4_timeout_selftest(ctypes.byref(c), 0, 4096, 256, h_q, 1, None, 0, 4096, 0, None, 4096, ws, withhold, cycles,
                                          None) == code
        assert L.rdkv_last_error_string()
    assert L.rdkv_launch_count() == before


def test_the_binding_is_imported_by_a_torch_without_cuda_names():
    """As a torch built for the CPU has none of them: the module loads, and what needs a GPU says so."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda')]: delattr(torch._C, name)\n"
            "from mixed_bit_kv_gb300 import rdkv\n"
            "assert rdkv.lib().rdkv_version() >= 1\n"
            "try: rdkv.Q4Cache(1, 1, 64, 64, 'cpu')\n"
            "except rdkv.RDKVError: print('refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.strip() == "refused", got.stderr


def test_the_tensors_behind_the_struct_change_in_place_only():
    cache = rdkv.Q4Cache.__new__(rdkv.Q4Cache)
    for name in ("pages", "bounds", "page_table", "lens", "status"):
        t = torch.zeros(3, dtype=torch.int32)
        setattr(cache, name, t)
        assert getattr(cache, name) is t
        with pytest.raises(rdkv.RDKVError):
            setattr(cache, name, t + 1)
        assert getattr(cache, name) is t and (t == 0).all()
    cache.lens += 1                                  # the same tensor
    cache.lens[0] = 7
    assert cache.lens.tolist() == [7, 1, 1]
    cache = rdkv.Q4Cache.__new__(rdkv.Q4Cache)
    cache.bounds = None                              # a cache without bounds gets none later
    with pytest.raises(rdkv.RDKVError):
        cache.bounds = torch.zeros(3)


def test_a_stream_of_another_device_is_refused():
    """(It was passed over: the call ran on the current stream of the cache's device.)"""
    cache = _cache()
    cache.device, cache._index = torch.device("cuda", 0), 0
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    q = torch.zeros(2, 1, 3, 64)
    for call in (lambda: rdkv.rdkv_q4_write(cache, q, q, stream=stream), lambda: rdkv.rdkv_q4_read(cache, 1, stream=stream),
                 lambda: rdkv.rdkv_q4_attn(cache, q, stream=stream), lambda: rdkv.rdkv_q4_select(cache, q, 1, stream=stream),
                 lambda: rdkv.rdkv_q4_status(cache, stream=stream), lambda: rdkv.rdkv_q4_timeout_selftest(cache, q, stream=stream)):
        with pytest.raises(rdkv.RDKVError, match="cuda:1"):
            call()


def test_workspaces_elsewhere_are_refused():
    """A host tensor's address would be one that the GPU cannot reach."""
    cache = _cache()
    rdkv._q4_check_ws(cache, torch.zeros(8, dtype=torch.uint8))
    for bad in (torch.zeros(8, dtype=torch.uint8, device="meta"), torch.zeros(8, 8, dtype=torch.uint8)[:, ::2]):
        with pytest.raises(rdkv.RDKVError):
            rdkv._q4_check_ws(cache, bad)


def test_counts_past_thirty_two_bits_are_refused_instead_of_wrapped():
    """2^32 rows would have been taken for none, and written nothing."""
    cache = _cache(h_kv=2)
    rows = torch.zeros(6, 2, 64, dtype=torch.float16)
    start = torch.zeros(3, dtype=torch.int32)
    assert rdkv._q4_rows(cache, rows, rows, start, 2 ** 31 - 1)[3] == 2 ** 31 - 1
    for bad in (2 ** 31, 2 ** 32, 2 ** 32 + 1, -1):
        with pytest.raises(rdkv.RDKVError):
            rdkv._q4_rows(cache, rows, rows, start, bad)
