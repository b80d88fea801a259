"""The 4-bit cache without a GPU: the oracle's pins, and what the calls refuse on the host."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from mixed_bit_kv_gb300 import rdkv


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return rdkv.lib()


# ---------------------------------------------------------------- oracle pins
def test_quantiser_is_the_pack_quantiser_and_its_error_is_half_a_step():
    x = np.random.default_rng(0).normal(size=(50, 3, 64)).astype(np.float32)
    codes, scale, zero = O.q4_quantize(x)
    ref = O.quantize_groups(x.reshape(50, 3, 2, 32), 4)
    assert np.array_equal(codes.reshape(50, 3, 2, 32), ref[0]) and np.array_equal(scale, ref[1])
    assert codes.max() == 15 and np.array_equal(zero, ref[2])
    # half a step, and the fp16 roundings of zero (2^-11 |zero|) and of fifteen scales (2^-11 of the range)
    step = scale.astype(np.float64)[..., None]
    bound = step / 2 + 2.0 ** -11 * (np.abs(zero.astype(np.float64))[..., None] + 15 * step) * 1.01
    err = np.abs(O.q4_values(codes, scale, zero) - x).reshape(50, 3, 2, 32)
    assert (err <= bound).all()


def test_quantiser_of_flat_extreme_and_non_finite_groups():
    x = np.zeros((4, 32), np.float32)
    x[0] = 2.5                                    # flat: scale 0
    x[1, :4] = [np.inf, -np.inf, 1e30, -1e30]
    x[2, :2] = [np.nan, 3.0]
    x[3] = np.nan
    codes, scale, zero = O.q4_quantize(x)
    val = O.q4_values(codes, scale, zero)
    assert (val[0] == 2.5).all() and (codes[0] == 0).all()
    assert list(codes[1, :4]) == [15, 0, 15, 0] and zero[1, 0] == -65504 and np.isfinite(val[1]).all()
    assert codes[2, 0] == 0 and zero[2, 0] == 0 and codes[2, 1] == 15
    assert (val[3] == 0).all()


def test_page_layout_by_hand():
    D = 64
    k = np.zeros((64, D), np.float32)
    k[:, 0], k[:, 1], k[:, 32] = 15.0, 1.0, 30.0  # group 0: scale 1; group 1: scale 2
    v = np.zeros((64, D), np.float32)
    v[:, 5], v[1::2, 7], v[:, 6] = 15.0, 3.0, -0.0
    page = O.q4_page_bytes(k, v)
    w = page.view(np.uint32)
    assert w[0] == 15 | 1 << 16                   # token 0, q 0, group 0: channel 0 at bit 0, channel 1 at 16
    assert w[1] == 15                             # token 0, q 0, group 1
    h = page.view(np.float16)
    assert h[1024:1028].tolist() == [1, 1, 2, 2]  # K scales of pair 0: group 0's two tokens, group 1's
    assert (h[1152:1280] == 0).all()
    vw = page[2560:].view(np.uint32)
    # pair 0, g 1 (channels 4 .. 7), group 0: channel 5 at bit 4, channel 7 at 12 and only in the odd token
    assert vw[2] == (15 << 4) | ((15 << 4 | 3 << 12) << 16)
    assert page.size == 5120


def test_bounds_and_selection_by_hand():
    k = np.arange(12, dtype=np.float64).reshape(3, 4)
    b = O.q4_bounds(k)
    assert b[0].tolist() == [0, 1, 2, 3] and b[1].tolist() == [8, 9, 10, 11]
    q = np.array([[1.0, -1, 0, 0], [0, 0, 2, 0]])
    assert O.q4_scores(q, b[None]).tolist() == [20.0]
    # no logit of a page's keys is larger than its score
    rng = np.random.default_rng(1)
    kk, qq = rng.normal(size=(64, 32)), rng.normal(size=(5, 32))
    kk = kk.astype(np.float16).astype(np.float64)
    assert (qq @ kk.T).max() <= O.q4_scores(qq, O.q4_bounds(kk)[None])[0] + 1e-12
    s = [9.0, 1.0, 5.0, 5.0, 5.0, 0.0, 2.0]
    assert O.q4_select(s, 4, 1, 1) == [0, 2, 3, 6] and O.q4_select(s, 7, 1, 1) == list(range(7))
    assert O.q4_select(s, 2, 1, 1) == [0, 6] and O.q4_select(s, 3, 0, 0) == [0, 2, 3]


# ---------------------------------------------------------------- refusals, before any launch
def _struct(**kw):
    f = dict(batch=2, h_kv=2, head_dim=64, n_pages=8, page_stride=4, pages=4096, bounds=8192, page_table=256, lens=512,
             status=1024)
    f.update(kw)
    return rdkv.Q4CacheStruct(*[f[n] for n, _ in rdkv.Q4CacheStruct._fields_])


BAD_CACHES = [(dict(head_dim=96), rdkv.RDKV_ERR_UNSUPPORTED), (dict(batch=0), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(h_kv=-1), rdkv.RDKV_ERR_INVALID_ARG), (dict(n_pages=0), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(page_stride=0), rdkv.RDKV_ERR_INVALID_ARG), (dict(page_stride=1 << 26), rdkv.RDKV_ERR_UNSUPPORTED),
              (dict(pages=None), rdkv.RDKV_ERR_INVALID_ARG), (dict(pages=4100), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(bounds=8200), rdkv.RDKV_ERR_INVALID_ARG), (dict(lens=None), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(page_table=None), rdkv.RDKV_ERR_INVALID_ARG), (dict(status=None), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(batch=1 << 15, h_kv=64), rdkv.RDKV_ERR_UNSUPPORTED)]


def _call(L, which, c, **kw):
    a = dict(dtype=0, k=4096, v=4096, stride=128, rows=3, total=1 << 40, starts=None, q=4096, q_stride=256, h_q=4, n_q=1, sel=None, n_sel=0, out=4096,
             out_dtype=0, keep=4, first=1, last=1, ws=4096, ws_bytes=1 << 40)
    a.update(kw)
    r = ctypes.byref(c) if c is not None else None
    if which == "write":
        return L.rdkv_q4_write(r, a["dtype"], a["k"], a["v"], a["total"], a["stride"], a["starts"], a["rows"], None)
    if which == "read":
        return L.rdkv_q4_read(r, a["dtype"], a["k"], a["v"], a["total"], a["stride"], a["starts"], None, a["rows"], None)
    if which == "attn":
        return L.rdkv_q4_attn(r, a["dtype"], a["q"], a["q_stride"], a["h_q"], a["n_q"], a["sel"], a["n_sel"], a["out"],
                              a["out_dtype"], None, a["ws"], a["ws_bytes"], None)
    return L.rdkv_q4_select(r, a["dtype"], a["q"], a["q_stride"], a["h_q"], a["n_q"], a["keep"], a["first"], a["last"],
                            a["out"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("which", ["write", "read", "attn", "select"])
def test_bad_caches_are_refused(L, which):
    before = L.rdkv_launch_count()
    for kw, code in BAD_CACHES:
        assert _call(L, which, _struct(**kw)) == code, (which, kw)
        assert L.rdkv_last_error_string()
    assert _call(L, which, None) == rdkv.RDKV_ERR_INVALID_ARG
    assert L.rdkv_launch_count() == before


@pytest.mark.parametrize("which,kw,code", [
    ("write", dict(dtype=3), rdkv.RDKV_ERR_UNSUPPORTED), ("write", dict(k=None), rdkv.RDKV_ERR_INVALID_ARG),
    ("write", dict(v=4098), rdkv.RDKV_ERR_INVALID_ARG), ("write", dict(stride=127), rdkv.RDKV_ERR_INVALID_ARG),
    ("write", dict(stride=132), rdkv.RDKV_ERR_INVALID_ARG), ("write", dict(rows=-1), rdkv.RDKV_ERR_INVALID_ARG),
    ("write", dict(total=2), rdkv.RDKV_ERR_INVALID_ARG), ("read", dict(total=2), rdkv.RDKV_ERR_INVALID_ARG),
    ("read", dict(total=-1, starts=4096), rdkv.RDKV_ERR_INVALID_ARG),
    ("read", dict(dtype=-1), rdkv.RDKV_ERR_UNSUPPORTED), ("read", dict(k=4104), rdkv.RDKV_ERR_INVALID_ARG),
    ("attn", dict(dtype=9), rdkv.RDKV_ERR_UNSUPPORTED), ("attn", dict(q=None), rdkv.RDKV_ERR_INVALID_ARG),
    ("attn", dict(q=4104), rdkv.RDKV_ERR_INVALID_ARG), ("attn", dict(q_stride=255), rdkv.RDKV_ERR_INVALID_ARG),
    ("attn", dict(q_stride=260), rdkv.RDKV_ERR_INVALID_ARG), ("attn", dict(h_q=3), rdkv.RDKV_ERR_INVALID_ARG),
    ("attn", dict(h_q=0), rdkv.RDKV_ERR_INVALID_ARG), ("attn", dict(h_q=18, q_stride=4096), rdkv.RDKV_ERR_UNSUPPORTED),
    ("attn", dict(n_q=0), rdkv.RDKV_ERR_INVALID_ARG), ("attn", dict(n_q=65), rdkv.RDKV_ERR_UNSUPPORTED),
    ("attn", dict(out=None), rdkv.RDKV_ERR_INVALID_ARG), ("attn", dict(out=4104), rdkv.RDKV_ERR_INVALID_ARG),
    ("attn", dict(out_dtype=2), rdkv.RDKV_ERR_UNSUPPORTED), ("attn", dict(sel=4096, n_sel=0), rdkv.RDKV_ERR_INVALID_ARG),
    ("attn", dict(ws=None), rdkv.RDKV_ERR_WORKSPACE), ("attn", dict(ws_bytes=16), rdkv.RDKV_ERR_WORKSPACE),
    ("attn", dict(ws=4100), rdkv.RDKV_ERR_WORKSPACE),
    ("select", dict(keep=0), rdkv.RDKV_ERR_INVALID_ARG), ("select", dict(first=3, last=2), rdkv.RDKV_ERR_INVALID_ARG),
    ("select", dict(first=-1), rdkv.RDKV_ERR_INVALID_ARG), ("select", dict(out=None), rdkv.RDKV_ERR_INVALID_ARG),
    ("select", dict(first=2 ** 31 - 1, last=2 ** 31 - 1), rdkv.RDKV_ERR_INVALID_ARG),
    ("select", dict(ws_bytes=16), rdkv.RDKV_ERR_WORKSPACE), ("select", dict(n_q=100), rdkv.RDKV_ERR_UNSUPPORTED),
])
def test_bad_arguments_are_refused(L, which, kw, code):
    before = L.rdkv_launch_count()
    assert _call(L, which, _struct(), **kw) == code
    assert L.rdkv_last_error_string() and L.rdkv_launch_count() == before


def test_no_rows_and_no_bounds(L):
    assert _call(L, "write", _struct(), rows=0, k=None, v=None) == rdkv.RDKV_OK
    assert _call(L, "read", _struct(), rows=0, k=None, v=None) == rdkv.RDKV_OK
    assert _call(L, "select", _struct(bounds=None)) == rdkv.RDKV_ERR_INVALID_ARG
    assert L.rdkv_q4_status(ctypes.byref(_struct(status=None)), None) == rdkv.RDKV_ERR_INVALID_ARG


def test_sizes(L):
    assert [L.rdkv_q4_page_bytes(d) for d in (64, 128, 96, 0, -64)] == [5120, 10240, 0, 0, 0]
    assert ctypes.sizeof(rdkv.Q4CacheStruct) == 64
    c = _struct()
    for fn in (L.rdkv_q4_attn_workspace_bytes, L.rdkv_q4_select_workspace_bytes):
        assert fn(ctypes.byref(c), 4, 1) > 0
        assert fn(ctypes.byref(c), 4, 1) % 16 == 0
        big = _struct(batch=512, h_kv=8)
        assert fn(ctypes.byref(big), 8, 15) > 0 and fn(ctypes.byref(big), 8, 16) == 0
        assert fn(ctypes.byref(c), 5, 1) == fn(ctypes.byref(c), 4, 65) == fn(ctypes.byref(_struct(head_dim=32)), 4, 1) == 0
    # the other calls of the library still take no bf16
    s = rdkv.make_shape(1, 64, 4, 2, 64, 0, "f16")
    s.dtype = rdkv.RDKV_BF16
    assert L.rdkv_score_workspace_bytes(ctypes.byref(s)) == 0


def test_the_binding_refuses_wrong_tensors(L):
    with pytest.raises(rdkv.RDKVError):
        rdkv.Q4Cache(1, 1, 96, 64, "cpu")
    with pytest.raises(rdkv.RDKVError):
        rdkv.Q4Cache(1, 1, 64, 64, "cpu")            # not on a GPU
    with pytest.raises(rdkv.RDKVError):
        rdkv.Q4Cache(0, 1, 64, 64, "cpu")
    cache = rdkv.Q4Cache.__new__(rdkv.Q4Cache)       # the checks of the rows alone, on CPU tensors
    cache.batch, cache.h_kv, cache.head_dim, cache.device, cache._seen = 2, 2, 64, torch.device("cpu"), {}
    rows = torch.zeros(2, 3, 2, 64, dtype=torch.float16)
    assert rdkv._q4_rows(cache, rows, rows, None, None) == (0, 6, 128, 3)
    wide = torch.zeros(2, 3, 6, 64, dtype=torch.float16)
    assert rdkv._q4_rows(cache, wide[:, :, 2:4], wide[:, :, 4:], None, None) == (0, 6, 384, 3)
    for k, v in ((rows, rows.float()), (rows.double(), rows.double()), (rows[..., ::2], rows[..., ::2]),
                 (rows.transpose(0, 1)[:2], rows.transpose(0, 1)[:2]), (wide[:, :2, :2], wide[:, :2, :2]),
                 (rows[:, :, :1], rows[:, :, :1]), (wide[:, :, :2], rows), (wide[:, :, ::3], wide[:, :, ::3])):
        with pytest.raises(rdkv.RDKVError):
            rdkv._q4_rows(cache, k, v, None, None)
    flat = rows.view(6, 2, 64)
    assert rdkv._q4_rows(cache, flat, flat, None, None) == (0, 6, 128, 3)
    assert rdkv._q4_rows(cache, flat[:5], flat[:5], flat, 4) == (0, 5, 128, 4)
    with pytest.raises(rdkv.RDKVError):
        rdkv._q4_rows(cache, flat[:5], flat[:5], None, None)
    q = torch.zeros(2, 3, 4, 64)
    assert rdkv._q4_queries(cache, q) == (1, 4, 3, 256)
    assert rdkv._q4_queries(cache, torch.zeros(2, 3, 8, 64)[:, :, 4:]) == (1, 4, 3, 512)
    assert rdkv._q4_queries(cache, torch.zeros(2, 8, 64)[:, 4:]) == (1, 4, 1, 512)
    for bad in (q[:1], q[..., :32], q.transpose(1, 2), q.long(), torch.zeros(2, 5, 4, 64)[:, :3]):
        with pytest.raises(rdkv.RDKVError):
            rdkv._q4_queries(cache, bad)
