"""The 8-bit cache without a GPU: the oracle's pins, and what the calls and the binding refuse on the host."""
import ctypes
import types

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
def test_codes_are_those_of_torch():
    """e4m3 as torch casts to it, over every code, every middle of two and random values."""
    every = torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    real = ~np.isnan(every)
    assert real.sum() == 254 and np.array_equal(O.q8_values(np.arange(256)[real], 0), every[real])
    g = O.Q8_GRID
    x = np.concatenate([g, (g[1:] + g[:-1]) / 2, np.nextafter((g[1:] + g[:-1]) / 2, 1e9, dtype=np.float32),
                        np.random.default_rng(0).normal(size=10000) * 100])
    x = np.clip(np.concatenate([x, -x]), -448, 448).astype(np.float32)
    codes = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.q8_codes(x, 0), codes)
    assert np.array_equal(O.q8_codes(x * 2.0 ** -9, -9), codes)


def test_scales_and_values_at_the_ends():
    assert O.q8_exponent(np.zeros(3)) == O.q8_exponent(np.full(3, 448.0 * 2.0 ** -24)) == -24
    assert [O.q8_exponent(np.array([x])) for x in (448.0, np.nextafter(448.0, 999), 449.0, 224.0, 57344.0, 1e30)] == [0, 1, 1, -1, 7, 7]
    v, e = O.q8_append(np.zeros((0, 4)), 5, np.array([[np.inf, -1e9, np.nan, 1.0]]))
    assert e == 7 and v.tolist() == [[57344.0, -57344.0, 0.0, 1.0]]
    # a half step is 2^-4 of a value down to 2^-6 of the scale, 2^-10 of the scale below
    x = np.random.default_rng(1).normal(size=(40, 64))
    v, e = O.q8_append(np.zeros((0, 64)), 0, x)
    assert (np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (e - 10))).all()


def test_a_larger_scale_keeps_the_values_that_stay_normal():
    x = np.random.default_rng(2).normal(size=(8, 64))
    held, e = O.q8_append(np.zeros((0, 64)), 0, x)
    both, now = O.q8_append(held, e, np.full((1, 64), 300.0))
    assert now == 0 > e
    normal = np.abs(held) >= 2.0 ** -6
    assert np.array_equal(both[:8][normal], held[normal]) and np.abs(both[:8] - held).max() <= 2.0 ** -10
    again, last = O.q8_append(both, now, np.full((1, 64), 1e-3))
    assert last == now and np.array_equal(again[:9], both)


def test_page_layout_by_hand():
    D = 128
    k, v = np.zeros((64, D)), np.zeros((64, D))
    k[0, 0], k[0, 63], k[0, 64], k[1, 0], k[3, 127] = 1.0, 2.0, 3.0, 4.0, 5.0
    v[0, 0], v[1, 0], v[2, 1], v[8, 9], v[63, 127] = 1.0, 2.0, 3.0, 4.0, 5.0
    page = O.q8_page_bytes(k, 0, v, 0)
    one, two, three, four, five = (int(O.q8_codes(np.array([float(x)]), 0)[0]) for x in range(1, 6))
    where = {0: one, 63: two, 128: three, 64: four, 256 + 128 + 64 + 63: five}
    base = 64 * D
    where.update({base: one, base + 1: two, base + 16 + 2: three, base + 1024 + 64 + 2: four, 128 * D - 1: five})
    assert {int(i): int(page[i]) for i in np.flatnonzero(page)} == where


def test_eviction_by_hand():
    m = np.array([5.0, 1.0, 3.0, 3.0, 0.0, -0.0, np.nan, 2.0])
    assert O.q8_evict(m, 8, 0, 0) == list(range(8)) and O.q8_evict(m, 9, 1, 1) == list(range(8))
    assert O.q8_evict(m, 3, 0, 0) == [0, 2, 6] and O.q8_evict(m, 4, 0, 0) == [0, 2, 3, 6]
    assert O.q8_evict(m, 7, 0, 0) == [0, 1, 2, 3, 4, 6, 7]          # -0 equals 0: the lower stays
    assert O.q8_evict(m, 3, 2, 1) == [0, 1, 7] and O.q8_evict(m, 1, 0, 1) == [7]


# ---------------------------------------------------------------- refusals
def _struct(**kw):
    a = dict(batch=2, h_kv=2, head_dim=64, n_pages=8, page_stride=4, pages=4096, scales=8192, page_table=256, lens=512, status=1024)
    a.update(kw)
    return rdkv.Q8CacheStruct(*a.values())


BAD_CACHES = [(dict(batch=0), rdkv.RDKV_ERR_INVALID_ARG), (dict(h_kv=0), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(n_pages=0), rdkv.RDKV_ERR_INVALID_ARG), (dict(page_stride=0), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(head_dim=96), rdkv.RDKV_ERR_UNSUPPORTED), (dict(page_stride=1 << 25), rdkv.RDKV_ERR_UNSUPPORTED),
              (dict(n_pages=2 ** 31 - 1), rdkv.RDKV_ERR_UNSUPPORTED), (dict(batch=1 << 20, h_kv=2), rdkv.RDKV_ERR_UNSUPPORTED),
              (dict(pages=None), rdkv.RDKV_ERR_INVALID_ARG), (dict(scales=None), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(page_table=None), rdkv.RDKV_ERR_INVALID_ARG), (dict(lens=None), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(status=None), rdkv.RDKV_ERR_INVALID_ARG), (dict(pages=4104), rdkv.RDKV_ERR_INVALID_ARG),
              (dict(scales=8196), rdkv.RDKV_ERR_INVALID_ARG)]


def _call(L, which, c, **kw):
    """A call with arguments that are right but for kw (its pointers are never read: it must refuse)."""
    a = dict(dtype=0, k=4096, v=4096, total=1 << 20, stride=128, starts=None, first=None, rows=3, q=4096, q_stride=256, h_q=4, n_q=1,
             mass=4096, mass_stride=256, out=4096, out_dtype=0, keep=8, first_n=1, last=1, kept=4096, ws=4096, ws_bytes=1 << 40,
             withhold=1, cycles=1000)
    a.update(kw)
    r = ctypes.byref(c) if c is not None else None
    if which == "write":
        return L.rdkv_q8_write(r, a["dtype"], a["k"], a["v"], a["total"], a["stride"], a["starts"], a["rows"], None)
    if which == "read":
        return L.rdkv_q8_read(r, a["dtype"], a["k"], a["v"], a["total"], a["stride"], a["starts"], a["first"], a["rows"], None)
    if which == "attn":
        return L.rdkv_q8_attn(r, a["dtype"], a["q"], a["q_stride"], a["h_q"], a["n_q"], a["mass"], a["mass_stride"], a["out"],
                              a["out_dtype"], None, a["ws"], a["ws_bytes"], None)
    if which == "selftest":
        return L.rdkv_q8_timeout_selftest(r, a["dtype"], a["q"], a["q_stride"], a["h_q"], a["n_q"], a["out"], a["out_dtype"], None,
                                          a["ws"], a["ws_bytes"], a["withhold"], a["cycles"], None)
    return L.rdkv_q8_evict(r, a["mass"], a["mass_stride"], a["keep"], a["first_n"], a["last"], a["kept"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("which", ["write", "read", "attn", "selftest", "evict"])
def test_bad_caches_are_refused(L, which):
    before = L.rdkv_launch_count()
    for kw, code in BAD_CACHES:
        assert _call(L, which, _struct(**kw)) == code, (which, kw)
        assert L.rdkv_last_error_string()
    assert _call(L, which, None) == rdkv.RDKV_ERR_INVALID_ARG
    assert L.rdkv_launch_count() == before


INVALID, UNSUPPORTED, WORKSPACE = rdkv.RDKV_ERR_INVALID_ARG, rdkv.RDKV_ERR_UNSUPPORTED, rdkv.RDKV_ERR_WORKSPACE


@pytest.mark.parametrize("which,kw,code", [
    ("write", dict(dtype=3), UNSUPPORTED), ("write", dict(k=None), INVALID), ("write", dict(v=4098), INVALID),
    ("write", dict(stride=127), INVALID), ("write", dict(stride=132), INVALID), ("write", dict(rows=-1), INVALID),
    ("write", dict(total=2), INVALID), ("read", dict(total=2), INVALID), ("read", dict(total=-1, starts=4096), INVALID),
    ("read", dict(dtype=-1), UNSUPPORTED), ("read", dict(k=4104), INVALID),
    ("attn", dict(dtype=9), UNSUPPORTED), ("attn", dict(q=None), INVALID), ("attn", dict(q=4104), INVALID),
    ("attn", dict(q_stride=255), INVALID), ("attn", dict(q_stride=260), INVALID), ("attn", dict(h_q=3), INVALID),
    ("attn", dict(h_q=0), INVALID), ("attn", dict(h_q=18, q_stride=4096), UNSUPPORTED), ("attn", dict(n_q=0), INVALID),
    ("attn", dict(n_q=65), UNSUPPORTED), ("attn", dict(out=None), INVALID), ("attn", dict(out=4104), INVALID),
    ("attn", dict(out_dtype=2), UNSUPPORTED), ("attn", dict(ws=None), WORKSPACE), ("attn", dict(ws_bytes=16), WORKSPACE),
    ("attn", dict(ws=4100), WORKSPACE), ("attn", dict(mass=4100), INVALID), ("attn", dict(mass_stride=255), INVALID),
    ("attn", dict(mass_stride=254), INVALID), ("attn", dict(mass_stride=257), INVALID),
    ("selftest", dict(withhold=0), INVALID), ("selftest", dict(withhold=-1), INVALID), ("selftest", dict(cycles=0), INVALID),
    ("selftest", dict(cycles=-5), INVALID), ("selftest", dict(h_q=3), INVALID), ("selftest", dict(ws_bytes=16), WORKSPACE),
    ("evict", dict(keep=0), INVALID), ("evict", dict(keep=-3), INVALID), ("evict", dict(first_n=-1), INVALID),
    ("evict", dict(last=-1), INVALID), ("evict", dict(first_n=5, last=4), INVALID),
    ("evict", dict(keep=2 ** 31 - 1, first_n=2 ** 31 - 1, last=2 ** 31 - 1), INVALID), ("evict", dict(mass=None), INVALID),
    ("evict", dict(kept=None), INVALID), ("evict", dict(kept=4098), INVALID), ("evict", dict(mass=4100), INVALID),
    ("evict", dict(mass_stride=255), INVALID), ("evict", dict(mass_stride=254), INVALID), ("evict", dict(ws=None), WORKSPACE),
    ("evict", dict(ws=4100), WORKSPACE), ("evict", dict(ws_bytes=16), WORKSPACE),
])
def test_bad_arguments_are_refused(L, which, kw, code):
    before = L.rdkv_launch_count()
    assert _call(L, which, _struct(), **kw) == code
    assert L.rdkv_last_error_string() and L.rdkv_launch_count() == before


def test_no_rows(L):
    assert _call(L, "write", _struct(), rows=0, k=None, v=None) == rdkv.RDKV_OK
    assert _call(L, "read", _struct(), rows=0, k=None, v=None) == rdkv.RDKV_OK
    assert L.rdkv_q8_status(ctypes.byref(_struct(status=None)), None) == rdkv.RDKV_ERR_INVALID_ARG


def test_sizes(L):
    assert [L.rdkv_q8_page_bytes(d) for d in (64, 128, 96, 0, -64)] == [8192, 16384, 0, 0, 0]
    assert ctypes.sizeof(rdkv.Q8CacheStruct) == 64
    c = _struct()
    r = ctypes.byref
    fn = L.rdkv_q8_attn_workspace_bytes
    assert fn(r(c), 4, 1, 0) > 0 and fn(r(c), 4, 1, 0) % 16 == 0
    # with mass: the rows' statistics and a logit for every row and position
    assert fn(r(c), 4, 1, 1) - fn(r(c), 4, 1, 0) >= 4 * 2 * 4 * 256 + 8 * 8
    # six query tokens of three heads: two chunks of five and one tokens for 16-bit outputs (both as large as the larger: 15 rows),
    # three of two for fp32's
    odd = fn(r(c), 6, 6, 1) - fn(r(c), 6, 6, 0)
    assert odd >= 4 * 4 * 2 * 15 * 256
    big = _struct(batch=512, h_kv=8)
    assert fn(r(big), 8, 15, 0) > 0 and fn(r(big), 8, 16, 0) == 0
    assert fn(r(c), 5, 1, 0) == fn(r(c), 4, 65, 0) == fn(r(_struct(head_dim=32)), 4, 1, 0) == 0
    # past 32 bits
    long = _struct(batch=256, h_kv=8, page_stride=2048, n_pages=1 << 20)
    assert fn(r(long), 64, 1, 1) - fn(r(long), 64, 1, 0) >= 4 * 256 * 64 * 131072
    assert L.rdkv_q8_evict_workspace_bytes(r(c)) >= 4 * (4 * 5 + 4 * 4 + 2 * 16)
    assert L.rdkv_q8_evict_workspace_bytes(r(_struct(head_dim=32))) == 0


def _cache(batch=2, h_kv=3, head_dim=64, tokens=256):
    cache = rdkv.Q8Cache.__new__(rdkv.Q8Cache)       # the checks alone, on CPU tensors
    cache.batch, cache.h_kv, cache.head_dim, cache.device, cache._seen, cache.max_tokens = (batch, h_kv, head_dim, torch.device("cpu"),
                                                                                          {}, tokens)
    return cache


def test_the_binding_refuses_wrong_tensors(L):
    for args in ((1, 1, 96, 64), (1, 1, 64, 64), (0, 1, 64, 64), (1, 1, 64, 0)):
        with pytest.raises(rdkv.RDKVError):
            rdkv.Q8Cache(*args, "cpu")
    cache = _cache()
    mass = torch.zeros(2, 3, 256)
    assert rdkv._q8_mass(cache, mass) == (mass.data_ptr(), 256)
    assert rdkv._q8_mass(cache, torch.zeros(2, 3, 300))[1] == 300
    for bad in (mass.double(), mass[..., :255], mass[:1], mass[:, :2], mass.view(6, 256), torch.zeros(2, 3, 512)[..., ::2],
                torch.zeros(2, 3, 256, device="meta"), mass.transpose(0, 1)):
        with pytest.raises(rdkv.RDKVError):
            rdkv._q8_mass(cache, bad)
    cache._index = 0
    cache.device = torch.device("cuda", 0)
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    q = torch.zeros(2, 1, 3, 64)
    for call in (lambda: rdkv.rdkv_q8_write(cache, q, q, stream=stream), lambda: rdkv.rdkv_q8_read(cache, 1, stream=stream),
                 lambda: rdkv.rdkv_q8_attn(cache, q, stream=stream), lambda: rdkv.rdkv_q8_evict(cache, mass, 3, stream=stream),
                 lambda: rdkv.rdkv_q8_status(cache, stream=stream), lambda: rdkv.rdkv_q8_timeout_selftest(cache, q, stream=stream)):
        with pytest.raises(rdkv.RDKVError, match="cuda:1"):
            call()


def test_counts_past_thirty_two_bits_are_refused_instead_of_wrapped(monkeypatch):
    cache = _cache()
    cache._index = 0
    monkeypatch.setattr(rdkv, "_current_device", lambda: 0)
    monkeypatch.setattr(rdkv, "_raw_stream", lambda device: 0)
    mass = torch.zeros(2, 3, 256)
    for keep, first, last in ((2 ** 31, 0, 0), (2 ** 32 + 1, 0, 0), (0, 0, 0), (-1, 0, 0), (4, 2 ** 32, 0), (4, 0, 2 ** 32), (4, -1, 0),
                              (4, 5, 0), (4, 0, 5)):
        with pytest.raises(rdkv.RDKVError, match="n_keep"):
            rdkv.rdkv_q8_evict(cache, mass, keep, n_first=first, n_last=last)


def test_the_tensors_behind_the_struct_change_in_place_only():
    cache = rdkv.Q8Cache.__new__(rdkv.Q8Cache)
    for name in ("pages", "scales", "page_table", "lens", "status"):
        t = torch.zeros(3, dtype=torch.int32)
        setattr(cache, name, t)
        with pytest.raises(rdkv.RDKVError):
            setattr(cache, name, t + 1)
        assert getattr(cache, name) is t
    cache.lens += 1
    assert cache.lens.tolist() == [1, 1, 1]


def _selftest(L, c, **kw):
    a = dict(mass=4096, mass_stride=256, keep=8, first_n=1, last=1, kept=4096, ws=4096, ws_bytes=1 << 40, withhold=1, cycles=1000)
    a.update(kw)
    return L.rdkv_q8_evict_timeout_selftest(ctypes.byref(c), a["mass"], a["mass_stride"], a["keep"], a["first_n"], a["last"], a["kept"],
                                            a["ws"], a["ws_bytes"], a["withhold"], a["cycles"], None)


def test_the_evictions_selftest_refuses_what_the_eviction_does(L):
    before = L.rdkv_launch_count()
    for kw, code in BAD_CACHES:
        assert _selftest(L, _struct(**kw)) == code, kw
    for kw, code in ((dict(withhold=0), INVALID), (dict(withhold=-1), INVALID), (dict(cycles=0), INVALID), (dict(cycles=-5), INVALID),
                     (dict(keep=0), INVALID), (dict(first_n=5, last=4), INVALID), (dict(mass=None), INVALID), (dict(kept=4098), INVALID),
                     (dict(mass_stride=254), INVALID), (dict(ws_bytes=16), WORKSPACE), (dict(ws=None), WORKSPACE)):
        assert _selftest(L, _struct(), **kw) == code, kw
    assert L.rdkv_launch_count() == before
    cache = _cache()
    cache._index = 0
    cache.device = torch.device("cuda", 0)
    with pytest.raises(rdkv.RDKVError, match="cuda:1"):
        rdkv.rdkv_q8_evict_timeout_selftest(cache, torch.zeros(2, 3, 256), 3, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))


# ---------------------------------------------------------------- order between blocks
def _source(name):
    import os
    return open(os.path.join(os.path.dirname(os.path.abspath(rdkv.__file__)), "csrc", name)).read()


def test_the_flags_of_the_pages_order_what_they_tell():
    """A page is overwritten after other blocks have read their rows out of it: the flag that says so is stored with
    release and polled with acquire at the GPU's scope, else the memory model orders neither side."""
    import re
    text = _source("q8_evict.cu")
    accesses = re.findall(r'asm volatile\("([^;]*);"[^;]*"l"\(flags [^;]*;', text)
    assert sorted(a.split(" ")[0] for a in accesses) == ["ld.acquire.gpu.global.s32", "st.release.gpu.global.s32"], accesses


def test_the_last_block_clears_the_counters_behind_the_others():
    """The block that counts itself last clears counters that the others have read and added to before they counted
    themselves: that order needs acquire and release on the count."""
    import re
    text = _source("q8_evict.cu")
    assert "atomicAdd(a.count + 2" not in text
    assert re.findall(r'asm volatile\("([^ ]*) [^;]*;"[^;]*"l"\(a\.count \+ 2\)', text) == ["atom.add.acq_rel.gpu.global.s32"]


def test_the_choice_ends_with_no_copy_under_way():
    """Every way out of the choice, whose weights arrive by cp.async, passes a wait behind the copies."""
    import re
    text = _source("q8_evict.cu")
    kernel = text[text.index("pick_kernel"):]
    kernel = kernel[:kernel.index("\n}\n")]
    first = kernel.index("cp.async.ca")
    ways_out = [m.start() for m in re.finditer(r"\breturn;", kernel) if m.start() > first]
    assert ways_out and all("cp.async.wait_all" in kernel[first:at] for at in ways_out)
