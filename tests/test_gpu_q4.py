"""GPU parity of the 4-bit cache (rdkv_q4_*) against the CPU oracle.

Written pages and bounds: every byte.  Rows read back: bit-exact (x^ rounded once).  Attention: against
float64 attention over the values the cache holds, within

  16-bit outputs  eps / 2 of the value (its rounding) + 3 2^-11 max|v| (the fp16 roundings of the
                  probabilities, each at most 2^-11 relative: once times scale and code, whose product is at
                  most the group's range <= 2 max|v|, once times the zero) + what the logits' error gives;
  fp32 outputs    what the logits' error gives + 2^-20 max|v|.

A logit's error is taken as 2^-17 of sum_c |q_c k_c| / sqrt(D) (some twenty fp32 sums of truncated
products, each 2^-22 of the sum of the magnitudes) + 2^-20 (the exponential), weights change by as much
relatively, and an output by twice that times max|v|; the log-sum-exp by that alone.  A sum of n fp32
terms is off by at most n 2^-24 of the sum of their magnitudes: that once more for the sum of the weights
(positive terms, so relatively) and for the sum of the weighted values (at most max|v| times the former).
Selections: equal, page for page."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
from mixed_bit_kv_gb300 import rdkv, synth

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if DEV is None:
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _rows(n, h, D, dt, seed, mag=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, D, generator=g) * mag
    x[:, :, 3] *= 10.0
    return x.to(dt)


def _cache(lens, h, D, stride=None, seed=0, extra=3, bounds=None, grow=0):
    """A cache of shuffled pages whose every byte, and bound, is NaN-like garbage until it is written."""
    B = len(lens)
    stride = stride or max(1, max(-(-n // 64) for n in lens))
    n = B * stride + extra
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed))
    table = order[:B * stride].to(torch.int32).view(B, stride)
    for b, t in enumerate(lens):                  # entries that no token needs (yet) are not read
        table[b, -(-t // 64) + grow:] = 1 << 30
    c = rdkv.Q4Cache(B, h, D, stride * 64, DEV, pages=torch.full((n, h, 80 * D), 0xFF, dtype=torch.uint8, device=DEV),
                     bounds=torch.full((n, h, 2, D), float("nan"), dtype=torch.float16, device=DEV) if bounds is None else bounds,
                     page_table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    return c


def _filled(lens, h, D, dt, seed=0, mag=1.0, **kw):
    """A cache written in one call, and the float64 values it holds, per sequence [n, h, D]."""
    c = _cache(lens, h, D, seed=seed, **kw)
    k, v = _rows(sum(lens), h, D, dt, seed + 1, mag), _rows(sum(lens), h, D, dt, seed + 2, mag)
    start = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    rdkv.rdkv_q4_write(c, k.to(DEV), v.to(DEV), row_start=start.to(DEV), max_rows=max(max(lens), 1))
    kh, vh = (O.q4_values(*O.q4_quantize(x.float().numpy())) for x in (k, v))
    cut = np.cumsum(lens)[:-1]
    return c, np.split(kh, cut), np.split(vh, cut)


def _check_attention(q, kh, vh, out, lse, pages=None):
    """q [B, T, Hq, D]; kh, vh per sequence [n, h, D]; pages [B, T, h, n_sel] or None."""
    q64, out64, lse64 = q.double().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    eps = torch.finfo(out.dtype).eps
    B, T, Hq, D = q64.shape
    for b in range(B):
        n, h = kh[b].shape[:2]
        G = Hq // h
        for t in range(T):
            m = max(0, n - T + t + 1)
            for j in range(Hq):
                rows = np.arange(m)
                if pages is not None:
                    rows = rows[np.isin(rows // 64, pages[b, t, j // G])]
                K, V = kh[b][rows, j // G], vh[b][rows, j // G]
                ref, ref_lse = O.attention_lse(q64[b, t, j], K, V)
                if len(rows) == 0:
                    assert (out64[b, t, j] == 0).all() and lse64[b, t, j] == -np.inf
                    continue
                logit = 2.0 ** -17 * (np.abs(K) @ np.abs(q64[b, t, j])).max() / math.sqrt(D) + 2.0 ** -20
                big = np.abs(V).max()
                tol = 2 * logit * big + (2.0 ** -20 + 2 * len(rows) * 2.0 ** -24) * big
                if out.dtype != torch.float32:
                    tol = tol + 3 * 2.0 ** -11 * big + eps / 2 * np.abs(ref)
                assert (np.abs(out64[b, t, j] - ref) <= tol).all(), (b, t, j, np.abs(out64[b, t, j] - ref).max(), np.max(tol))
                assert abs(lse64[b, t, j] - ref_lse) <= logit + 2.0 ** -22 * abs(ref_lse) + len(rows) * 2.0 ** -24, (b, t, j)


# ---------------------------------------------------------------- write and read
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,h", [(64, 1), (64, 3), (128, 2)])
def test_written_pages_bounds_and_rows_read_back(D, h, dtype):
    dt, lens, new = TYPES[dtype], [70, 0, 1, 200, 64, 129], [33, 0, 1, 200, 64, 1]
    c = _cache([a - b for a, b in zip(lens, new)], h, D, stride=4, grow=4)
    old = [a - b for a, b in zip(lens, new)]
    k = [_rows(n, h, D, dt, 10 + i) for i, n in enumerate(lens)]
    v = [_rows(n, h, D, dt, 30 + i) for i, n in enumerate(lens)]

    def write(lo, hi):
        n = [b - a for a, b in zip(lo, hi)]
        start = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
        c.lens.copy_(torch.tensor(hi, dtype=torch.int32))
        kk, vv = (torch.cat([x[i][lo[i]:hi[i]] for i in range(6)] + [x[0][:2]]).to(DEV) for x in (k, v))  # two rows of nobody
        rdkv.rdkv_q4_write(c, kk, vv, row_start=start, max_rows=max(n))

    write([0] * 6, old)
    write(old, lens)
    assert rdkv.rdkv_q4_status(c) == 0
    pages, bounds = c.pages.cpu().numpy(), c.bounds.cpu()
    used = set()
    for i, n in enumerate(lens):
        for p in range(-(-n // 64)):
            phys = int(c.page_table[i, p])
            used.add(phys)
            part = slice(64 * p, min(n, 64 * p + 64))
            for j in range(h):
                exp = O.q4_page_bytes(k[i][part, j].float().numpy(), v[i][part, j].float().numpy(),
                                      np.full(80 * D, 0xFF, np.uint8), range(min(64, n - 64 * p)))
                assert np.array_equal(pages[phys, j], exp), (i, p, j)
                b = O.q4_bounds(O.q4_values(*O.q4_quantize(k[i][part, j].float().numpy())))
                assert np.array_equal(bounds[phys, j].numpy(), b), (i, p, j)
    rest = [p for p in range(pages.shape[0]) if p not in used]
    assert (pages[rest] == 0xFF).all() and bounds[rest].isnan().all()
    # every row back, from the middle of pages on, into rows that are otherwise left alone
    first = [5, 0, 0, 63, 64, 100]
    n = [lens[0] - 5, 2, 1, 130, 3, 60]  # sequence 1 is empty, 4 has no row at 64, 5 has 29 from there
    start = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
    out = tuple(torch.full((sum(n) + 2, h, D), 7.0, dtype=dt, device=DEV) for _ in range(2))
    rdkv.rdkv_q4_read(c, max(n), row_start=start, first=torch.tensor(first, dtype=torch.int32, device=DEV), out=out)
    assert rdkv.rdkv_q4_status(c) == 0
    for x, got in ((k, out[0]), (v, out[1])):
        got, r = got.cpu(), 0
        for i in range(6):
            val = torch.from_numpy(O.q4_values(*O.q4_quantize(x[i].float().numpy()))).to(dt)[first[i]:first[i] + n[i]]
            assert torch.equal(got[r:r + len(val)], val), i
            assert (got[r + len(val):r + n[i]] == 7.0).all()
            r += n[i]
        assert (got[r:] == 7.0).all()


def test_uniform_rows_of_a_strided_projection_and_empty_slots():
    lens, h, D = [5, 0, 64, 66], 2, 128
    c = _cache(lens, h, D, stride=2)
    qkv = torch.randn(4, 3, 5 * h, D, dtype=torch.float32, generator=torch.Generator().manual_seed(0)).half().to(DEV)
    rdkv.rdkv_q4_write(c, qkv[:, :, h:2 * h], qkv[:, :, 4 * h:])
    out = torch.zeros(4, 3, 3 * h, D, dtype=torch.float16, device=DEV)
    first = torch.tensor([2, 0, 61, 63], dtype=torch.int32, device=DEV)
    rdkv.rdkv_q4_read(c, 3, first=first, out=(out[:, :, :h], out[:, :, h:2 * h]))
    assert rdkv.rdkv_q4_status(c) == 0
    for lo, hi, src in ((0, h, qkv[:, :, h:2 * h]), (h, 2 * h, qkv[:, :, 4 * h:])):
        val = torch.from_numpy(O.q4_values(*O.q4_quantize(src.float().cpu().numpy()))).half()
        val[1] = 0
        assert torch.equal(out[:, :, lo:hi].cpu(), val)
    assert (out[:, :, 2 * h:] == 0).all()
    # a second write of the same rows changes nothing; no bounds, no bounds written
    before = c.pages.clone()
    rdkv.rdkv_q4_write(c, qkv[:, :, h:2 * h], qkv[:, :, 4 * h:])
    assert torch.equal(c.pages, before)
    plain = rdkv.Q4Cache(4, h, D, 128, DEV, bounds=False, lens=c.lens)
    rdkv.rdkv_q4_write(plain, qkv[:, :, h:2 * h], qkv[:, :, 4 * h:])
    for i, p in ((0, 0), (2, 0), (3, 1)):
        got = plain.pages[plain.page_table[i, p].long()]
        x = c.pages[c.page_table[i, p].long()]
        a = torch.stack(rdkv.rdkv_q4_read(plain, 3, first=first))
        b = torch.stack(rdkv.rdkv_q4_read(c, 3, first=first))
        assert torch.equal(a[:, i], b[:, i]) and got.shape == x.shape


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_flat_huge_tiny_and_non_finite_rows(dtype):
    dt, h, D = TYPES[dtype], 1, 64
    x = torch.randn(12, h, D, generator=torch.Generator().manual_seed(3)).to(dt)
    x[0] = 2.5
    x[1, 0, :4] = torch.tensor([float("inf"), float("-inf"), 60000.0, -60000.0]).to(dt)
    x[2, 0, 0], x[2, 0, 40:44] = float("nan"), float("nan")
    x[3] = float("nan")
    x[4] = x[4] * 1e-7
    x[5] = x[5] * 3000
    x[6] = float("inf")
    x[7] = 0.0
    x[8] = -0.0
    x[9] = x[9] * 2.0 ** -14
    c = _cache([12], h, D)
    rdkv.rdkv_q4_write(c, x[None].to(DEV), x[None].to(DEV))
    exp = O.q4_page_bytes(x[:, 0].float().numpy(), x[:, 0].float().numpy(), np.full(80 * D, 0xFF, np.uint8), range(12))
    assert np.array_equal(c.pages[c.page_table[0, 0].long(), 0].cpu().numpy(), exp)
    k, v = rdkv.rdkv_q4_read(c, 12, dtype=dt)
    val = torch.from_numpy(O.q4_values(*O.q4_quantize(x.float().numpy())))
    val = (val.clamp(-65504, 65504) if dtype == "f16" else val).to(dt)
    assert torch.equal(k[0].cpu(), val) and torch.equal(v[0].cpu(), val) and k.isfinite().all()


def test_positions_past_two_to_the_thirty_first_elements():
    """Pages far into the pool and rows far into the tensors: offsets beyond 32 bits."""
    h, D, n = 8, 128, 2_200_000                   # 2.2 M rows of 1024 values: 2.25e9 elements, 2.8 GB of pages
    stride = -(-n // 64)
    c = rdkv.Q4Cache(1, h, D, stride * 64, DEV, lens=torch.tensor([n], dtype=torch.int32, device=DEV))
    k = torch.zeros(n, h, D, dtype=torch.float16, device=DEV)
    tail = _rows(40, h, D, torch.float16, 5).to(DEV)
    k[-40:] = tail
    rdkv.rdkv_q4_write(c, k[None], k[None])
    assert rdkv.rdkv_q4_status(c) == 0
    first = torch.tensor([n - 40], dtype=torch.int32, device=DEV)
    a, b = rdkv.rdkv_q4_read(c, 40, first=first)
    val = torch.from_numpy(O.q4_values(*O.q4_quantize(tail.float().cpu().numpy()))).half()
    assert torch.equal(a[0].cpu(), val) and torch.equal(b[0].cpu(), val)
    a, b = rdkv.rdkv_q4_read(c, n, out=(k[None], k.clone()[None]))
    assert torch.equal(a[0, -40:].cpu(), val) and (a[0, :-40] == 0).all()
    # the attention over it: the other keys are zero, so that each weighs exp(0)
    q = _rows(1, 2 * h, D, torch.float16, 6)
    out, lse = rdkv.rdkv_q4_attn(c, q.to(DEV))
    assert rdkv.rdkv_q4_status(c) == 0
    kt = O.q4_values(*O.q4_quantize(tail.float().cpu().numpy()))
    for j in range(2 * h):
        s = kt[:, j // 2] @ q[0, j].double().numpy() / math.sqrt(D)
        total = np.exp(s).sum() + n - 40
        ref = (np.exp(s) @ kt[:, j // 2]) / total
        assert abs(lse[0, j].item() - math.log(total)) <= 2.0 ** -17 * 200 + 2.0 ** -20
        assert np.abs(out[0, j].double().cpu().numpy() - ref).max() <= 2.0 ** -11 * np.abs(ref).max() * 4 + 2.0 ** -24


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("D,h,G,T,lens", [
    (64, 1, 4, 1, [513]), (128, 2, 1, 1, [1, 64, 0, 65]), (128, 1, 8, 1, [1500, 63]), (64, 3, 5, 2, [2, 130, 1, 0, 128]),
    (128, 2, 3, 5, [3, 5, 64, 700, 66]), (128, 1, 8, 4, [300, 2, 64]), (64, 2, 2, 9, [200, 8, 0]), (128, 1, 7, 64, [65, 40, 300]),
])
def test_attention(D, h, G, T, lens, dtype, out):
    dt = TYPES[dtype]
    c, kh, vh = _filled(lens, h, D, dt)
    q = _rows(len(lens) * T, h * G, D, dt, 9).view(len(lens), T, h * G, D)
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), out_dtype=TYPES[out])
    assert rdkv.rdkv_q4_status(c) == 0
    _check_attention(q, kh, vh, o, lse)


@pytest.mark.parametrize("mag_q,mag", [(30.0, 1.0), (1e-3, 1e-3), (1.0, 300.0), (1e-6, 1e-4), (300.0, 2e-3), (0.0, 1.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_attention_of_large_and_small_values(dtype, mag_q, mag):
    """Sharp rows (one key takes all), flat ones, and values far from one."""
    dt, lens = TYPES[dtype], [900, 65]
    c, kh, vh = _filled(lens, 1, 128, dt, mag=mag)
    q = _rows(2, 4, 128, dt, 9, mag_q).view(2, 1, 4, 128)
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV))
    assert rdkv.rdkv_q4_status(c) == 0
    _check_attention(q, kh, vh, o, lse)


def test_attention_with_values_that_grow_along_the_cache():
    """Keys and values whose scale rises and falls by 2^20 from page to page: every rescaling on the way."""
    n, D = 64 * 40, 64
    c = _cache([n], 1, D)
    k, v = _rows(n, 1, D, torch.float32, 1), _rows(n, 1, D, torch.float32, 2)
    step = torch.arange(n).div(64, rounding_mode="floor").float()
    v = v * 2.0 ** (10 * torch.sin(step / 3))[:, None, None]
    k = k * (1 + step / 10)[:, None, None]
    rdkv.rdkv_q4_write(c, k[None].to(DEV), v[None].to(DEV))
    kh, vh = (O.q4_values(*O.q4_quantize(x.numpy())) for x in (k, v))
    for dt in (torch.float16, torch.float32):
        q = _rows(1, 8, D, dt, 9).view(1, 1, 8, D)
        o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV))
        _check_attention(q, [kh], [vh], o, lse)


def test_attention_of_many_short_and_few_long_sequences():
    lens = [1 + 37 * i % 190 for i in range(300)] + [9000]
    c, kh, vh = _filled(lens, 2, 64, torch.float16)
    q = _rows(len(lens), 6, 64, torch.float16, 9).view(len(lens), 1, 6, 64)
    for _ in range(3):  # the workspace is as it was
        o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV))
    assert rdkv.rdkv_q4_status(c) == 0
    _check_attention(q, kh, vh, o, lse)
    a, _ = rdkv.rdkv_q4_attn(c, q.to(DEV))
    assert torch.equal(a, o)                      # no order of arrival in the results


def test_attention_of_strided_queries_without_n_q_and_into_given_outputs():
    lens = [100, 3, 64]
    c, kh, vh = _filled(lens, 2, 128, torch.bfloat16)
    qkv = _rows(3, 10, 128, torch.bfloat16, 4).to(DEV)
    q = qkv[:, 2:8]
    out, lse = torch.empty(3, 6, 128, device=DEV), torch.empty(3, 6, device=DEV)
    a = rdkv.rdkv_q4_attn(c, q, out=out, lse=lse)
    assert a[0] is out and a[1] is lse
    _check_attention(q[:, None].cpu(), kh, vh, out[:, None], lse[:, None])
    with pytest.raises(rdkv.RDKVError):
        rdkv.rdkv_q4_attn(c, q, out=out.half())
    with pytest.raises(rdkv.RDKVError):
        rdkv.rdkv_q4_attn(c, q.float(), out_dtype=torch.float16)
    with pytest.raises(rdkv.RDKVError):
        rdkv.rdkv_q4_attn(c, q, sel=torch.zeros(3, 2, 4, device=DEV))
    with pytest.raises(rdkv.RDKVError):
        rdkv.rdkv_q4_attn(c, q.cpu())


# ---------------------------------------------------------------- selection
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,h,G,T,lens,keep,first,last", [
    (64, 1, 4, 1, [64 * 30 + 5], 7, 1, 2), (128, 2, 3, 1, [64 * 50, 64 * 4 + 1, 0, 5000], 9, 1, 1),
    (128, 1, 8, 3, [64 * 20 + 1, 64 * 9], 6, 0, 0), (64, 2, 1, 1, [64 * 700], 33, 2, 3), (128, 1, 2, 1, [64 * 12], 12, 1, 1),
    (64, 1, 5, 1, [64 * 13 - 1], 3, 2, 1), (64, 1, 1, 1, [64 * 300], 1, 0, 0),
])
def test_selection_and_the_attention_over_it(D, h, G, T, lens, keep, first, last, dtype):
    dt = TYPES[dtype]
    c, kh, vh = _filled(lens, h, D, dt)
    q = _rows(len(lens) * T, h * G, D, dt, 9).view(len(lens), T, h * G, D)
    sel = rdkv.rdkv_q4_select(c, q.to(DEV), keep, n_first=first, n_last=last)
    assert rdkv.rdkv_q4_status(c) == 0
    q64 = q.double().numpy()
    for b, n in enumerate(lens):
        bounds = [O.q4_bounds(kh[b][64 * p:64 * p + 64].reshape(-1, h * D)).reshape(2, h, D) for p in range(-(-n // 64))]
        for t in range(T):
            P = max(0, -(-(n - T + t + 1) // 64))
            for j in range(h):
                s = O.q4_scores(q64[b, t, j * G:(j + 1) * G], np.stack([e[:, j] for e in bounds])[:P]) if P else []
                exp = O.q4_select(s, keep, first, last)
                assert sel[b, t, j].tolist() == exp + [-1] * (keep - len(exp)), (b, t, j)
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), sel=sel)
    _check_attention(q, kh, vh, o, lse, sel.cpu().numpy())
    for _ in range(2):
        assert torch.equal(rdkv.rdkv_q4_select(c, q.to(DEV), keep, n_first=first, n_last=last), sel)


def test_equal_scores_take_the_lower_page():
    n, D = 64 * 200, 64
    c = _cache([n], 1, D)
    one = _rows(64, 1, D, torch.float16, 1)
    k = one.repeat(200, 1, 1)                     # every page the same
    k[64 * 150:64 * 151] *= 2
    rdkv.rdkv_q4_write(c, k[None].to(DEV), k[None].to(DEV))
    q = _rows(1, 4, D, torch.float16, 2).to(DEV)
    assert rdkv.rdkv_q4_select(c, q, 20, 0, 1)[0, 0].tolist() == list(range(18)) + [150, 199]
    assert rdkv.rdkv_q4_select(c, torch.zeros_like(q), 20, 1, 1)[0, 0].tolist() == list(range(19)) + [199]


def test_near_scores_are_told_apart():
    """Pages whose scores differ by a few units of the 33rd bit: next to the border the order is that of
    exact sums."""
    P, D = 600, 64
    c = _cache([64 * P], 1, D)
    g = torch.Generator().manual_seed(4)
    c.bounds[:] = 0
    base = torch.randn(D, generator=g).half()
    e = base.repeat(P, 1)
    small = torch.randperm(P, generator=g)
    e[:, 5] = (small.float() * 2.0 ** -24).half()  # one channel tells the pages apart, by fp16's smallest steps
    c.bounds[c.page_table[0, :P].long(), 0, 0] = e.to(DEV)
    c.bounds[c.page_table[0, :P].long(), 0, 1] = e.to(DEV)
    q = torch.randn(1, 2, D, generator=g).half()
    s = O.q4_scores(q[0].double().numpy(), np.stack([e.numpy()] * 2, 1))
    exp = O.q4_select(s, 50, 1, 1)
    assert rdkv.rdkv_q4_select(c, q.to(DEV), 50)[0, 0].tolist() == exp


@pytest.mark.parametrize("P,keep,first,last", [(8192, 100, 1, 1), (8193, 64, 0, 2), (20011, 3000, 5, 5), (20011, 1, 0, 0)])
def test_selection_over_rows_longer_than_shared_memory(P, keep, first, last):
    D, h = 64, 2
    c = rdkv.Q4Cache(1, h, D, 64 * P, DEV, pages=torch.zeros(1, h, 80 * D, dtype=torch.uint8, device=DEV).expand(P, -1, -1).contiguous(),
                     lens=torch.tensor([64 * P - 7], dtype=torch.int32, device=DEV))
    g = torch.Generator().manual_seed(P)
    e = torch.randn(P, h, 2, D, generator=g).sort(2).values.half()
    c.bounds.copy_(e)
    q = torch.randn(1, 3 * h, D, generator=g).half()
    for _ in range(2):
        sel = rdkv.rdkv_q4_select(c, q.to(DEV), keep, n_first=first, n_last=last)
        for j in range(h):
            s = O.q4_scores(q[0, 3 * j:3 * j + 3].double().numpy(), e[:, j].numpy())
            assert sel[0, j].tolist() == O.q4_select(s, keep, first, last)
    # the same workspace serves other shapes in between
    small, kh, vh = _filled([64 * 9], 1, 64, torch.float16)
    small._ws = c._ws
    qs = _rows(1, 2, 64, torch.float16, 1)
    rdkv.rdkv_q4_select(small, qs.to(DEV), 3)
    assert torch.equal(rdkv.rdkv_q4_select(c, q.to(DEV), keep, n_first=first, n_last=last), sel)


def test_a_callers_own_pages():
    lens = [64 * 9 + 3, 70]
    c, kh, vh = _filled(lens, 2, 64, torch.float16)
    q = _rows(2, 4, 64, torch.float16, 9).view(2, 1, 4, 64)
    sel = torch.tensor([[[9, -1, 3, 50, -7], [-1, -1, -1, -1, -1]], [[1, 2, 3, 4, 5], [0, 1, -1, 64, 1 << 30]]], dtype=torch.int32)
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), sel=sel[:, None].to(DEV))
    assert rdkv.rdkv_q4_status(c) == 0
    _check_attention(q, kh, vh, o, lse, sel[:, None].numpy())


# ---------------------------------------------------------------- bad device data, streams, graphs
@pytest.mark.parametrize("lens,h,G,T", [([64 * 47 - 3] * 25, 4, 5, 1), ([64 * 300], 1, 8, 3), ([70, 64 * 40, 0], 2, 3, 2), ([1], 1, 1, 64)])
@pytest.mark.parametrize("D", [64, 128])
def test_nothing_is_written_outside_workspaces_and_outputs(D, lens, h, G, T):
    """Guard words behind every workspace and output stay as they were; the counters are zero again."""
    c, _, _ = _filled(lens, h, D, torch.bfloat16)
    B = len(lens)
    q = _rows(B * T, h * G, D, torch.bfloat16, 9).view(B, T, h * G, D).to(DEV)

    def guarded(shape, dtype):
        n = math.prod(shape)
        big = torch.full((n + 4096,), 77, dtype=dtype, device=DEV)
        return big, big[:n].view(shape)

    for kind in ("select", "attn", "attn sel", "attn f32"):
        fn = rdkv.lib().rdkv_q4_select_workspace_bytes if kind == "select" else rdkv.lib().rdkv_q4_attn_workspace_bytes
        nb = fn(ctypes.byref(c.c), h * G, T)
        big = torch.full((nb + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        big[:rdkv.Q4_COUNTER_BYTES] = 0
        ws = big[:nb]
        for _ in range(2):
            if kind == "select":
                guards = [guarded((B, T, h, 9), torch.int32)]
                rdkv.rdkv_q4_select(c, q, 9, out=guards[0][1], ws=ws)
                sel = guards[0][1].clone()
                assert (sel >= -1).all() and (sel < c.page_table.shape[1]).all()
            else:
                guards = [guarded(q.shape, torch.float32 if kind == "attn f32" else q.dtype), guarded(q.shape[:-1], torch.float32)]
                rdkv.rdkv_q4_attn(c, q, sel=sel if kind == "attn sel" else None, out=guards[0][1], lse=guards[1][1], ws=ws)
        assert (big[nb:] == 0xA5).all(), kind
        for b, x in guards:
            assert (b[x.numel():] == 77).all(), kind
        assert (ws[:rdkv.Q4_COUNTER_BYTES] == 0).all(), kind
    assert rdkv.rdkv_q4_status(c) == 0


def test_bad_pages_and_lengths_are_left_out_and_reported():
    lens = [200, 130]
    c, kh, vh = _filled(lens, 1, 64, torch.float16, stride=4, grow=4)
    q = _rows(2, 2, 64, torch.float16, 9).view(2, 1, 2, 64)
    ok = c.page_table.clone()
    for bad in (-1, c.pages.shape[0], 1 << 30):
        c.page_table.copy_(ok)
        c.page_table[0, 1] = bad
        o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV))
        assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        assert rdkv.rdkv_q4_status(c) == 0
        keep = np.r_[0:64, 128:200]
        _check_attention(q, [kh[0][keep], kh[1]], [vh[0][keep], vh[1]], o, lse)
        rdkv.rdkv_q4_select(c, q.to(DEV), 3)
        assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        before = c.pages.clone()
        row = _rows(2 * 80, 1, 64, torch.float16, 3).view(2, 80, 1, 64).to(DEV)
        c.lens.copy_(torch.tensor([140, 130], dtype=torch.int32))  # rows of positions 60 .. 139: pages 0, 1 and 2
        rdkv.rdkv_q4_write(c, row, row)
        assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        k = rdkv.rdkv_q4_read(c, 80, first=torch.tensor([60, 50], dtype=torch.int32, device=DEV),
                              out=(torch.zeros_like(row), torch.zeros_like(row)))[0]
        assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        assert (k[0, 4:68] == 0).all() and (k[0, :4] != 0).any() and (k[0, 68:] != 0).any()
        c.pages.copy_(before)
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.page_table.copy_(ok)
    row = _rows(2, 1, 64, torch.float16, 3).view(2, 1, 1, 64).to(DEV)
    before = c.pages.clone()
    for n, code in (([257, -3], rdkv.RDKV_ERR_CAPACITY), ([1 << 30, 0], rdkv.RDKV_ERR_CAPACITY)):
        c.lens.copy_(torch.tensor(n, dtype=torch.int32))
        rdkv.rdkv_q4_write(c, row, row)
        assert rdkv.rdkv_q4_status(c) == code
        assert torch.equal(c.pages, before)
    # more rows than tokens, than max_rows, backwards, or past the last row
    c.lens.copy_(torch.tensor([5, 130], dtype=torch.int32))
    rows = _rows(20, 1, 64, torch.float16, 3).to(DEV)
    for start, most in (([0, 6, 6], 20), ([0, 4, 4], 3), ([4, 0, 0], 20), ([-3, 0, 0], 20), ([17, 21, 21], 20),
                        ([2 ** 31 - 4, 2 ** 31 - 1, 2 ** 31 - 1], 20)):
        rdkv.rdkv_q4_write(c, rows, rows, row_start=torch.tensor(start, dtype=torch.int32, device=DEV), max_rows=most)
        assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        assert torch.equal(c.pages, before)
    guard = torch.full((24, 1, 64), 7.0, dtype=torch.float16, device=DEV)
    out = guard[:20].view(20, 1, 64), guard.clone()[:20]
    rdkv.rdkv_q4_read(c, 20, row_start=torch.tensor([17, 21, 21], dtype=torch.int32, device=DEV), out=out)
    assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_ERR_INVALID_ARG
    assert (guard == 7).all() and (out[1] == 7).all()


def test_a_side_stream_two_graphs_and_replays():
    """Steps of write, select and attention: eager on a side stream, then captured twice (two graphs of the
    same cache) and replayed with other lengths and rows."""
    B, h, G, D = 3, 2, 4, 128
    base = [64 * 7 - 1, 5, 64 * 12]
    c, _, _ = _filled(base, h, D, torch.bfloat16, stride=14, grow=1)
    q = torch.zeros(B, 1, h * G, D, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(B, 1, h, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step():
        c.lens.add_(1)
        rdkv.rdkv_q4_write(c, k, v)
        sel = rdkv.rdkv_q4_select(c, q, 5)
        return rdkv.rdkv_q4_attn(c, q), rdkv.rdkv_q4_attn(c, q, sel=sel), sel

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    ref = rdkv.Q4Cache(B, h, D, 14 * 64, DEV, pages=c.pages.clone(), bounds=c.bounds.clone(), page_table=c.page_table,
                       lens=c.lens.clone())
    torch.cuda.synchronize()
    for i in range(5):
        q.copy_(_rows(B, h * G, D, torch.bfloat16, 100 + i).view(q.shape))
        k.copy_(_rows(B, h, D, torch.bfloat16, 200 + i).view(k.shape))
        v.copy_(_rows(B, h, D, torch.bfloat16, 300 + i).view(k.shape))
        g, got = graphs[i % 2]
        g.replay()
        ref.lens.add_(1)
        rdkv.rdkv_q4_write(ref, k, v)
        sel = rdkv.rdkv_q4_select(ref, q, 5)
        dense, sparse = rdkv.rdkv_q4_attn(ref, q), rdkv.rdkv_q4_attn(ref, q, sel=sel)
        torch.cuda.synchronize()
        assert torch.equal(got[2], sel)
        for a, b in ((got[0], dense), (got[1], sparse)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert torch.equal(c.pages, ref.pages) and torch.equal(c.lens, ref.lens)
    # a stream given by name: what is allocated there belongs to it
    out, _ = rdkv.rdkv_q4_attn(c, q, stream=side)
    side.synchronize()
    assert torch.equal(out, graphs[0][1][0][0])
    # both graphs at once, on two streams: neither touches what the other counts with
    c.lens.sub_(2)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(1):
        with torch.cuda.stream(one):
            for _ in range(1):
                a = rdkv.rdkv_q4_attn(c, q)
        with torch.cuda.stream(two):
            b = rdkv.rdkv_q4_attn(c, q)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and rdkv.rdkv_q4_status(c) == 0


# ---------------------------------------------------------------- a run of them together
def test_generation_after_a_compressed_prompt():
    """The prompt in the TriZone zones, what is generated after it in the 4-bit cache: every step writes its
    token, attends both and merges; then the oldest generated rows are read back and become a segment."""
    w = synth.WORKLOADS["llama3b"].scaled(n_tokens=900, h_q=6, h_kv=2, window=64, batch=2)
    q, k, v = (t.to(DEV) for t in synth.prefill_batch(w))
    shape = rdkv.shape_of(q, k, w.window)
    sc = rdkv.rdkv_score(shape, q, k, v)
    al = rdkv.rdkv_allocate(shape, sc["g_tok"], sc["w_chan"], k, 2.5, 2.5)
    zones = rdkv.rdkv_pack(shape, al["plan"], k, v, al["bits_tok"], al["bits_chan"], w.window)
    ref = O.pack(k.cpu().numpy(), v.cpu().numpy(), al["bits_tok"].cpu().numpy(), al["bits_chan"].cpu().numpy(), w.window,
                 cap_c=w.window)
    un = O.unpack(ref, w.head_dim)
    gen = rdkv.Q4Cache(w.batch, w.h_kv, w.head_dim, 256, DEV)
    kept_k, kept_v = [], []
    for step in range(70):
        qn, kn, vn = synth.decode_step(w, step)
        gen.lens.add_(1)
        rdkv.rdkv_q4_write(gen, kn[:, None].to(DEV), vn[:, None].to(DEV))
        outs, lses = torch.empty(2, *qn.shape, device=DEV), torch.empty(2, *qn.shape[:2], device=DEV)
        rdkv.rdkv_decode_attn_lse(zones, qn.to(DEV), out=outs[0], lse=lses[0])
        rdkv.rdkv_q4_attn(gen, qn.to(DEV), out=outs[1], lse=lses[1])
        out, lse = rdkv.rdkv_merge_attn(outs, lses)
        kept_k.append(O.q4_values(*O.q4_quantize(kn.float().numpy())))
        kept_v.append(O.q4_values(*O.q4_quantize(vn.float().numpy())))
        if step in (0, 1, 63, 64, 69):
            zo, zl = O.decode_lse(ref, qn.numpy(), unpacked=un)
            K, V = np.stack(kept_k, 1), np.stack(kept_v, 1)
            G = w.h_q // w.h_kv
            go, gl = np.zeros_like(zo), np.zeros_like(zl)
            for b in range(w.batch):
                for j in range(w.h_q):
                    go[b, j], gl[b, j] = O.attention_lse(qn[b, j].double().numpy(), K[b, :, j // G], V[b, :, j // G])
            mo, ml = O.merge_attention(np.stack([zo, go]), np.stack([zl, gl]))
            assert np.abs(out.cpu().numpy() - mo).max() <= 2e-3 and np.abs(lse.cpu().numpy() - ml).max() <= 2e-3
    assert rdkv.rdkv_q4_status(gen) == 0
    # the first 64 generated rows of every sequence, weighed by a recent query, as a segment of their own
    ks, vs = rdkv.rdkv_q4_read(gen, 64, dtype=torch.float16)
    seg = rdkv.Shape(w.batch, 64, w.h_q, w.h_kv, w.head_dim, 0, rdkv.RDKV_F16)
    qr, lr = qn[:, None].contiguous().to(DEV), lse[:, None].contiguous()
    rs = rdkv.rdkv_recompress_score(seg, ks, vs, qr, lr, float(w.n_tokens))
    ra = rdkv.rdkv_allocate_at_levels(seg, rdkv.plan_levels(al["plan"]), rs["g_tok"], sc["w_chan"], ks)
    part = rdkv.rdkv_pack(seg, ra["plan"], ks, vs, ra["bits_tok"], ra["bits_chan"], 0)
    pref = O.pack(ks.cpu().numpy(), vs.cpu().numpy(), ra["bits_tok"].cpu().numpy(), ra["bits_chan"].cpu().numpy(), 0, cap_c=0)
    assert np.array_equal(part.zone_a_bytes().cpu().numpy(), pref["zone_a"][:int(part.sizes.zone_a_bytes)])
    po, pl = rdkv.rdkv_decode_attn_lse(part, qn.to(DEV))
    eo, el = O.decode_lse(pref, qn.numpy())
    assert np.abs(po.cpu().numpy() - eo).max() <= 2e-3
