"""GPU parity of the 8-bit cache (rdkv_q8_*) against the CPU oracle.

Written pages, scales and rows read back: every bit.  Evicted: positions, rows, scales and weights, every bit.
Attention: against float64 attention over the values the cache holds.  With S = sum_c |q_c k_c| / sqrt(D), the errors counted are

  a logit   D / 16 products of 16 terms and an accumulator, each term cut below 2^-23 of the largest: 17 D / 16 2^-23 S; fp32
            queries in two fp16 parts: 2^-22 S; the factors of the row, the page and the sum's rounding: 2^-21 of the logit;
            the exponential: 2^-20.  A weight changes by as much relatively, an output by twice that times max|v|, the
            log-sum-exp by that alone;
  sums      four products of 16 terms a page: 68 2^-23, and n fp32 sums, n 2^-24, once for the weights and once for the
            weighted values: 2 n 2^-24; a weight below fp16's normal range, 2^-25 of what is held 2^11 times: 2^-34 of
            max|v| for each of n keys;
  16 bits   a weight's rounding to fp16, 2^-11 (fp32 outputs: two parts, 2^-22), and the output's own, eps / 2 of it.

An accumulated weight is a sum of weights p, each off by its logit's error and the log-sum-exp's, plus the rounding of the sums."""
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


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rows(n, h, D, dt, seed, mag=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, D, generator=g) * mag
    x[:, :, 3] *= 10.0
    return x.to(dt)


def _cache(lens, h, D, stride=None, seed=0, extra=3, grow=0):
    """A cache of shuffled pages whose every code is a NaN, and every scale, until it is written."""
    B = len(lens)
    stride = stride or max(1, max(-(-n // 64) for n in lens))
    n = B * stride + extra
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed))
    table = order[:B * stride].to(torch.int32).view(B, stride)
    for b, t in enumerate(lens):                  # entries that no token needs (yet) are not read
        table[b, -(-t // 64) + grow:] = 1 << 30
    return rdkv.Q8Cache(B, h, D, stride * 64, DEV, pages=torch.full((n, h, 128 * D), 0xFF, dtype=torch.uint8, device=DEV),
                        scales=torch.full((n, h, 2), float("nan"), device=DEV), page_table=table.to(DEV), lens=_ints(lens))


class Held:
    """What one sequence's cache holds, by the oracle: values [n, h, D] and exponents [pages, h] of keys and values."""

    def __init__(self, h, D):
        self.h, self.D = h, D
        self.x = [np.zeros((0, h, D)), np.zeros((0, h, D))]
        self.e = [np.zeros((0, h), int), np.zeros((0, h), int)]

    def write(self, k, v):
        for s, new in enumerate((k, v)):
            new = new.double().numpy()
            while len(new):
                n = len(self.x[s])
                m = min(len(new), 64 - n % 64)
                rows, es = [], []
                for j in range(self.h):
                    held = self.x[s][n - n % 64:, j]
                    r, e = O.q8_append(held, self.e[s][-1, j] if n % 64 else 0, new[:m, j])
                    rows.append(r)
                    es.append(e)
                self.x[s] = np.concatenate([self.x[s][:n - n % 64], np.stack(rows, 1)])
                self.e[s] = np.concatenate([self.e[s][:n // 64], [es]]).astype(int)
                new = new[m:]

    def evict(self, kept):
        """kept [h, n]: positions; a page whose rows all stay keeps its scale."""
        n = kept.shape[1]
        for s in (0, 1):
            x = np.stack([self.x[s][kept[j], j] for j in range(self.h)], 1)
            e = np.zeros((-(-n // 64), self.h), int)
            for p in range(len(e)):
                for j in range(self.h):
                    rows = kept[j, 64 * p:64 * p + 64]
                    if len(rows) == 64 and np.array_equal(rows, np.arange(64 * p, 64 * p + 64)):
                        e[p, j] = self.e[s][p, j]
                        continue
                    y = x[64 * p:64 * p + 64, j]
                    e[p, j] = O.q8_exponent(y)
                    x[64 * p:64 * p + 64, j] = O.q8_values(O.q8_codes(y, e[p, j]), e[p, j])
            self.x[s], self.e[s] = x, e

    @property
    def k(self):
        return self.x[0]

    @property
    def v(self):
        return self.x[1]


def _copy(x):
    y = Held(x.h, x.D)
    y.x, y.e = list(x.x), list(x.e)
    return y


def _write(c, held, k, v):
    """Rows k, v [n, h, D] a sequence, behind what the sequences hold."""
    n = [len(x) for x in k]
    for b in range(c.batch):
        held[b].write(k[b], v[b])
    c.lens.copy_(_ints([len(x.k) for x in held]))
    rdkv.rdkv_q8_write(c, torch.cat(k).to(DEV), torch.cat(v).to(DEV), row_start=_ints([0] + list(np.cumsum(n))), max_rows=max(max(n), 1))


def _filled(lens, h, D, dt, seed=0, mag=1.0, **kw):
    """A cache written in one call, and what it holds."""
    c = _cache(lens, h, D, seed=seed, **kw)
    held = [Held(h, D) for _ in lens]
    _write(c, held, [_rows(n, h, D, dt, seed + 10 * i + 1, mag) for i, n in enumerate(lens)],
           [_rows(n, h, D, dt, seed + 10 * i + 2, mag) for i, n in enumerate(lens)])
    return c, held


def _check_held(c, held):
    """Pages (what the sequences hold of them), scales and rows read back: equal."""
    D, h = c.head_dim, c.h_kv
    pages, scales, table = c.pages.cpu().numpy(), c.scales.cpu().numpy(), c.page_table.cpu().numpy()
    one = np.zeros((64, D))
    for b, x in enumerate(held):
        n = len(x.k)
        for p in range(-(-n // 64)):
            m = min(64, n - 64 * p)
            for j in range(h):
                e = [x.e[s][p, j] for s in (0, 1)]
                assert scales[table[b, p], j].tolist() == [2.0 ** e[0], 2.0 ** e[1]], (b, p, j)
                if p not in (0, n // 64) and (b + p + j) % 7:      # (the oracle's byte order is slow)
                    continue
                sides = []
                for s in (0, 1):
                    side = one.copy()
                    side[:m] = x.x[s][64 * p:64 * p + m, j]
                    sides.append(side)
                full = O.q8_page_bytes(sides[0], e[0], sides[1], e[1])
                live = O.q8_page_bytes(np.where(np.arange(64)[:, None] < m, 448.0, 0.0) + one, 0,
                                       np.where(np.arange(64)[:, None] < m, 448.0, 0.0) + one, 0) != 0
                got = pages[table[b, p], j]
                # (0 and -0 stand for one value)
                same = (got == full) | ((got & 0x7F) == 0) & ((full & 0x7F) == 0)
                assert same[live].all(), (b, p, j)
    lens = [len(x.k) for x in held]
    k, v = rdkv.rdkv_q8_read(c, max(max(lens), 1), row_start=_ints([0] + list(np.cumsum(lens))), n_rows=sum(lens), dtype=torch.float32)
    assert np.array_equal(k.double().cpu().numpy(), np.concatenate([x.k for x in held]))
    assert np.array_equal(v.double().cpu().numpy(), np.concatenate([x.v for x in held]))
    assert rdkv.rdkv_q8_status(c) == 0


def _check_attention(q, held, out, lse, mass=None, before=None):
    """q [B, T, Hq, D]; mass and what it held before [B, h, slots]."""
    q64, out64, lse64 = q.double().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    eps = torch.finfo(out.dtype).eps
    B, T, Hq, D = q64.shape
    for b in range(B):
        n, h = held[b].k.shape[:2]
        G = Hq // h
        want = None if mass is None else before[b].double().cpu().numpy()
        tol_m = None if mass is None else (T * G + 1) * 2.0 ** -24 * np.abs(want)
        for t in range(T):
            m = max(0, n - T + t + 1)
            for j in range(Hq):
                K, V = held[b].k[:m, j // G], held[b].v[:m, j // G]
                if m == 0:
                    assert (out64[b, t, j] == 0).all() and lse64[b, t, j] == -np.inf
                    continue
                ref, ref_lse = O.attention_lse(q64[b, t, j], K, V)
                s = K @ q64[b, t, j] / math.sqrt(D)
                mags = np.abs(K) @ np.abs(q64[b, t, j]) / math.sqrt(D)
                logit = mags.max() * (17 * D / 16 * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -21 * np.abs(s).max() + 2.0 ** -20
                big = np.abs(V).max()
                tol = (2 * logit + 68 * 2.0 ** -23 + 2 * m * 2.0 ** -24 + m * 2.0 ** -34) * big
                if out.dtype != torch.float32:
                    tol = tol + 2.0 ** -11 * big + eps / 2 * np.abs(ref)
                else:
                    tol = tol + 2.0 ** -22 * big
                assert (np.abs(out64[b, t, j] - ref) <= tol).all(), (b, t, j, np.abs(out64[b, t, j] - ref).max(), np.max(tol))
                lse_tol = logit + 2.0 ** -22 * abs(ref_lse) + m * 2.0 ** -24
                assert abs(lse64[b, t, j] - ref_lse) <= lse_tol, (b, t, j, abs(lse64[b, t, j] - ref_lse), lse_tol)
                if mass is not None:
                    p = np.exp(s - ref_lse)
                    want[j // G, :m] += p
                    tol_m[j // G, :m] += p * (logit + lse_tol + (T * G + 1) * 2.0 ** -24) + 2.0 ** -120
        if mass is not None:
            diff = np.abs(mass[b].double().cpu().numpy() - want)
            assert (diff <= tol_m + 2.0 ** -24 * np.abs(want)).all(), (b, (diff - tol_m).max())


# ---------------------------------------------------------------- write and read
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,h", [(64, 1), (64, 3), (128, 2)])
def test_written_pages_scales_and_rows_read_back(D, h, dtype):
    dt, lens, new = TYPES[dtype], [70, 0, 1, 200, 64, 129], [33, 0, 1, 195, 64, 1]
    c = _cache([a - b for a, b in zip(lens, new)], h, D, stride=4, grow=4)
    held = [Held(h, D) for _ in lens]
    for lo, hi in (([0] * 6, [a - b for a, b in zip(lens, new)]), ([a - b for a, b in zip(lens, new)], lens)):
        _write(c, held, [_rows(y - x, h, D, dt, 10 + i, 1.0 + 3.0 * (x > 0)) for i, (x, y) in enumerate(zip(lo, hi))],
               [_rows(y - x, h, D, dt, 30 + i, 1.0 + 3.0 * (x > 0)) for i, (x, y) in enumerate(zip(lo, hi))])
        _check_held(c, held)
    # in other types, from inside, into given tensors that keep what no row fills
    first = [3, 0, 0, 60, 63, 100]
    k = torch.full((6, 50, h, D), 7.0, dtype=dt, device=DEV)
    v = k.clone()
    rdkv.rdkv_q8_read(c, 50, first=_ints(first), out=(k, v))
    for got, name in ((k, "k"), (v, "v")):
        for b in range(6):
            x = getattr(held[b], name)[first[b]:first[b] + 50]
            assert torch.equal(got[b, :len(x)].cpu(), torch.from_numpy(x).to(dt)) and (got[b, len(x):] == 7).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_tokens_that_raise_the_scales_one_by_one(D, dtype):
    """Each token larger than all before it: the earlier codes are taken in the new scale again and again, tokens at
    even and odd slots, past a page's end; then small ones, which raise nothing."""
    c = _cache([0], 2, D, stride=2, grow=2)
    held = [Held(2, D)]
    for i in range(70):
        mag = 2.0 ** (min(i, 66) * 0.35 - 13)
        _write(c, held, [_rows(1, 2, D, TYPES[dtype], i, mag)], [_rows(1, 2, D, TYPES[dtype], 100 + i, mag / 3)])
    _check_held(c, held)
    for n in (2, 3, 9, 17):
        _write(c, held, [_rows(n, 2, D, TYPES[dtype], n, 4.0)], [_rows(n, 2, D, TYPES[dtype], 50 + n, 40.0)])
    _check_held(c, held)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 63, 64, 65, 130])
@pytest.mark.parametrize("at", [0, 1, 7, 8, 33, 63])
def test_runs_of_any_length_at_any_slot(n, at):
    """Every kind of launch (a token, some, whole pages) at even and odd starts and ends; [batch, n] rows of a strided
    projection, an empty slot among them."""
    h, D = 2, 128
    c = _cache([at, at], h, D, stride=4, grow=4)
    held = [Held(h, D), Held(h, D)]
    if at:
        _write(c, held, [_rows(at, h, D, torch.bfloat16, 1), _rows(0, h, D, torch.bfloat16, 1)],
               [_rows(at, h, D, torch.bfloat16, 2), _rows(0, h, D, torch.bfloat16, 1)])
    qkv = torch.zeros(2, n, 7, D, dtype=torch.bfloat16)
    for i in range(7):
        qkv[:, :, i] = _rows(2 * n, 1, D, torch.bfloat16, 20 + i, 1 + 5 * (i % 2)).view(2, n, D)
    held[0].write(qkv[0, :, 3:5], qkv[0, :, 5:7])
    c.lens.copy_(_ints([at + n, 0]))
    x = qkv.to(DEV)
    rdkv.rdkv_q8_write(c, x[:, :, 3:5], x[:, :, 5:7])
    _check_held(c, held)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,h,most", [(128, 2, 1), (64, 3, 20), (128, 1, 130), (64, 1, 64)])
def test_rows_out_of_and_into_wider_ones_and_behind_the_last(D, h, most, dtype):
    """Ragged rows inside wider ones: what lies beside them, between the sequences and behind the last one is neither taken
    nor written."""
    new = [most, 0, (most + 1) // 2, 1]
    old = [63, 5, 0, 100]
    c = _cache(old, h, D, stride=5, grow=5)
    held = [Held(h, D) for _ in old]
    _write(c, held, [_rows(n, h, D, TYPES[dtype], i) for i, n in enumerate(old)], [_rows(n, h, D, TYPES[dtype], 10 + i) for i, n in enumerate(old)])
    rows = sum(new) + 9
    wide = torch.full((rows, 2 * h + 1, D), float("nan"), dtype=TYPES[dtype])
    start = [0] + list(np.cumsum(new))
    for b, n in enumerate(new):
        wide[start[b]:start[b + 1], :2 * h] = _rows(n, 2 * h, D, TYPES[dtype], 20 + b)
        held[b].write(wide[start[b]:start[b + 1], :h], wide[start[b]:start[b + 1], h:2 * h])
    c.lens.copy_(_ints([a + b for a, b in zip(old, new)]))
    x = wide.to(DEV)
    rdkv.rdkv_q8_write(c, x[:, :h], x[:, h:2 * h], row_start=_ints(start), max_rows=most)
    _check_held(c, held)
    back = torch.full_like(x, 7.0)
    rdkv.rdkv_q8_read(c, most, row_start=_ints(start), first=_ints(old), out=(back[:, :h], back[:, h:2 * h]))
    got = back.cpu()
    assert (got[:, 2 * h:] == 7).all() and (got[start[-1]:] == 7).all()
    for b, n in enumerate(new):
        for s in (0, 1):
            want = torch.from_numpy(held[b].x[s][old[b]:]).to(TYPES[dtype])
            assert torch.equal(got[start[b]:start[b + 1], s * h:(s + 1) * h], want)
    assert rdkv.rdkv_q8_status(c) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_flat_huge_tiny_and_non_finite_rows(dtype):
    D, dt = 64, TYPES[dtype]
    x = _rows(64 * 8, 1, D, torch.float32, 1)
    x[:64] = 0.0
    x[64:128] = -0.0
    x[130, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, -math.nan, 6e4, -5.8e4])
    x[192:256] = math.nan
    x[256:320] *= 1e-6
    x[320:384] *= 1e4 if dtype == "f16" else 1e30
    x[384:448] *= 2.0 ** -24 if dtype == "f16" else 1e-38
    x[448:512] = 448.0
    c = _cache([len(x)], 1, D)
    held = [Held(1, D)]
    _write(c, held, [x.to(dt)], [x.flip(0).to(dt)])
    _check_held(c, held)
    e = held[0].e[0][:, 0].tolist()
    assert [e[i] for i in (0, 1, 2, 3, 5, 6, 7)] == [-24, -24, 7, -24, 7, -24, 0]
    k = rdkv.rdkv_q8_read(c, len(x), dtype=dt)[0]
    assert k.isfinite().all() and (k[0, 192:256] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,h,lens", [(128, 8, [32768]), (128, 3, [9001, 64, 5000]), (64, 8, [20011, 1])])
def test_long_prompts_of_every_type(D, h, lens, dtype):
    """Whole prompts, against the definition in torch's casts: the smallest scale of each (page, head), the nearest code."""
    c = _cache(lens, h, D)
    g = torch.Generator(device=DEV).manual_seed(3)
    rows = []
    for i in (0, 1):
        x = torch.randn(sum(lens), h, D, generator=g, device=DEV)
        x *= (torch.randn(x.shape[:2], generator=g, device=DEV) * 4 - 3).exp2()[..., None]  # rows of many sizes
        rows.append(x.to(TYPES[dtype]))
    start = [0] + list(np.cumsum(lens))
    rdkv.rdkv_q8_write(c, *rows, row_start=_ints(start), max_rows=max(lens))
    got = rdkv.rdkv_q8_read(c, max(lens), row_start=_ints(start), n_rows=sum(lens), dtype=torch.float32)
    table = c.page_table.long().cpu()
    for s in (0, 1):
        for b, n in enumerate(lens):
            pages = -(-n // 64)
            x = torch.zeros(pages * 64, h, D, dtype=torch.float64, device=DEV)
            x[:n] = rows[s][start[b]:start[b + 1]].double().clamp(-O.Q8_MOST, O.Q8_MOST)  # (some are infinite in fp16)
            x = x.view(pages, 64, h, D)
            top = x.abs().amax((1, 3))
            edges = torch.tensor([448.0 * 2.0 ** e for e in range(-24, 7)], dtype=torch.float64, device=DEV)
            scale = (torch.searchsorted(edges, top) - 24).double().exp2()
            assert torch.equal(c.scales[table[b, :pages].to(DEV), :, s].double(), scale)
            y = (x / scale[:, None, :, None]).float().to(torch.float8_e4m3fn).double() * scale[:, None, :, None]
            assert int((got[s][start[b]:start[b + 1]].double() != y.view(-1, h, D)[:n]).sum()) == 0
    assert rdkv.rdkv_q8_status(c) == 0


def test_positions_past_two_to_the_thirty_first_bytes():
    """Pages that lie beyond 2^31 (and 2^32) bytes of the pool; weights and logits beyond 2^31 elements."""
    h, D, n = 8, 128, 34000  # 4.5 GB
    c = rdkv.Q8Cache(1, h, D, 192, DEV, pages=torch.empty(n, h, 128 * D, dtype=torch.uint8, device=DEV),
                     page_table=_ints([[n - 1, 17000, n - 2]]))
    held = [Held(h, D)]
    _write(c, held, [_rows(150, h, D, torch.float16, 1)], [_rows(150, h, D, torch.float16, 2)])
    _check_held(c, held)
    q = _rows(1, 2 * h, D, torch.float16, 3).view(1, 1, 2 * h, D)
    mass = c.new_mass()
    out, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
    _check_attention(q, held, out, lse, mass, torch.zeros_like(mass))
    kept = rdkv.rdkv_q8_evict(c, mass, 100, n_last=10)
    m = mass.clone()
    held[0].evict(kept[0].cpu().numpy())
    c.lens.clamp_(max=100)
    _check_held(c, held)
    assert (m[..., 100:] == 0).all()


def test_weights_and_logits_past_two_to_the_thirty_first_elements():
    B, h, G, D, stride = 300, 8, 8, 64, 1792     # logits: 300 x 64 x 114,688 = 2.2e9
    lens = [0] * B
    lens[-1] = 130
    lens[3] = 1
    table = torch.zeros(B, stride, dtype=torch.int32, device=DEV)
    table[-1, :3] = _ints([1, 2, 3])
    c = rdkv.Q8Cache(B, h, D, stride * 64, DEV, pages=torch.full((5, h, 128 * D), 0xFF, dtype=torch.uint8, device=DEV), page_table=table)
    held = [Held(h, D) for _ in lens]
    _write(c, held, [_rows(n, h, D, torch.float16, i) for i, n in enumerate(lens)], [_rows(n, h, D, torch.float16, 500 + i) for i, n in enumerate(lens)])
    q = _rows(B, h * G, D, torch.float16, 3).view(B, 1, h * G, D)
    mass = c.new_mass()
    out, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
    pick = [3, B - 1]
    m = mass[pick][..., :192]
    _check_attention(q[pick], [held[i] for i in pick], out[pick], lse[pick], m, torch.zeros_like(m))
    mass[pick] = 0
    assert not mass.any() and not out[[0, 5, B - 2]].any()
    mass[-1, :, :130] = torch.rand(h, 130, device=DEV)
    before = mass[-1].cpu().numpy()
    kept = rdkv.rdkv_q8_evict(c, mass, 70, n_last=5).cpu()
    assert all(kept[-1, j].tolist() == O.q8_evict(before[j, :130], 70, 0, 5) for j in range(h))
    assert (kept[3, :, 0] == 0).all() and (kept[3, :, 1:] == -1).all() and (kept[0] == -1).all()
    assert rdkv.rdkv_q8_status(c) == 0


# ---------------------------------------------------------------- attention
CASES = [(64, 1, 4, 1, [513]), (128, 2, 3, 1, [1, 64, 65, 0, 300]), (64, 3, 8, 1, [640, 63]), (128, 1, 1, 1, [129]), (128, 2, 4, 4, [200, 3, 1, 0, 77]),
         (64, 2, 5, 3, [70, 250]), (128, 1, 8, 2, [1000]), (64, 1, 2, 64, [100, 30]), (128, 8, 7, 5, [90]), (128, 1, 8, 64, [150])]


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("D,h,G,T,lens", CASES)
def test_attention_and_the_weights_of_its_keys(D, h, G, T, lens, dtype, out):
    c, held = _filled(lens, h, D, TYPES[dtype], seed=D + T)
    q = _rows(len(lens) * T, h * G, D, TYPES[dtype], 9).view(len(lens), T, h * G, D)
    o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), out_dtype=TYPES[out])
    assert o.dtype == TYPES[out]
    _check_attention(q, held, o, lse)
    mass = torch.rand(c.batch, h, c.max_tokens, generator=torch.Generator().manual_seed(1)).to(DEV) * 3
    before = mass.clone()
    o2, lse2 = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass, out_dtype=TYPES[out])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check_attention(q, held, o2, lse2, mass, before)
    for b, n in enumerate(lens):
        assert torch.equal(mass[b, :, n:], before[b, :, n:])
    again = before.clone()
    rdkv.rdkv_q8_attn(c, q.to(DEV), mass=again, out_dtype=TYPES[out])
    assert torch.equal(mass, again) and rdkv.rdkv_q8_status(c) == 0


@pytest.mark.parametrize("D,h,G,T", [(64, 1, 1, 1), (128, 3, 8, 1), (64, 2, 3, 7), (128, 1, 8, 64)])
@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32")])
def test_one_sequence_that_holds_nothing_or_less_than_the_queries(D, h, G, T, dtype, out):
    """(An empty one alone has no items to divide its blocks by.)"""
    for n in (0, 1, T // 2):
        c, held = _filled([n], h, D, TYPES[dtype], stride=3, grow=3)
        q = _rows(T, h * G, D, TYPES[dtype], 5).view(1, T, h * G, D)
        mass = c.new_mass()
        for _ in range(2):
            before = mass.clone()
            o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass, out_dtype=TYPES[out])
            _check_attention(q, held, o, lse, mass, before)
        assert not mass[..., n:].any()
        assert torch.equal(rdkv.rdkv_q8_attn(c, q.to(DEV), out_dtype=TYPES[out])[0], o)
        kept = rdkv.rdkv_q8_evict(c, mass, 5)
        assert kept.tolist() == [[list(range(min(n, 5))) + [-1] * (5 - min(n, 5))] * h] or n > 5
        c.lens.clamp_(max=5)
        assert rdkv.rdkv_q8_status(c) == 0


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("lens,h,G,T", [([20000], 2, 4, 1), ([64 * 40 + 9] * 40, 2, 3, 1), ([9000, 1, 0, 4000], 1, 8, 4), ([1] * 70, 1, 5, 1)])
def test_attention_over_many_blocks(lens, h, G, T, dtype, out):
    D = 128
    c, held = _filled(lens, h, D, TYPES[dtype])
    q = _rows(len(lens) * T, h * G, D, TYPES[dtype], 9).view(len(lens), T, h * G, D)
    mass = c.new_mass()
    o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass, out_dtype=TYPES[out])
    _check_attention(q, held, o, lse, mass, torch.zeros_like(mass))
    rest = torch.arange(c.max_tokens, device=DEV) >= c.lens[:, None, None]
    assert not mass[rest.expand_as(mass)].any()
    # a token's weights sum to one a head
    assert torch.allclose(mass.sum(-1), torch.tensor([min(T, n) * float(G) for n in lens], device=DEV)[:, None].expand(-1, h), rtol=1e-4)


# Units of two to four pages, one to three pages a warp: in 66 to 152 of 152 blocks four or five of the eight warps hold the end of a unit
# that another one began, more than the block's shared memory has places for.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,batch", [(130, 70), (190, 95), (256, 114)])
def test_many_short_units_of_sixteen_rows(n, batch, D):
    lens, h, G, T = [n - b % 3 for b in range(batch)], 8, 4, 4
    c, held = _filled(lens, h, D, torch.bfloat16)
    q = _rows(batch * T, h * G, D, torch.bfloat16, 9).view(batch, T, h * G, D)
    mass = c.new_mass()
    o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
    _check_attention(q, held, o, lse, mass, torch.zeros_like(mass))
    for _ in range(3):
        o2, lse2 = rdkv.rdkv_q8_attn(c, q.to(DEV))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert rdkv.rdkv_q8_status(c) == 0


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T", [1, 4])
def test_attention_over_values_whose_scales_differ_by_two_to_the_thirtieth(T, dtype):
    """Pages of values from 2^-24 to 2^6, weights that favour each in turn: the sums keep the digits of whichever
    contributes."""
    D, h, G, n = 64, 1, 4, 64 * 8
    for turn in range(4):
        k, v = _rows(n, h, D, torch.float32, 1), _rows(n, h, D, torch.float32, 2)
        for p in range(8):
            v[64 * p:64 * p + 64] *= 2.0 ** (-24 + 30 * ((p * 3 + turn) % 8) / 7)
        q = _rows(T, G, D, TYPES[dtype], 3)
        k[64 * turn:64 * turn + 64] += q[0, 0].float() * (0, 0.05, 0.15, 0.4)[turn]
        c = _cache([n], h, D)
        held = [Held(h, D)]
        _write(c, held, [k.to(TYPES[dtype])], [v.to(TYPES[dtype])])
        q = q.view(1, T, G, D)
        mass = c.new_mass()
        o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
        _check_attention(q, held, o, lse, mass, torch.zeros_like(mass))


@pytest.mark.parametrize("mag_q,mag", [(1e-4, 1.0), (30.0, 1.0), (1.0, 1e-3), (0.05, 300.0), (0.0, 1.0), (1.0, 0.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_attention_of_large_and_small_values(dtype, mag_q, mag):
    c, held = _filled([300, 64], 2, 64, TYPES[dtype], mag=mag)
    q = _rows(2, 6, 64, TYPES[dtype], 9, mag_q).view(2, 1, 6, 64)
    mass = c.new_mass()
    o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
    _check_attention(q, held, o, lse, mass, torch.zeros_like(mass))


@pytest.mark.parametrize("exponent", [-126, -100, -84, 40, 100])
def test_queries_from_the_smallest_to_large_numbers(exponent):
    """fp32 and bf16 queries far outside fp16's range: rows are taken times a power of two."""
    for dtype in ("f32", "bf16"):
        c, held = _filled([130], 1, 64, TYPES[dtype], mag=2.0 ** max(-8, -exponent // 8))
        q = (_rows(1, 3, 64, torch.float32, 9) * 2.0 ** exponent).to(TYPES[dtype]).view(1, 1, 3, 64)
        o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV))
        assert o.isfinite().all() and lse.isfinite().all()
        _check_attention(q, held, o, lse)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_queries_next_to_the_largest_numbers(dtype, T):
    """Rows up to 2^127.4 over keys whose scales are the smallest: every logit is finite, and so is every result."""
    c, held = _filled([130], 1, 128, TYPES[dtype], mag=2.0 ** -18)
    q = _rows(T, 3, 128, torch.float32, 9)
    q = (q / q.abs().max() * 1.3 * 2.0 ** 127).to(TYPES[dtype]).view(1, T, 3, 128)
    mass = c.new_mass()
    o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
    assert o.isfinite().all() and lse.isfinite().all() and mass.isfinite().all()
    _check_attention(q, held, o, lse, mass, torch.zeros_like(mass))


def test_a_nan_query_is_nan_alone_and_adds_no_weight():
    D, h, G, T = 64, 2, 3, 2
    c, held = _filled([200, 70], h, D, torch.float16)
    for out in (torch.float16, torch.float32):
        q = _rows(2 * T, h * G, D, torch.float16, 9).view(2, T, h * G, D)
        clean_mass = c.new_mass()
        ref, ref_lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=clean_mass, out_dtype=out)
        q[1, 0, 4, 7] = math.nan
        mass = c.new_mass()
        o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass, out_dtype=out)
        assert o[1, 0, 4].isnan().all() and lse[1, 0, 4].isnan()
        o[1, 0, 4], lse[1, 0, 4] = ref[1, 0, 4], ref_lse[1, 0, 4]
        assert torch.equal(o, ref) and torch.equal(lse, ref_lse)
        assert torch.equal(mass[0], clean_mass[0]) and torch.equal(mass[1, 0], clean_mass[1, 0])
        less = (clean_mass[1, 1].double() - mass[1, 1].double())
        assert mass.isfinite().all() and (less >= -1e-6).all() and abs(float(less.sum()) - 1) < 1e-3


def test_lse_of_a_few_keys():
    """One key's lse is its logit: the sum's exponent and the reference do not round it twice."""
    for D in (64, 128):
        for out in ("f16", "f32"):
            c, held = _filled([1, 2, 3], 1, D, torch.float16)
            q = _rows(3, 5, D, torch.float16, 7).view(3, 1, 5, D)
            _, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), out_dtype=TYPES[out])
            for b in range(3):
                for j in range(5):
                    s = held[b].k[:, 0] @ q[b, 0, j].double().numpy() / math.sqrt(D)
                    mags = (np.abs(held[b].k[:, 0]) @ np.abs(q[b, 0, j].double().numpy())).max() / math.sqrt(D)
                    ref = np.log(np.exp(s - s.max()).sum()) + s.max()
                    assert abs(float(lse[b, 0, j]) - ref) <= 17 * D / 16 * 2.0 ** -23 * mags + 4 * 2.0 ** -23 * (abs(ref) + np.abs(s).max()) + 2.0 ** -21


def test_strided_queries_without_n_q_and_into_given_outputs():
    B, h, G, D = 3, 2, 4, 64
    c, held = _filled([100, 5, 64], h, D, torch.bfloat16)
    qkv = _rows(B, h * G + 2 * h, D, torch.bfloat16, 4).to(DEV)
    q = qkv[:, :h * G]
    ref = rdkv.rdkv_q8_attn(c, q.contiguous())
    out, lse = torch.full((B, h * G, D), 5.0, device=DEV), torch.full((B, h * G), 5.0, device=DEV)
    got = rdkv.rdkv_q8_attn(c, q, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    _check_attention(q.cpu()[:, None], held, out[:, None], lse[:, None])
    assert torch.equal(rdkv.rdkv_q8_attn(c, q)[0], ref[0])


# ---------------------------------------------------------------- eviction
def _evicted(c, held, mass, keep, first, last):
    """Evicts, checks kept, weights and rows; the cache and held are then at the new lengths."""
    before = mass.cpu().numpy().copy()
    kept = rdkv.rdkv_q8_evict(c, mass, keep, n_first=first, n_last=last)
    got, now = kept.cpu().numpy(), mass.cpu().numpy()
    for b, x in enumerate(held):
        n = len(x.k)
        rows = []
        for j in range(c.h_kv):
            want = O.q8_evict(before[b, j, :n], keep, first, last)
            assert got[b, j].tolist() == want + [-1] * (keep - len(want)), (b, j)
            m = before[b, j].copy()
            if n > keep:
                m[:keep] = before[b, j][want]
                m[keep:n] = 0
            assert np.array_equal(now[b, j].view(np.int32), m.view(np.int32)), (b, j)
            rows.append(want)
        if n > keep:
            x.evict(np.array(rows))
    c.lens.clamp_(max=keep)
    _check_held(c, held)
    return kept


def _weights(c, seed, kind="spread"):
    g = torch.Generator().manual_seed(seed)
    m = torch.rand(c.batch, c.h_kv, c.max_tokens, generator=g)
    if kind == "spread":
        m = (6 * m - 8).exp2() * (torch.rand(m.shape, generator=g) > 0.2)
    elif kind == "equal":
        m[:] = 0.25
    elif kind == "few":
        m = (m * 3).floor()
    elif kind == "near":
        m = 1 + (m * 50).floor() * 2.0 ** -23
    elif kind == "any":
        m = (torch.randint(0, 2 ** 32, m.shape, generator=g, dtype=torch.int64) - 2 ** 31).int().view(torch.float32)
        m[..., ::11], m[..., 1::11], m[..., 2::11], m[..., 3::11] = 0.0, -0.0, math.inf, -math.inf
    return m.to(DEV)


@pytest.mark.parametrize("kind", ["spread", "equal", "few", "near", "any"])
@pytest.mark.parametrize("D,h,lens,keep,first,last", [
    (64, 1, [513], 200, 4, 64), (128, 2, [300, 100, 0, 129, 1], 128, 0, 0), (64, 3, [200, 640, 201], 199, 1, 198), (128, 1, [65, 64, 63], 64, 0, 1),
    (64, 2, [700, 90], 1, 0, 0), (64, 2, [700, 90], 1, 1, 0), (64, 1, [257], 256, 0, 256), (128, 1, [5, 2, 3], 2, 1, 1), (64, 1, [1200], 1137, 3, 100)])
def test_eviction(D, h, lens, keep, first, last, kind):
    c, held = _filled(lens, h, D, torch.float16, seed=3)
    mass = _weights(c, 5, kind)
    _evicted(c, held, mass, keep, first, last)


@pytest.mark.parametrize("kind", ["spread", "few", "any"])
@pytest.mark.parametrize("n,keep,last", [(64 * 65, 4096, 500), (64 * 300 + 7, 3000, 0), (64 * 1030, 64 * 1029, 1), (64 * 520, 17, 3)])
def test_eviction_of_long_rows(n, keep, last, kind):
    """Rows spread over clusters of two to eight blocks."""
    D, h = 64, 2
    c, held = _filled([n], h, D, torch.float16)
    _evicted(c, held, _weights(c, 6, kind), keep, 4 if keep > 17 else 0, last)


@pytest.mark.parametrize("kind", ["spread", "few", "any"])
def test_eviction_of_rows_longer_than_shared_memory(kind):
    """More than 131,072 tokens: a warp's last pages' weights are loaded again for every digit."""
    D, n, keep = 64, 210_011, 70_001
    c = rdkv.Q8Cache(1, 1, D, n, DEV)
    c.lens += n
    x = torch.randn(2, 1, n, 1, D, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    rdkv.rdkv_q8_write(c, x[0], x[1])
    mass = _weights(c, 9, kind)
    before, rows = mass[0, 0].cpu().numpy(), rdkv.rdkv_q8_read(c, n, dtype=torch.float32)
    kept = rdkv.rdkv_q8_evict(c, mass, keep, n_first=3, n_last=1000)[0, 0]
    want = O.q8_evict(before[:n], keep, 3, 1000)
    assert kept.tolist() == want
    now = mass[0, 0].cpu().numpy()
    assert np.array_equal(now[:keep].view(np.int32), before[want].view(np.int32)) and not now[keep:n].any()
    c.lens.clamp_(max=keep)
    for a, b in zip(rdkv.rdkv_q8_read(c, keep, dtype=torch.float32), rows):
        # (values below 2^-6 of a scale, 2^-5 at most here, are rounded once more: half of its 2^-9)
        assert (a[0] - b[0][kept.long()]).abs().max() <= 2.0 ** -15
    assert float(c.scales.max()) <= 2.0 ** -5 and rdkv.rdkv_q8_status(c) == 0


def test_eviction_moves_rows_between_pages_of_different_scales():
    D, h, n = 128, 2, 64 * 9 + 30
    k, v = _rows(n, h, D, torch.float32, 1), _rows(n, h, D, torch.float32, 2)
    for p in range(10):
        k[64 * p:64 * p + 64] *= 2.0 ** (5 * p - 30)
        v[64 * p:64 * p + 64] *= 2.0 ** (15 - 5 * p)
    c = _cache([n], h, D)
    held = [Held(h, D)]
    _write(c, held, [k], [v])
    mass = _weights(c, 7)
    for keep in (500, 431, 70, 3):
        _evicted(c, held, mass, keep, 1, 2)


def test_eviction_of_many_sequences_and_again_and_again():
    """More pages than blocks at once; then tokens behind the rows that stayed, and the next eviction."""
    D, h = 64, 2
    lens = [64 * 20 + i for i in range(48)]
    c, held = _filled(lens, h, D, torch.float16)
    mass = _weights(c, 8)
    for step in range(3):
        _evicted(c, held, mass, 900 - 100 * step, 2, 64)
        _write(c, held, [_rows(50 + step, h, D, torch.float16, 10 * step + i, 2.0) for i in range(48)],
               [_rows(50 + step, h, D, torch.float16, 700 + 10 * step + i, 2.0) for i in range(48)])
        mass += 0.01 * (torch.arange(c.max_tokens, device=DEV) < c.lens[:, None, None])
    _check_held(c, held)


def _whole_rows(batch, n, h, D, seed):
    """Rows fp16 [batch, n, h, D] that every scale a page of them can take holds exactly: codes of three digits, each page's
    largest 448 2^0 .. 448 2^4, no value below 2^-6 of the largest scale."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (8 + torch.randint(0, 8, (batch, n, h, D), generator=g, device=DEV)) * torch.randint(0, 6, (batch, n, h, D), generator=g, device=DEV).exp2()
    x *= torch.randint(0, 2, x.shape, generator=g, device=DEV) * 2 - 1
    x[..., 5] = 448.0
    page = torch.arange(n, device=DEV) // 64 * 7 + torch.arange(batch, device=DEV)[:, None]
    return (x * (page % 5).exp2()[..., None, None]).half()


def _check_moved(c, mass, x, n, keep, first, last):
    """Evicts sequences of n rows x (a pair, as _whole_rows makes them) and compares every position, weight and value."""
    before = mass.clone()
    kept = rdkv.rdkv_q8_evict(c, mass, keep, n_first=first, n_last=last)
    host = before.cpu().numpy()
    want = torch.tensor([[O.q8_evict(host[b, j, :n], keep, first, last) for j in range(c.h_kv)] for b in range(c.batch)], dtype=torch.int32)
    assert torch.equal(kept.cpu(), want)
    c.lens.clamp_(max=keep)
    at = kept.long()
    assert torch.equal(mass[..., :keep].view(torch.int32), before.gather(-1, at).view(torch.int32))
    assert not mass[..., keep:n].any() and torch.equal(mass[..., n:].view(torch.int32), before[..., n:].view(torch.int32))
    rows = [y.gather(1, at.transpose(1, 2)[..., None].expand(-1, -1, -1, c.head_dim)) for y in x]
    got = rdkv.rdkv_q8_read(c, keep)
    assert torch.equal(got[0], rows[0]) and torch.equal(got[1], rows[1])
    assert rdkv.rdkv_q8_status(c) == 0
    return rows


@pytest.mark.parametrize("kind", ["spread", "few"])
@pytest.mark.parametrize("D,h,batch", [(128, 2, 60), (64, 3, 50)])
def test_evictions_of_more_pages_than_run_at_once(D, h, batch, kind):
    """A block fills one page after another."""
    n, keep = 64 * 17 + 5, 900
    c = _cache([n] * batch, h, D)
    x = [_whole_rows(batch, n, h, D, i) for i in (1, 2)]
    rdkv.rdkv_q8_write(c, *x)
    assert all(torch.equal(a, b) for a, b in zip(rdkv.rdkv_q8_read(c, n), x))
    mass = _weights(c, 11, kind)
    # of half of the sequences the first eight pages stay as they are: turns that fill nothing
    mass[::2, :, :512] = 100.0
    assert batch * h * -(-keep // 64) > 8 * torch.cuda.get_device_properties(DEV).multi_processor_count
    x = _check_moved(c, mass, x, n, keep, 4, 64)
    _check_moved(c, mass, x, keep, 511, 0, 100)


@pytest.mark.parametrize("kind", ["spread", "few", "near"])
def test_evictions_of_rows_whose_warps_look_up_more_pages_than_lanes(kind):
    """More than 262,144 tokens: a warp of the choice has more than 32 pages, whose places it looks up 32 at a time."""
    D, n, keep = 64, 300_011, 123_457
    c = _cache([n], 1, D, seed=7)
    x = [_whole_rows(1, n, 1, D, i) for i in (3, 4)]
    rdkv.rdkv_q8_write(c, *x)
    _check_moved(c, _weights(c, 12, kind), x, n, keep, 3, 1000)


@pytest.mark.parametrize("D,h,G", [(128, 2, 4), (64, 1, 5)])
def test_sequences_much_shorter_than_their_table(D, h, G):
    """Tables of 131,072 tokens, whose entries behind the sequences may be anything: attended with weights, brought down and
    attended again as in tables that are as long as the sequences."""
    lens, stride, keep = [4160, 4096, 70, 4159, 0, 4100], 2048, 4096
    short, held = _filled(lens, h, D, torch.float16)
    pages = short.page_table.shape[1]
    table = torch.full((len(lens), stride), -1 << 31, dtype=torch.int32, device=DEV)
    table[:, :pages] = short.page_table
    long = rdkv.Q8Cache(len(lens), h, D, stride * 64, DEV, pages=short.pages.clone(), scales=short.scales.clone(), page_table=table,
                        lens=short.lens.clone())
    q = _rows(len(lens) * 2, h * G, D, torch.float16, 5).view(len(lens), 2, h * G, D)
    results = []
    for c in (short, long):
        mass = c.new_mass()
        got = [*rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass), rdkv.rdkv_q8_evict(c, mass, keep, n_first=4, n_last=512)]
        c.lens.clamp_(max=keep)
        got += rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass, out_dtype=torch.float32)
        assert not mass[..., max(lens):].any() and rdkv.rdkv_q8_status(c) == 0
        results.append(got + [mass[..., :pages * 64].clone(), c.pages, c.scales.view(torch.int32)])
    # (the items, and so the order of every sum, come from the lengths)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    _check_attention(q[:1], held[:1], results[0][0][:1], results[0][1][:1])


def test_a_budget_as_large_as_the_argument_allows():
    """(The positions' loop, and the count of pages to fill, passed 2^31.)"""
    c, held = _filled([130], 1, 64, torch.float16)
    mass = _weights(c, 1)
    before = mass.clone()
    for keep in (2 ** 31 - 1, 2 ** 31 - 64, 131):
        kept = rdkv.rdkv_q8_evict(c, mass, keep, n_first=keep)
        assert torch.equal(kept[0, 0, :130].cpu(), torch.arange(130, dtype=torch.int32)) and int(kept[0, 0, 130:].max()) == -1
        assert int(kept[0, 0, 130:].min()) == -1
        del kept
    assert torch.equal(mass, before) and rdkv.rdkv_q8_status(c) == 0
    _check_held(c, held)


def test_other_sequences_of_the_pool_keep_their_pages():
    """Two caches in one pool: what one evicts touches no page of the other, and no page of no one."""
    D, h = 64, 2
    pool = torch.randint(0, 127, (40, h, 128 * D), dtype=torch.uint8, device=DEV)
    scales = torch.rand(40, h, 2, device=DEV)
    order = torch.randperm(40)[:20].int()
    c = rdkv.Q8Cache(1, h, D, 20 * 64, DEV, pages=pool, scales=scales, page_table=order.view(1, 20).to(DEV), lens=_ints([20 * 64 - 3]))
    before, sc = pool.clone(), scales.clone()
    mass = torch.rand(1, h, 20 * 64 + 64, device=DEV)
    rdkv.rdkv_q8_evict(c, mass, 300)
    own = torch.zeros(40, dtype=torch.bool)
    own[order[:5].long()] = True                 # pages that hold the 300 rows now
    assert torch.equal(pool[~own], before[~own]) and torch.equal(scales[~own], sc[~own])
    assert not torch.equal(pool[own], before[own]) and rdkv.rdkv_q8_status(c) == 0


# ---------------------------------------------------------------- bad device data, workspaces, streams, graphs
def test_bad_pages_and_lengths_are_left_out_and_reported():
    lens = [200, 130]
    c, held = _filled(lens, 1, 64, torch.float16, stride=4, grow=4)
    q = _rows(2, 2, 64, torch.float16, 9).view(2, 1, 2, 64)
    ok = c.page_table.clone()
    for bad in (-1, c.pages.shape[0], 1 << 30):
        c.page_table[0, 1] = bad
        mass = c.new_mass()
        o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
        assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_INVALID_ARG and rdkv.rdkv_q8_status(c) == 0
        keep = np.r_[0:64, 128:200]
        part = [Held(1, 64), held[1]]
        part[0].x = [x[keep] for x in held[0].x]
        _check_attention(q, part, o, lse)
        assert not mass[0, 0, 64:128].any() and abs(float(mass[0].sum()) - 2) < 1e-4
        before, sc = c.pages.clone(), c.scales.clone()
        mass = _weights(c, 3)
        m0 = mass.clone()
        kept = rdkv.rdkv_q8_evict(c, mass, 100)  # the first sequence stays as it is, the second is brought down
        assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        assert (kept[0] == -1).all() and torch.equal(mass[0], m0[0])
        assert kept[1, 0].tolist() == O.q8_evict(m0[1, 0, :130].cpu().numpy(), 100, 0, 0)
        own = [int(p) for p in c.page_table[1, :2]]
        rest = [p for p in range(c.pages.shape[0]) if p not in own]
        assert torch.equal(c.pages[rest], before[rest]) and torch.equal(c.scales[rest].view(torch.int32), sc[rest].view(torch.int32))
        c.pages.copy_(before)
        c.scales.copy_(sc)
        row = _rows(2 * 80, 1, 64, torch.float16, 3).view(2, 80, 1, 64).to(DEV)
        c.lens.copy_(_ints([140, 130]))          # rows of positions 60 .. 139: pages 0, 1 and 2
        rdkv.rdkv_q8_write(c, row, row)
        assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        k = rdkv.rdkv_q8_read(c, 80, first=_ints([60, 50]), out=(torch.zeros_like(row), torch.zeros_like(row)))[0]
        assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_INVALID_ARG
        assert (k[0, 4:68] == 0).all() and (k[0, :4] != 0).any() and (k[0, 68:] != 0).any()
        c.pages.copy_(before)
        c.scales.copy_(sc)
        c.page_table.copy_(ok)
        c.lens.copy_(_ints(lens))
    row = _rows(2, 1, 64, torch.float16, 3).view(2, 1, 1, 64).to(DEV)
    before = c.pages.clone()
    for n, code in (([257, -3], rdkv.RDKV_ERR_CAPACITY), ([1 << 30, 0], rdkv.RDKV_ERR_CAPACITY), ([-5, -1], rdkv.RDKV_ERR_INVALID_ARG)):
        c.lens.copy_(_ints(n))
        rdkv.rdkv_q8_write(c, row, row)
        assert rdkv.rdkv_q8_status(c) == code and torch.equal(c.pages, before)
        if max(n) < 1:                           # (a length past the table: the table's tokens, which were not all written)
            mass = c.new_mass()
            out, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
            assert rdkv.rdkv_q8_status(c) == code and not out.any() and (lse == -math.inf).all() and not mass.any()
            assert (rdkv.rdkv_q8_evict(c, mass, 3) == -1).all()
            assert rdkv.rdkv_q8_status(c) == code and torch.equal(c.pages, before)
    for lens_past in ([257, 130], [1 << 30, 130]):
        c, held = _filled([256, 130], 1, 64, torch.float16, stride=4)
        c.page_table[1, 3] = 0
        c.lens.copy_(_ints(lens_past))
        o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV))
        assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_CAPACITY
        _check_attention(q, held, o, lse)
        kept = rdkv.rdkv_q8_evict(c, _weights(c, 3), 200)
        assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_CAPACITY and int(kept[0].max()) < 256 and (kept[1, 0, 130:] == -1).all()


@pytest.mark.parametrize("lens,h,G,T", [([64 * 47 - 3] * 25, 4, 5, 1), ([64 * 300], 1, 8, 3), ([70, 64 * 40, 0], 2, 3, 2), ([1], 1, 1, 64)])
@pytest.mark.parametrize("D", [64, 128])
def test_nothing_is_written_outside_workspaces_and_outputs(D, lens, h, G, T):
    """Guard words behind every workspace, output and weight stay as they were; the counters are zero again."""
    c, _ = _filled(lens, h, D, torch.bfloat16)
    B = len(lens)
    q = _rows(B * T, h * G, D, torch.bfloat16, 9).view(B, T, h * G, D).to(DEV)

    def guarded(shape, dtype):
        n = math.prod(shape)
        big = torch.full((n + 4096,), 77, dtype=dtype, device=DEV)
        return big, big[:n].view(shape)

    for kind in ("attn", "attn f32", "mass", "mass f32", "evict"):
        if kind == "evict":
            nb = rdkv.lib().rdkv_q8_evict_workspace_bytes(ctypes.byref(c.c))
        else:
            nb = rdkv.lib().rdkv_q8_attn_workspace_bytes(ctypes.byref(c.c), h * G, T, "mass" in kind)
        big = torch.full((nb + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        big[:rdkv.Q8_COUNTER_BYTES] = 0
        ws = big[:nb]
        for _ in range(2):
            mass = guarded((B, h, c.max_tokens), torch.float32)
            if kind == "evict":
                guards = [mass, guarded((B, h, 100), torch.int32)]
                rdkv.rdkv_q8_evict(c, mass[1], 100, n_first=1, n_last=2, out=guards[1][1], ws=ws)
            else:
                guards = [mass, guarded(q.shape, torch.float32 if "f32" in kind else q.dtype), guarded(q.shape[:-1], torch.float32)]
                rdkv.rdkv_q8_attn(c, q, mass=mass[1] if "mass" in kind else None, out=guards[1][1], lse=guards[2][1], ws=ws)
        assert (big[nb:] == 0xA5).all(), kind
        for b, x in guards:
            assert (b[x.numel():] == 77).all(), kind
        assert (ws[:rdkv.Q8_COUNTER_BYTES] == 0).all(), kind
    assert rdkv.rdkv_q8_status(c) == 0


def test_one_workspace_serves_calls_of_any_shape_in_turn():
    caches = [_filled([64 * 50, 300], 2, 128, torch.float16), _filled([700], 1, 64, torch.float16)]
    nb = max(rdkv.lib().rdkv_q8_attn_workspace_bytes(ctypes.byref(c.c), 8 * c.h_kv, 4, 1) for c, _ in caches)
    nb = max(nb, *(rdkv.lib().rdkv_q8_evict_workspace_bytes(ctypes.byref(c.c)) for c, _ in caches))
    ws = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    for turn in range(3):
        for c, held in caches:
            mass = _weights(c, turn)
            keep = len(held[0].k) - 150
            before = mass.cpu().numpy()
            kept = rdkv.rdkv_q8_evict(c, mass, keep, n_last=7, ws=ws).cpu().numpy()
            for b, x in enumerate(held):
                if len(x.k) > keep:
                    assert all(kept[b, j].tolist() == O.q8_evict(before[b, j, :len(x.k)], keep, 0, 7) for j in range(c.h_kv))
                    x.evict(kept[b])
            c.lens.clamp_(max=keep)
            _check_held(c, held)
            for G, T, out in ((3, 1, torch.float16), (8, 4, torch.float16), (5, 2, torch.float32)):
                q = _rows(c.batch * T, c.h_kv * G, c.head_dim, torch.float16, turn).view(c.batch, T, -1, c.head_dim)
                mass = c.new_mass()
                o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass, out_dtype=out, ws=ws)
                _check_attention(q, held, o, lse, mass, torch.zeros_like(mass))


def test_a_side_stream_and_two_graphs_replayed_in_turn_and_at_once():
    """Steps of write, attention with weights and eviction: eager on a side stream, then captured twice and replayed
    with other rows; both graphs of two caches at once beside eager calls."""
    B, h, G, D, budget = 3, 2, 4, 128, 64 * 8

    def fresh(seed):
        return _filled([64 * 8 - 1, 500, 64 * 8], h, D, torch.bfloat16, stride=10, grow=10, seed=seed)[0]

    c = fresh(0)
    mass = c.new_mass()
    q = torch.zeros(B, 1, h * G, D, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(B, 1, h, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step(c, mass):
        c.lens.add_(1)
        rdkv.rdkv_q8_write(c, k, v)
        out, lse = rdkv.rdkv_q8_attn(c, q, mass=mass)
        kept = rdkv.rdkv_q8_evict(c, mass, budget, n_first=2, n_last=100)
        c.lens.clamp_(max=budget)
        return out, lse, kept

    def twin(c, mass):
        return rdkv.Q8Cache(B, h, D, 640, DEV, pages=c.pages.clone(), scales=c.scales.clone(), page_table=c.page_table,
                            lens=c.lens.clone()), mass.clone()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c, mass)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(c, mass)
        graphs.append((g, got))
    ref, ref_mass = twin(c, mass)
    torch.cuda.synchronize()
    for i in range(6):
        q.copy_(_rows(B, h * G, D, torch.bfloat16, 100 + i).view(q.shape))
        k.copy_(_rows(B, h, D, torch.bfloat16, 200 + i).view(k.shape))
        v.copy_(_rows(B, h, D, torch.bfloat16, 300 + i).view(k.shape))
        g, got = graphs[i % 2]
        g.replay()
        want = step(ref, ref_mass)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(mass, ref_mass) and torch.equal(c.lens, ref.lens)
        held = [rdkv.rdkv_q8_read(x, 512, dtype=torch.float32, out=tuple(torch.zeros(B, 512, h, D, device=DEV) for _ in "kv")) for x in (c, ref)]
        assert all(torch.equal(a, b) for a, b in zip(*held))
    # graphs of two caches at once, beside eager calls on a third stream
    other, other_mass = twin(c, mass)
    third, third_mass = twin(c, mass)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        got2 = step(other, other_mass)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(one):
            graphs[0][0].replay()
        with torch.cuda.stream(two):
            g2.replay()
        with torch.cuda.stream(side):
            got3 = step(third, third_mass)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(graphs[0][1], got2, got3))
    assert torch.equal(mass, other_mass) and torch.equal(mass, third_mass)
    assert rdkv.rdkv_q8_status(c) == rdkv.rdkv_q8_status(other) == rdkv.rdkv_q8_status(third) == 0


@pytest.mark.parametrize("withhold", [1, 3])
@pytest.mark.parametrize("dtype,out,D,G,T,lens", [("f16", "f16", 128, 3, 1, [64 * 30, 100, 0]), ("f16", "f16", 64, 4, 4, [64 * 200, 7]),
                                                  ("f32", "f32", 128, 8, 1, [64 * 90 - 5] * 3)])
def test_waits_that_run_out_are_reported_and_the_workspace_serves_on(withhold, dtype, out, D, G, T, lens):
    import time
    h = 2
    c, held = _filled(lens, h, D, TYPES[dtype])
    q = _rows(len(lens) * T, h * G, D, TYPES[dtype], 9).view(len(lens), T, h * G, D)
    nb = rdkv.lib().rdkv_q8_attn_workspace_bytes(ctypes.byref(c.c), h * G, T, 0)
    ws = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        o, lse = rdkv.rdkv_q8_timeout_selftest(c, q.to(DEV), out_dtype=TYPES[out], withhold=withhold, ws=ws)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 5
        with_status = rdkv.rdkv_q8_status(c)
        assert with_status == rdkv.RDKV_ERR_TIMEOUT and rdkv.rdkv_q8_status(c) == 0
        assert o.isfinite().all() and not lse.isnan().any()
        assert (ws[:rdkv.Q8_COUNTER_BYTES] == 0).all()
        o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), out_dtype=TYPES[out], ws=ws)
        _check_attention(q, held, o, lse)
    assert rdkv.rdkv_q8_status(c) == 0


@pytest.mark.parametrize("withhold", [1, 3])
@pytest.mark.parametrize("D,h,n,keep,batch", [(128, 2, 64 * 30, 600, 3), (64, 3, 64 * 200 + 5, 3001, 1), (64, 2, 64 * 20 + 3, 900, 60)])
def test_evictions_whose_waits_run_out_are_reported_and_the_workspace_serves_on(withhold, D, h, n, keep, batch):
    """The sequences that were to be brought down are lost, and nothing else is: sequences within the budget, other pages,
    scales and weights; written anew on the same workspace they are brought down as ever."""
    import time
    lens = [n] * batch + [keep, 70, 0]
    c, held = _filled(lens, h, D, torch.float16)
    whole = [_rows(n, h, D, torch.float16, 900 + i) for i in range(2)]
    ws = torch.zeros(rdkv.lib().rdkv_q8_evict_workspace_bytes(ctypes.byref(c.c)), dtype=torch.uint8, device=DEV)
    own = torch.zeros(c.pages.shape[0], dtype=torch.bool)
    own[c.page_table[:batch, :-(-n // 64)].long().flatten().cpu()] = True
    for _ in range(2):
        mass = _weights(c, 4)
        m0, pages, scales = mass.clone(), c.pages.clone(), c.scales.clone().view(torch.int32)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        kept = rdkv.rdkv_q8_evict_timeout_selftest(c, mass, keep, n_first=2, n_last=60, withhold=withhold, wait_cycles=200_000, ws=ws)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 5
        assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_TIMEOUT and rdkv.rdkv_q8_status(c) == 0
        assert (ws[:rdkv.Q8_COUNTER_BYTES] == 0).all()
        assert torch.equal(c.pages[~own], pages[~own]) and torch.equal(c.scales.view(torch.int32)[~own], scales[~own])
        assert torch.equal(mass[batch:], m0[batch:]) and torch.equal(mass[:batch, :, n:], m0[:batch, :, n:])
        for b in (batch, batch + 1, batch + 2):
            want = list(range(lens[b])) + [-1] * (keep - lens[b])
            assert kept[b].tolist() == [want] * h
        # written anew
        for b in range(batch):
            held[b] = Held(h, D)
            if b == 0:
                held[0].write(*whole)
            else:
                held[b].x, held[b].e = held[0].x, held[0].e
        rows = [x[None].expand(batch, -1, -1, -1).reshape(-1, h, D).to(DEV) for x in whole]
        c.lens.copy_(_ints(lens))
        rdkv.rdkv_q8_write(c, *rows, row_start=_ints([n * i for i in range(batch + 1)] + [n * batch] * 3), max_rows=n)
        _check_held(c, held)
    before = mass.copy_(m0).cpu().numpy()
    kept = rdkv.rdkv_q8_evict(c, mass, keep, n_first=2, n_last=60, ws=ws).cpu().numpy()
    for b in range(batch):
        rows = np.array([O.q8_evict(before[b, j, :n], keep, 2, 60) for j in range(h)])
        assert np.array_equal(kept[b], rows)
        if b in (0, batch // 2, batch - 1):
            assert np.array_equal(np.take_along_axis(before[b], rows, 1), mass[b, :, :keep].cpu().numpy())
        held[b] = _copy(held[b])
        held[b].evict(rows)
    c.lens.clamp_(max=keep)
    _check_held(c, held)


def test_weights_without_a_log_sum_exp_and_behind_a_wait_that_ran_out():
    """lse may be NULL; after a wait that ran out nothing is added until the status is read."""
    c, held = _filled([300, 64], 2, 64, torch.float16)
    q = _rows(2, 6, 64, torch.float16, 9).view(2, 1, 6, 64).to(DEV)
    want = c.new_mass()
    out, _ = rdkv.rdkv_q8_attn(c, q, mass=want)
    nb = rdkv.lib().rdkv_q8_attn_workspace_bytes(ctypes.byref(c.c), 6, 1, 1)
    ws, mass, got = torch.zeros(nb, dtype=torch.uint8, device=DEV), c.new_mass(), torch.empty_like(out)
    s = torch.cuda.current_stream().cuda_stream

    def call():
        code = rdkv.lib().rdkv_q8_attn(ctypes.byref(c.c), rdkv.RDKV_F16, q.data_ptr(), 6 * 64, 6, 1, mass.data_ptr(), mass.shape[2],
                                       got.data_ptr(), rdkv.RDKV_F16, None, ws.data_ptr(), nb, s)
        assert code == rdkv.RDKV_OK

    call()
    assert torch.equal(got, out) and torch.equal(mass, want)
    c.status.fill_(rdkv.RDKV_ERR_TIMEOUT)
    call()
    assert torch.equal(mass, want)
    assert rdkv.rdkv_q8_status(c) == rdkv.RDKV_ERR_TIMEOUT
    call()
    assert torch.equal(mass, want + want) and rdkv.rdkv_q8_status(c) == 0


# ---------------------------------------------------------------- a run of them together
def test_a_prompt_scored_evicted_and_decoded_at_a_budget():
    """The prompt's weights from its scorer, its rows in the cache; brought down to a budget, then steps that write,
    attend with weights and evict whenever a page more than the budget is held; merged with a TriZone cache's attention."""
    w = synth.WORKLOADS["llama3b"].scaled(n_tokens=900, h_q=6, h_kv=2, window=64, batch=2)
    q, k, v = (t.to(DEV) for t in synth.prefill_batch(w))
    shape = rdkv.shape_of(q, k, w.window)
    sc = rdkv.rdkv_score(shape, q, k, v)
    c = rdkv.Q8Cache(w.batch, w.h_kv, w.head_dim, 960, DEV)
    held = [Held(w.h_kv, w.head_dim) for _ in range(w.batch)]
    _write(c, held, [x.cpu() for x in k], [x.cpu() for x in v])
    mass = c.new_mass()
    mass[..., :900] = sc["w_tok"]
    budget = 400
    _evicted(c, held, mass, budget, 4, 100)
    for step in range(130):
        qn, kn, vn = synth.decode_step(w, step)
        for b in range(w.batch):
            held[b].write(kn[b][None], vn[b][None])
        c.lens.add_(1)
        rdkv.rdkv_q8_write(c, kn[:, None].to(DEV), vn[:, None].to(DEV))
        before = mass.clone()
        out, lse = rdkv.rdkv_q8_attn(c, qn.to(DEV), mass=mass, out_dtype=torch.float32)
        if step % 16 == 0:
            _check_attention(qn[:, None], held, out[:, None], lse[:, None], mass, before)
        if len(held[0].k) == budget + 64:
            _evicted(c, held, mass, budget, 4, 100)
    # joined with the attention over a compressed cache of the same prompt
    al = rdkv.rdkv_allocate(shape, sc["g_tok"], sc["w_chan"], k, 2.5, 2.5)
    zones = rdkv.rdkv_pack(shape, al["plan"], k, v, al["bits_tok"], al["bits_chan"], w.window)
    outs, lses = torch.empty(2, *qn.shape, device=DEV), torch.empty(2, *qn.shape[:2], device=DEV)
    rdkv.rdkv_decode_attn_lse(zones, qn.to(DEV), out=outs[0], lse=lses[0])
    outs[1], lses[1] = out, lse
    both, lse2 = rdkv.rdkv_merge_attn(outs, lses)
    mo, ml = O.merge_attention(outs.cpu().numpy(), lses.cpu().numpy())
    assert np.abs(both.cpu().numpy() - mo).max() <= 2e-3 and np.abs(lse2.cpu().numpy() - ml).max() <= 2e-3
    assert rdkv.rdkv_q8_status(c) == 0


def test_a_prompt_in_a_long_table_goes_on_in_a_short_one():
    """A second cache on the same pages and scales, with a table for the budget and what is written before the next
    eviction; the weights stay where they are."""
    h, G, D, n, budget = 2, 3, 64, 64 * 60 + 11, 64 * 6
    long, held = _filled([n, 300], h, D, torch.float16)
    mass = _weights(long, 4)
    _evicted(long, held, mass, budget, 4, 50)
    pages = budget // 64 + 1
    c = rdkv.Q8Cache(2, h, D, pages * 64, DEV, pages=long.pages, scales=long.scales,
                     page_table=long.page_table[:, :pages].contiguous(), lens=long.lens)
    spare = sorted(set(range(c.pages.shape[0])) - set(c.page_table.flatten().tolist()))
    c.page_table[1, -(-300 // 64):] = _ints(spare[:pages - -(-300 // 64)])
    for step in range(70):
        k, v = ([_rows(1, h, D, torch.float16, 1000 * i + 2 * step + b) for b in (0, 1)] for i in (1, 2))
        _write(c, held, k, v)
        q = _rows(2, h * G, D, torch.float16, 5000 + step).view(2, 1, h * G, D)
        before = mass.clone()
        out, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
        if step % 20 == 0:
            _check_attention(q, held, out, lse, mass, before)
        if len(held[0].k) == budget + 64:
            _evicted(c, held, mass, budget, 4, 50)
    assert rdkv.rdkv_q8_status(c) == rdkv.rdkv_q8_status(long) == 0


@pytest.mark.parametrize("exponent", [20, 30, 60])
@pytest.mark.parametrize("T", [1, 4])
def test_equal_logits_of_any_size_share_the_weight_over_pages_of_different_scales(T, exponent):
    """Every key the same: the mean of all values, however large the logit is beside the values' scales."""
    D, n = 64, 64 * 5
    for dtype in ("bf16", "f32"):
        k = _rows(1, 1, D, torch.float32, 1).sign().expand(n, 1, D).to(TYPES[dtype])
        v = _rows(n, 1, D, torch.float32, 2)
        for p in range(5):
            v[64 * p:64 * p + 64] *= 2.0 ** (3 - 4 * p)
        c = _cache([n], 1, D)
        held = [Held(1, D)]
        _write(c, held, [k], [v.to(TYPES[dtype])])
        q = (_rows(T, 3, D, torch.float32, 3).sign() * 2.0 ** exponent).to(TYPES[dtype]).view(1, T, 3, D)
        mass = c.new_mass()
        o, lse = rdkv.rdkv_q8_attn(c, q.to(DEV), mass=mass)
        for t in range(T):
            m = n - T + t + 1
            mean = torch.from_numpy(held[0].v[:m, 0].mean(0))
            # (weights are exactly equal: the roundings of the sums and of the output)
            tol = (68 * 2.0 ** -23 + 2 * n * 2.0 ** -24) * held[0].v.max() + torch.finfo(o.dtype).eps / 2 * mean.abs()
            assert ((o[0, t].double().cpu() - mean).abs() <= tol).all()
        assert lse.isfinite().all() and abs(float(mass.double().sum()) / (3 * T) - 1) < 1e-4
