"""The 4-bit cache's calls at the edges of what they take, on a GPU: selections, non-finite and huge queries, values next
to fp16's largest, groups of very different size, waits that run out, ties, graphs that run at once."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from mixed_bit_kv_gb300 import rdkv
from test_gpu_q4 import DEV, TYPES, _cache, _check_attention, _filled, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if DEV is None:
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


# ---------------------------------------------------------------- selections
@pytest.mark.parametrize("T", [1, 3])
def test_an_empty_or_misshapen_selection_is_refused(T):
    """Not taken for every position, and not for another order of the same numbers."""
    c, kh, vh = _filled([200, 70], 2, 64, torch.float16)
    q = _rows(2 * T, 4, 64, torch.float16, 9).view(2, T, 4, 64)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device=DEV)
    sel = torch.zeros(2, T, 2, 4, dtype=torch.int32, device=DEV)
    for bad in (sel[..., :0], torch.empty(2, T, 2, 0, dtype=torch.int32, device=DEV), sel.view(2, 2, T, 4) if T > 1 else sel.view(1, 2, 2, 4),
                sel.view(-1, 4)):
        with pytest.raises(rdkv.RDKVError):
            rdkv.rdkv_q4_attn(c, q.to(DEV), sel=bad, out=out)
    assert (out == 7).all()
    sel[:] = -1                                    # a selection of no page that has a size: nothing is seen
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), sel=sel)
    assert (o == 0).all() and (lse == -math.inf).all() and rdkv.rdkv_q4_status(c) == 0


# ---------------------------------------------------------------- non-finite and huge queries
@pytest.mark.parametrize("dtype,out,D,G,T", [("f16", "f16", 128, 4, 1), ("bf16", "bf16", 64, 3, 4), ("f32", "f32", 64, 8, 1),
                                             ("f16", "f32", 128, 5, 2), ("bf16", "bf16", 128, 8, 2), ("f16", "f16", 64, 1, 1)])
@pytest.mark.parametrize("selected", [False, True])
def test_a_nan_query_is_nan_in_out_and_lse_alone(dtype, out, D, G, T, selected):
    """One channel of one query row per sequence is NaN: that row is NaN over whatever it sees (pieces of several blocks, one
    page, a single token), 0 and -inf over nothing, and the other rows hold what they should."""
    dt, lens, h = TYPES[dtype], [9000, 65, 0, T, 1], 2
    c, kh, vh = _filled(lens, h, D, dt)
    q = _rows(len(lens) * T, h * G, D, dt, 9).view(len(lens), T, h * G, D)
    bad = T - 1, G - 1                             # the last token's last head of the first KV head
    q[:, bad[0], bad[1], 5] = float("nan")
    sel = None
    if selected:
        sel = torch.arange(3, dtype=torch.int32).repeat(len(lens), T, h, 1)
        sel[0, :, :, 2] = 140
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), sel=None if sel is None else sel.to(DEV), out_dtype=TYPES[out])
    assert rdkv.rdkv_q4_status(c) == 0
    for b, n in enumerate(lens):
        row, of = o[b, bad[0], bad[1]], lse[b, bad[0], bad[1]]
        if n:
            assert row.isnan().all() and of.isnan(), b
        else:
            assert (row == 0).all() and of == -math.inf
    # and nothing else is: four of the five sequences hold a token, the other heads hold the formula's values
    assert o.isnan().sum() == 4 * D and lse.isnan().sum() == 4
    fine = [i for i in range(h * G) if i != bad[1]]
    for j in range(h):
        heads = [i for i in fine if i // G == j]
        if heads:
            _check_attention(q[:, :, heads], [x[:, j:j + 1] for x in kh], [x[:, j:j + 1] for x in vh], o[:, :, heads], lse[:, :, heads],
                             None if sel is None else sel[:, :, j:j + 1].numpy())


@pytest.mark.parametrize("dtype,out,T", [("bf16", "bf16", 1), ("bf16", "bf16", 3), ("f32", "f32", 1), ("bf16", "f32", 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("exponent", [90, 112, 114, 120, 127])
def test_queries_as_large_as_their_type_allows(exponent, D, dtype, out, T):
    """Queries of up to 2^128 against keys so small that the logits are finite: one key takes all, and lse is its logit.

    A logit is off by at most 2^-17 of sum_c |q_c k_c| / sqrt(D) (the bound of the other tests); seeds are such that the best
    key leads by more than twice that, so the others weigh nothing, and an output is the best key's value: rounded to the
    output's type (eps / 2), with the weight and weight times scale in fp16 (2^-11 each) for 16-bit outputs, 2^-20 for fp32."""
    lens = [700, 40]
    c = _cache(lens, 1, D)
    k = [(_rows(n, 1, D, torch.float32, 20 + i) * 2.0 ** (6 - exponent / 6)).to(TYPES[dtype]) for i, n in enumerate(lens)]
    v = [_rows(n, 1, D, TYPES[dtype], 30 + i) for i, n in enumerate(lens)]
    start = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=DEV)
    rdkv.rdkv_q4_write(c, torch.cat(k).to(DEV), torch.cat(v).to(DEV), row_start=start, max_rows=max(lens))
    g = torch.Generator().manual_seed(7)
    q = (torch.rand(2, T, 4, D, generator=g) * 1.9 + 0.05) * torch.where(torch.rand(2, T, 4, D, generator=g) < 0.5, -1.0, 1.0)
    q = (q * 2.0 ** exponent).to(TYPES[dtype])
    assert q.isfinite().all()
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), out_dtype=TYPES[out])
    assert rdkv.rdkv_q4_status(c) == 0
    eps = torch.finfo(TYPES[out]).eps / 2
    checked = 0
    for b, n in enumerate(lens):
        kh, vh = (O.q4_values(*O.q4_quantize(x[b].float().numpy()))[:, 0] for x in (k, v))
        for t in range(T):
            for j in range(4):
                s = kh[:n - T + t + 1] @ q[b, t, j].double().numpy() / math.sqrt(D)
                off = 2.0 ** -17 * (np.abs(kh) @ np.abs(q[b, t, j].double().numpy())).max() / math.sqrt(D)
                assert s.max() < 2.0 ** 127 and abs(lse[b, t, j].item() - s.max()) <= off + 2.0 ** -20 * abs(s.max()), (b, t, j)
                if np.sort(s)[-1] - np.sort(s)[-2] > 2 * off + 40:
                    best = vh[s.argmax()]
                    tol = eps * np.abs(best) + (2.0 ** -20 if out == "f32" else 2 * 2.0 ** -11) * np.abs(vh).max()
                    assert (np.abs(o[b, t, j].double().cpu().numpy() - best) <= tol).all(), (b, t, j)
                    checked += 1
    assert checked >= 6 * T


def test_a_nan_lse_stays_in_the_merge():
    outs = torch.randn(3, 5, 64, device=DEV)
    lses = torch.tensor([[0.5, float("nan"), -math.inf, 1.0, -math.inf], [1.5, 2.0, float("nan"), -math.inf, -math.inf],
                         [-math.inf, -math.inf, -math.inf, 3.0, -math.inf]], device=DEV)
    outs[0, 1], outs[1, 2] = float("nan"), float("nan")
    out, lse = rdkv.rdkv_merge_attn(outs, lses)
    assert out[1:3].isnan().all() and lse[1:3].isnan().all()
    assert (out[4] == 0).all() and lse[4] == -math.inf
    for r in (0, 3):
        w = lses[:, r].double().softmax(0)
        exp = (w[:, None] * outs[:, r].double()).sum(0)
        # three products, two sums, a quotient and the exponentials: a few roundings of 2^-24
        assert (out[r].double() - exp).abs().max() <= 2.0 ** -20 * outs[:, r].abs().max()
        assert abs(lse[r].double() - lses[:, r].double().logsumexp(0)) <= 2.0 ** -20 * 4


def test_a_nan_query_stays_nan_behind_the_merge_with_another_cache():
    c, kh, vh = _filled([70, 70], 1, 64, torch.float32)
    q = _rows(2, 2, 64, torch.float32, 9)
    q[1, 0, 3] = float("nan")
    outs, lses = torch.zeros(2, 2, 2, 64, device=DEV), torch.zeros(2, 2, 2, device=DEV)
    rdkv.rdkv_q4_attn(c, q.to(DEV), out=outs[0], lse=lses[0])
    out, lse = rdkv.rdkv_merge_attn(outs, lses)
    assert out[1, 0].isnan().all() and lse[1, 0].isnan()
    assert out[0].isfinite().all() and out[1, 1].isfinite().all() and lse[0].isfinite().all() and lse[1, 1].isfinite()


# ---------------------------------------------------------------- values next to fp16's largest
@pytest.mark.parametrize("D,G,T", [(128, 8, 1), (64, 4, 1), (128, 8, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_outputs_of_values_next_to_the_largest_fp16(dtype, D, G, T):
    """Every value is 65504 (or -65504) and so is every mean of them.  The later keys' weights lie where fp16 rounds
    them up by almost 2^-11: their sum is up to 2^-11 larger than the sum they are divided by, which rounds past
    fp16's largest value, so outputs in fp16 have to end there."""
    B, n = 1500, 256
    c = _cache([n] * B, 1, D)
    k = torch.zeros(B, n, 1, D)
    k[:, 64:] = 1.0                                # logits: 0, and the log of the weights below
    v = torch.full((B, n, 1, D), 65504.0)
    v[..., 1::2] = -65504.0
    v[:, :, :, 32:] = 65504.0
    k, v = k.to(TYPES[dtype]).to(DEV), v.half().to(TYPES[dtype]).to(DEV)
    rdkv.rdkv_q4_write(c, k, v)
    w = torch.linspace(4.5e-4, 7e-4, T * G)
    q = (torch.log1p(w) / math.sqrt(D)).view(1, T, G, 1).expand(B, T, G, D).contiguous().to(TYPES[dtype])
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV))
    held = rdkv.rdkv_q4_read(c, 1, dtype=torch.float32)[1][0, 0, 0]
    # eps / 2 of the value; 2^-11 and once more 2^-11 for the weights and weight times scale; fp16's largest value
    eps = torch.finfo(TYPES[dtype]).eps / 2
    exp = held.double()
    assert o.isfinite().all()
    assert ((o.double() - exp).abs() <= (eps + 2 * 2.0 ** -11) * 65504).all()


# ---------------------------------------------------------------- fp32 outputs
def _check_fp32_outputs(k, v, q, logit):
    """fp32 outputs of one sequence (k, v [n, 1, D], q [1, 1, G, D]) against 64 bits, relative to what each group of 32
    channels weighs: sum_t p_t max_c |v_tc| over its own channels c, not over the largest of another group.

    A value is taken as the group's middle (|middle| + |code - 8| scale <= 2.1 max_c |v_tc|) and the code's part, whose
    weight times scale is held in 22 bits (2^-23) and summed with cuts of at most 17 2^-23 of the largest product twice
    for every 32 tokens: together below 2^-17.5; n / 32 sums of those are rounded, 2^-24 each.  `logit` is the largest
    error of a logit; it and the exponential (2^-21) change the weights and their sum."""
    n, _, D = k.shape
    c = _cache([n], 1, D)
    rdkv.rdkv_q4_write(c, k[None].to(DEV), v[None].to(DEV))
    kh, vh = (O.q4_values(*O.q4_quantize(x.float().numpy()))[:, 0] for x in (k, v))
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), out_dtype=torch.float32)
    assert rdkv.rdkv_q4_status(c) == 0
    big = np.repeat(np.abs(vh).reshape(n, D // 32, 32).max(-1), 32, 1)
    for j in range(q.shape[2]):
        s = kh @ q[0, 0, j].double().numpy() / math.sqrt(D)
        p = np.exp(s - s.max())
        tol = (2 * (logit + 2.0 ** -21) + 2.0 ** -17.5 + n / 32 * 2.0 ** -24) * (p @ big) / p.sum()
        err = np.abs(o[0, 0, j].double().cpu().numpy() - p @ vh / p.sum())
        assert (err <= tol).all(), (j, (err / tol).max())
        assert abs(lse[0, 0, j].item() - (s.max() + math.log(p.sum()))) <= logit + 2.0 ** -21 + n * 2.0 ** -24 / 8


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_fp32_outputs_where_one_key_takes_the_weight_and_others_the_values(D, dtype):
    """The first key weighs 2^e and its value is zero; the other keys weigh 1 and hold the same value each, so that
    nothing averages out.  A logit is one product (a few roundings of 2^-24 of up to 14.3)."""
    n = 64 * 20
    g = torch.Generator().manual_seed(1)
    k, v = torch.zeros(n, 1, D), torch.randn(1, 1, D, generator=g).repeat(n, 1, 1)
    k[0], v[0] = 1.0, 0.0
    q = torch.zeros(1, 1, 6, D)
    q[..., 3] = torch.tensor([3.37, 9.61, 12.71, 13.19, 16.23, 20.6]) * math.log(2) * math.sqrt(D)
    _check_fp32_outputs(*(x.to(TYPES[dtype]) for x in (k, v, q)), logit=4 * 2.0 ** -24 * 14.3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("ratio", [1.0, 2.0 ** 10, 2.0 ** 20])
@pytest.mark.parametrize("n", [1, 3, 64, 64 * 9 + 1])
def test_fp32_outputs_of_groups_of_very_different_size(n, ratio, D, dtype):
    """The first two groups' values are `ratio` apart.  The logits are exact: 0, or one product with a key of 0 or 1."""
    g = torch.Generator().manual_seed(2)
    k = torch.randint(0, 2, (n, 1, 1), generator=g).float().expand(n, 1, D).contiguous()
    v = torch.randn(n, 1, D, generator=g)
    v[..., :32] *= math.sqrt(ratio)
    v[..., 32:64] /= math.sqrt(ratio)
    q = torch.zeros(1, 1, 4, D)
    q[..., 3] = torch.tensor([0.0, 0.1, 1.3, 3.3]) * math.sqrt(D)
    _check_fp32_outputs(*(x.to(TYPES[dtype]) for x in (k, v, q)), logit=4 * 2.0 ** -24 * 3.3)


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("D,T,mag", [(64, 1, 1e-3), (128, 1, 1.0), (128, 2, 1e-3), (64, 2, 100.0)])
def test_lse_of_a_few_keys(D, T, mag, dtype, out):
    """Keys of zero: every weight is one, exactly, and so are their sums up to 2^24: lse is the log of their number, to the
    roundings of a base-2 log, of its sum with the reference (zero) and of the factor ln 2 (2^-24 each, and 2^-23 for
    the log): whatever the values' scale is."""
    lens = [T, T + 1, T + 2, T + 4, T + 6, 40, 63, 64, 65, 128, 129, 200, 700, 3001]
    c = _cache(lens, 1, D)
    v = _rows(sum(lens), 1, D, TYPES[dtype], 3, mag)
    start = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    rdkv.rdkv_q4_write(c, torch.zeros_like(v).to(DEV), v.to(DEV), row_start=start, max_rows=max(lens))
    q = _rows(len(lens) * T, 4, D, TYPES[dtype], 9).view(len(lens), T, 4, D)
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), out_dtype=TYPES[out])
    exp = torch.tensor([[math.log(n - T + t + 1) for t in range(T)] for n in lens], dtype=torch.float64)[..., None]
    assert ((lse.double().cpu() - exp).abs() <= 5 * 2.0 ** -24 * exp).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0.0, 20.0])
def test_fp32_logits_of_single_keys(shift, dtype, D):
    """One key a sequence: lse is its logit.  Queries are held in two fp16 parts (22 bits: 2^-22), whose products with
    code - 8 are summed 16 at a time with at most 17 cuts of 2^-23 of the largest, twice a group; the group's middle
    (`shift` makes it the larger part) is a fp32 product with the sum of the queries: some eight roundings of 2^-24 with the
    sums over groups.  One part of the queries alone would be 2^-12 of each channel off, beyond this in most rows."""
    B, h, G = 60, 2, 8
    c = _cache([1] * B, h, D)
    x = (_rows(B, h, D, torch.float32, 3) + shift).to(TYPES[dtype])
    rdkv.rdkv_q4_write(c, x[:, None].to(DEV), x[:, None].to(DEV))
    q = _rows(B, h * G, D, torch.float32, 4).view(B, 1, h * G, D).to(TYPES[dtype])
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), out_dtype=torch.float32)
    codes, scale, zero = O.q4_quantize(x.float().numpy())
    codes = codes.reshape(B, h, 1, -1, 32).astype(np.float64) - 8
    scale, zero = scale.astype(np.float64)[:, :, None, :, None], zero.astype(np.float64)[:, :, None, :, None]
    qg = q.double().numpy().reshape(B, h, G, -1, 32)
    exp = (qg * (zero + 8 * scale + scale * codes)).sum((-2, -1)) / math.sqrt(D)
    tol = (2.0 ** -22 + 34 * 2.0 ** -23) * (np.abs(qg * codes) * scale).sum((-2, -1)) + 2.0 ** -21 * (np.abs(zero + 8 * scale) * np.abs(qg)).sum((-2, -1))
    err = np.abs(lse.double().cpu().numpy().reshape(B, h, G) - exp)
    assert (err <= tol / math.sqrt(D) + 2.0 ** -23 * np.abs(exp)).all(), (err / tol).max()


# ---------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("dtype,out,D,G,T,lens", [
    ("f16", "f16", 128, 4, 1, [64 * 700, 65, 0, 1]), ("bf16", "bf16", 64, 3, 1, [64 * 700 - 5]), ("f16", "f16", 128, 8, 2, [64 * 300, 64 * 30 + 1]),
    ("f32", "f32", 64, 5, 1, [64 * 500, 3]), ("bf16", "f32", 128, 8, 4, [64 * 100, 0, 130]), ("f16", "f16", 64, 1, 1, [1 + 37 * i % 190 for i in range(300)]),
])
@pytest.mark.parametrize("withhold", [1, 2, 7, 65])
def test_waits_that_run_out_are_reported_and_the_workspace_serves_on(withhold, dtype, out, D, G, T, lens):
    """Pages that are waited for and never copied, all of them and a few: the call ends, reports RDKV_ERR_TIMEOUT, writes
    every row and nothing else, leaves its counters at zero, and the calls after it on the same workspace are right."""
    dt, h = TYPES[dtype], 2
    c, kh, vh = _filled(lens, h, D, dt)
    B = len(lens)
    q = _rows(B * T, h * G, D, dt, 9).view(B, T, h * G, D).to(DEV)
    ref = rdkv.rdkv_q4_attn(c, q, out_dtype=TYPES[out])
    sel = torch.arange(3, dtype=torch.int32, device=DEV).repeat(B, T, h, 1)
    ref_sel = rdkv.rdkv_q4_attn(c, q, sel=sel, out_dtype=TYPES[out])
    assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_OK
    for pages in (None, sel):
        ws = c.workspace("attn", h * G, T, torch.cuda.current_stream().cuda_stream)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        o, lse = rdkv.rdkv_q4_timeout_selftest(c, q, sel=pages, out_dtype=TYPES[out], withhold=withhold)
        b.record()
        hit = any((p + j) % withhold == 0 for n in lens for p in range(-(-n // 64)) for j in range(h)
                  if pages is None or p < 3)
        assert rdkv.rdkv_q4_status(c) == (rdkv.RDKV_ERR_TIMEOUT if hit else rdkv.RDKV_OK)
        b.synchronize()
        assert a.elapsed_time(b) < 1000            # a limit of about a millisecond a warp (an ordinary limit is two seconds)
        assert (ws[:rdkv.Q4_COUNTER_BYTES] == 0).all()
        assert o.isfinite().all() and not lse.isnan().any() and (lse < math.inf).all()
        for _ in range(2):
            for x, y in ((rdkv.rdkv_q4_attn(c, q, out_dtype=TYPES[out]), ref), (rdkv.rdkv_q4_attn(c, q, sel=sel, out_dtype=TYPES[out]), ref_sel)):
                assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_OK
        if withhold == 1:                          # no page at all: nothing is seen
            assert (o == 0).all() and (lse == -math.inf).all()


# ---------------------------------------------------------------- selections of many pages next to one another
def _bounded(P, h, D, bounds):
    """A cache of P pages whose bounds are given and whose pages are not read."""
    c = rdkv.Q4Cache(1, h, D, 64 * P, DEV, pages=torch.zeros(P, h, 80 * D, dtype=torch.uint8, device=DEV),
                     lens=torch.tensor([64 * P - 5], dtype=torch.int32, device=DEV))
    c.bounds.copy_(bounds)
    return c


def _check_selection(c, q, bounds, keep, first, last, missing=(), limit=None):
    """Against 64 bits; pages in `missing` (no valid place) come behind all others."""
    h = bounds.shape[1]
    G = q.shape[1] // h
    run = lambda: rdkv.rdkv_q4_select(c, q.to(DEV), keep, n_first=first, n_last=last)
    sel = run()
    for j in range(h):
        s = O.q4_scores(q[0, G * j:G * j + G].double().numpy(), bounds[:, j].double().numpy())
        s[list(missing)] = -np.inf
        assert sel[0, j].tolist() == O.q4_select(s, keep, first, last), j
    assert torch.equal(run(), sel)
    if limit is not None:                          # (a step for every pair of pages: 20 to 100 ms)
        best = math.inf
        for _ in range(5):                         # the fastest of five: the host may be held up between the events
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            run()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        assert best < limit


@pytest.mark.parametrize("P,keep,first,last", [(33, 8, 1, 1), (600, 64, 0, 0), (8193, 9, 2, 3), (16500, 100, 1, 2), (16500, 16000, 1, 1), (20011, 1, 0, 0)])
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (64, "f32")])
def test_selection_among_equal_and_nearly_equal_scores(D, dtype, P, keep, first, last):
    """All scores equal; in runs of equal ones; a zero query; scores that differ in their last bits.  The order is exact,
    and the time goes with the number of pages."""
    g = torch.Generator().manual_seed(P)
    q = torch.randn(1, 6, D, generator=g).to(TYPES[dtype])
    one = torch.randn(1, 2, 2, D, generator=g).sort(2).values.half()
    c = _bounded(P, 2, D, one.expand(P, -1, -1, -1))
    _check_selection(c, q, one.expand(P, -1, -1, -1), keep, first, last, limit=5.0)
    _check_selection(c, torch.zeros_like(q), one.expand(P, -1, -1, -1), keep, first, last, limit=5.0)
    steps = torch.randint(0, 40, (P, 1, 1, 1), generator=g)
    near = one.repeat(P, 1, 1, 1)                  # one channel tells the pages apart, by forty of fp16's smallest steps
    near[:, :, :, 5] = (steps[..., 0].float() * 2.0 ** -24).half()
    c.bounds.copy_(near)
    _check_selection(c, q, near, keep, first, last, limit=5.0)
    runs = one * (1 + steps.float() / 64).half()   # forty scores, each of many pages
    c.bounds.copy_(runs)
    _check_selection(c, q, runs, keep, first, last, limit=5.0)


@pytest.mark.parametrize("P,keep,first,last", [(16500, 64, 1, 2), (300, 20, 2, 2)])
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (64, "f32")])
def test_pages_without_a_place_or_kept_anyway_do_not_blur_the_others(D, dtype, P, keep, first, last):
    """A page outside the pool has no score, and a first or last page may have a huge one: neither makes the others'
    order uncertain (a page that has no place comes behind all that have one, in order)."""
    g = torch.Generator().manual_seed(P)
    q = torch.randn(1, 6, D, generator=g).to(TYPES[dtype])
    e = torch.randn(P, 2, 2, D, generator=g).sort(2).values.half()
    huge = e.clone()
    huge[:first, :, 0], huge[P - last:, :, 1] = -60000.0, 60000.0
    c = _bounded(P, 2, D, huge)
    _check_selection(c, q, huge, keep, first, last, limit=0.4)
    missing = [7, 77, P - last - 1]
    c.page_table[0, missing] = torch.tensor([-1, P, 1 << 30], dtype=torch.int32, device=DEV)
    _check_selection(c, q, huge, keep, first, last, missing, limit=0.4)
    assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_ERR_INVALID_ARG
    # fewer scores than pages to keep: the others follow in order
    some = torch.randperm(P, generator=g)[:P - first - last - 5].tolist()
    missing = sorted({*missing, *(p for p in some if first <= p < P - last)})
    c.page_table[0, missing] = -1
    _check_selection(c, q, huge, keep, first, last, missing)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exponent", [-120, -60, 60, 101, 115, 127])
@pytest.mark.parametrize("P", [40, 700])
def test_selection_for_queries_of_any_size(P, exponent, dtype):
    """The sums' range is that of the queries: up to 2^127 times 65504 times the channels."""
    g = torch.Generator().manual_seed(P)
    e = (torch.randn(P, 2, 2, 64, generator=g) * 2.0 ** torch.randint(-8, 9, (P, 2, 1, 1), generator=g)).sort(2).values.half()
    e[3, :, 1, 7] = 65504.0
    q = torch.randn(1, 4, 64, generator=g).div(8).mul(2.0 ** exponent).to(TYPES[dtype])
    assert q.isfinite().all()
    c = _bounded(P, 2, 64, e)
    _check_selection(c, q, e, 12, 1, 1)
    q[:, 1] *= 2.0 ** -20                          # heads of very different size
    _check_selection(c, q, e, 12, 1, 1)


@pytest.mark.parametrize("P", [40, 700])
def test_selection_for_queries_with_heads_below_the_normal_numbers(P):
    """A head of 2^-140 beside one of 2^-60 whose sums are negative everywhere: the small head's sums are the scores."""
    g = torch.Generator().manual_seed(P)
    e = (torch.rand(P, 1, 2, 64, generator=g) + 0.5).sort(2).values.half()
    q = torch.zeros(1, 2, 64)
    q[0, 0] = -(2.0 ** -60)
    c = _bounded(P, 1, 64, e)
    for least in (0, -2):
        q[0, 1] = torch.randint(least, 3, (64,), generator=g).float() * 2.0 ** -140
        q[0, 1, 5] = 0.0
        _check_selection(c, q, e, 12, 1, 1)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("P", [40, 700])
def test_heads_that_are_not_finite_leave_the_selection_to_the_others(P, dtype):
    g = torch.Generator().manual_seed(P)
    e = (torch.randn(P, 2, 2, 128, generator=g) - 3 * (torch.rand(P, 2, 1, 1, generator=g) < 0.5)).sort(2).values.half()
    q = torch.randn(1, 6, 128, generator=g).to(TYPES[dtype])
    c = _bounded(P, 2, 128, e)
    fine = rdkv.rdkv_q4_select(c, q[:, [0, 2, 3, 5]].contiguous().to(DEV), 12)
    bad = q.clone()
    bad[0, 1, 9], bad[0, 4, 100], bad[0, 4, 3] = float("nan"), float("inf"), float("-inf")
    assert torch.equal(rdkv.rdkv_q4_select(c, bad.to(DEV), 12), fine)
    for value in (float("nan"), float("inf")):     # no head left: the first pages and the last
        bad = q.clone()
        bad[0, 3:] = value
        got = rdkv.rdkv_q4_select(c, bad.to(DEV), 12)
        assert got[0, 1].tolist() == list(range(11)) + [P - 1]
        assert torch.equal(got[0, 0], rdkv.rdkv_q4_select(c, q.to(DEV), 12)[0, 0])


# ---------------------------------------------------------------- lengths that do not fit
def test_rows_without_row_start_for_too_short_lengths_are_reported():
    """A length of zero is an empty slot; one below the number of rows, negative ones among them, is a mistake."""
    for n, code in ((0, rdkv.RDKV_OK), (1, rdkv.RDKV_ERR_INVALID_ARG), (-1, rdkv.RDKV_ERR_INVALID_ARG), (-2 ** 31, rdkv.RDKV_ERR_INVALID_ARG), (2, rdkv.RDKV_OK)):
        c, _, _ = _filled([70, 70], 1, 64, torch.float16)
        before = c.pages.clone()
        c.lens.copy_(torch.tensor([n, 70], dtype=torch.int32))
        rows = _rows(4, 1, 64, torch.float16, 3).view(2, 2, 1, 64).to(DEV)
        rdkv.rdkv_q4_write(c, rows, rows)
        assert rdkv.rdkv_q4_status(c) == code
        first = c.page_table[0, 0].long()
        assert torch.equal(c.pages[first], before[first]) == (n != 2) and not torch.equal(c.pages, before)


def test_lengths_that_no_sequence_can_have_are_reported_by_every_call():
    for lens, code in (([130, 257, 0], rdkv.RDKV_ERR_CAPACITY), ([-1, 130, 0], rdkv.RDKV_ERR_INVALID_ARG), ([256, 0, 2 ** 31 - 1], rdkv.RDKV_ERR_CAPACITY)):
        c, _, _ = _filled([256, 256, 256], 2, 64, torch.float16)
        q = _rows(3 * 2, 4, 64, torch.float16, 9).view(3, 2, 4, 64).to(DEV)
        rows = _rows(3, 2, 64, torch.float16, 3).view(3, 1, 2, 64).to(DEV)
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        held = torch.tensor([min(max(n, 0), 256) for n in lens], dtype=torch.int32)
        sel = rdkv.rdkv_q4_select(c, q, 3)
        assert rdkv.rdkv_q4_status(c) == code
        out, lse = rdkv.rdkv_q4_attn(c, q, sel=sel)
        assert rdkv.rdkv_q4_status(c) == code
        rdkv.rdkv_q4_write(c, rows, rows)
        assert rdkv.rdkv_q4_status(c) == code
        rdkv.rdkv_q4_read(c, 257)
        assert rdkv.rdkv_q4_status(c) == code
        c, _, _ = _filled([256, 256, 256], 2, 64, torch.float16)  # as if the table's end were the length
        c.lens.copy_(held)
        ref = rdkv.rdkv_q4_select(c, q, 3)
        assert torch.equal(sel, ref) and torch.equal(rdkv.rdkv_q4_attn(c, q, sel=ref)[0], out)
        assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_OK


def test_replaced_lengths_are_refused_and_raised_ones_seen():
    c, kh, vh = _filled([200], 1, 64, torch.float16)
    q = _rows(1, 2, 64, torch.float16, 9).view(1, 1, 2, 64)
    with pytest.raises(rdkv.RDKVError):
        c.lens = c.lens - 100
    c.lens -= 100
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV))
    _check_attention(q, [kh[0][:100]], [vh[0][:100]], o, lse)
    with pytest.raises(rdkv.RDKVError):
        c.page_table = c.page_table.clone()


# ---------------------------------------------------------------- at the same time
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
def test_two_captured_graphs_run_at_once(dtype, out):
    """Two graphs of calls on one cache, whose sequences span several blocks of some SMs, replayed on two streams without
    waiting for one another, beside eager calls on a third: each has counters of its own, and every result is right."""
    dt, h, G, D = TYPES[dtype], 1, 4, 128
    c, _, _ = _filled([64 * 90 + 3, 64 * 61], h, D, dt)
    streams = [torch.cuda.Stream() for _ in range(3)]
    qs = [_rows(2, h * G, D, dt, 50 + i).view(2, 1, h * G, D).to(DEV) for i in range(3)]

    def step(q):
        sel = rdkv.rdkv_q4_select(c, q, 40)
        return (*rdkv.rdkv_q4_attn(c, q, out_dtype=TYPES[out]), *rdkv.rdkv_q4_attn(c, q, sel=sel, out_dtype=TYPES[out]), sel)

    used, workspace = set(), c.workspace

    def recorded(*args):
        ws = workspace(*args)
        used.add(ws.data_ptr())
        return ws

    c.workspace = recorded
    refs = [step(q) for q in qs]
    torch.cuda.synchronize()
    graphs, got, places = [], [], [set(used)]
    for q in qs[:2]:
        used.clear()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([step(q) for _ in range(12)])
        graphs.append(g)
        places.append(set(used))
    torch.cuda.synchronize()
    assert all(places) and not (places[0] & places[1] or places[0] & places[2] or places[1] & places[2])
    for _ in range(10):
        for steps in got:
            for x in steps:
                for t in x:
                    t.fill_(-7)
        torch.cuda.synchronize()
        for _ in range(6):                         # each replay overwrites the same outputs
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            with torch.cuda.stream(streams[2]):
                eager = [step(qs[2]) for _ in range(4)]
        torch.cuda.synchronize()
        for steps, ref in (*zip(got, refs), (eager, refs[2])):
            for x in steps:
                for a, b in zip(x, ref):
                    assert torch.equal(a, b)
    assert rdkv.rdkv_q4_status(c) == rdkv.RDKV_OK


def test_workspaces_on_the_host_are_refused_before_any_launch():
    c, kh, vh = _filled([200], 1, 64, torch.float16)
    q = _rows(1, 2, 64, torch.float16, 9).view(1, 1, 2, 64).to(DEV)
    host = torch.zeros(64 << 20, dtype=torch.uint8)
    before = rdkv.lib().rdkv_launch_count()
    for call in (lambda ws: rdkv.rdkv_q4_attn(c, q, ws=ws), lambda ws: rdkv.rdkv_q4_select(c, q, 2, ws=ws),
                 lambda ws: rdkv.rdkv_q4_timeout_selftest(c, q, ws=ws)):
        for ws in (host, host.to(DEV)[::2]):
            with pytest.raises(rdkv.RDKVError):
                call(ws)
    assert rdkv.lib().rdkv_launch_count() == before


def test_counts_past_thirty_two_bits_are_refused_by_the_selection():
    c, kh, vh = _filled([200], 1, 64, torch.float16)
    q = _rows(1, 2, 64, torch.float16, 9).view(1, 1, 2, 64).to(DEV)
    out = torch.zeros(1, 1, 1, 3, dtype=torch.int32, device=DEV)
    for n in ((3, 2 ** 32, 1), (3, 1, 2 ** 32 + 1), (3, -1, 1), (3, 2, 2), (0, 0, 0), (-1, 0, 0)):
        with pytest.raises(rdkv.RDKVError):
            rdkv.rdkv_q4_select(c, q, n[0], n_first=n[1], n_last=n[2], out=out)
    with pytest.raises(rdkv.RDKVError):
        rdkv.rdkv_q4_read(c, 2 ** 32, row_start=torch.tensor([0, 1], dtype=torch.int32, device=DEV), n_rows=1)
