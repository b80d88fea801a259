"""The 8-bit paged cache's operators as they are measured: writing rows and reading them back, attention over the
cache with and without the keys' accumulated weights, and eviction by those weights.

A page holds 64 tokens of one sequence for every KV head; the keys and the values of a (page, head) are fp8 (e4m3)
codes with one power of two each as their scale: x^ = scale * code.  The scale is the smallest 2^e, -24 <= e <= 7,
with max |x| <= 448 2^e; rows written behind others raise it when they need more (the earlier codes are then taken
in the new scale) and never lower it.  `pack_keys` and `pack_values` write the byte order with torch operations, so
that a packed cache can be made without the library.
"""
import math

import torch

own = False

PAGE = 64
LOW, HIGH = -24, 7              # exponents of a scale
BIG = 448.0 * 2.0 ** HIGH       # rows are cut to +-BIG
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 chats: a single new token of each is stored in a page that others began (latency)
        dict(name="store_step", op="store", batch=32, h_kv=8, d=128, dtype="bf16", len=2047, rows=1),
        # the prompt of the 3B-shaped layer written whole after its prefill
        dict(name="store_prompt", op="store", batch=1, h_kv=8, d=128, dtype="f16", len=32768, rows=32768),
        # a chunked prefill's ragged chunks, started inside pages, small heads in fp32
        dict(name="store_ragged", op="store", batch=8, h_kv=4, d=64, dtype="f32", len=3001, rows=777),
        # the tiny single layer: the smallest attention call (latency)
        dict(name="attn_tiny", op="attn", batch=1, h_q=4, h_kv=1, d=64, dtype="f32", len=513, n_q=1, mass=False),
        # four drafted tokens of each of sixteen chats checked at once
        dict(name="attn_draft", op="attn", batch=16, h_q=32, h_kv=8, d=128, dtype="f16", len=8191, n_q=4, mass=False),
        # the batched decode: eight ragged sequences, the last slot empty
        dict(name="attn_batch", op="attn", batch=8, h_q=32, h_kv=8, d=128, dtype="bf16", len=32768, n_q=1, mass=False),
        # one decode token of the 72B-shaped layer at its full length
        dict(name="attn_72b", op="attn", batch=1, h_q=64, h_kv=8, d=128, dtype="f16", len=262144, n_q=1, mass=False),
        # one decode token of the 3B-shaped layer, the keys' weights accumulated
        dict(name="weigh_3b", op="attn", batch=1, h_q=24, h_kv=8, d=128, dtype="f16", len=32777, n_q=1, mass=True),
        # the batched decode of sixteen chats that are kept at a budget
        dict(name="weigh_batch", op="attn", batch=16, h_q=32, h_kv=8, d=128, dtype="bf16", len=8192, n_q=1, mass=True),
        # sixteen chats a page above their budget brought back to it (the recurring step)
        dict(name="evict_step", op="evict", batch=16, h_kv=8, d=128, dtype="bf16", len=4160, keep=4096, first=4, last=512),
        # small heads in fp32, budgets that end inside pages, some sequences within them
        dict(name="evict_ragged", op="evict", batch=8, h_kv=4, d=64, dtype="f32", len=3001, keep=1777, first=1, last=300),
        # the 8B-shaped layer's long prompt brought down to a quarter after its prefill
        dict(name="evict_prompt", op="evict", batch=1, h_kv=8, d=128, dtype="f16", len=131072, keep=32768, first=4, last=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("store", "attn", "attn", "evict"))
    d, h_kv, dtype = rng.choice((64, 128, 128)), rng.choice((1, 2, 4, 8)), rng.choice(("f16", "bf16", "f32"))
    batch = _log(rng, 1, 48)
    most = 1_500_000 // (batch * h_kv)  # (tokens, heads) of the largest listed attention: 2,097,152
    if op == "store":
        rows = _log(rng, 1, max(2, min(16384, most // 4)))
        return dict(op=op, batch=batch, h_kv=h_kv, d=d, dtype=dtype, rows=rows, len=rows + rng.randrange(0, 500))
    if op == "evict":
        length = _log(rng, 2, max(3, min(100_000, most // 2)))
        keep = rng.randrange(max(1, length // 8), length)
        first = min(rng.choice((0, 1, 4)), keep)
        return dict(op=op, batch=batch, h_kv=h_kv, d=d, dtype=dtype, len=length, keep=keep, first=first,
                    last=rng.randrange(0, keep - first + 1) // 2)
    n_q = rng.choice((1, 1, 2, 3, 5, 8))
    length = _log(rng, 1, max(2, min(200_000, most // n_q)))
    return dict(op=op, batch=batch, h_q=rng.randrange(1, 9) * h_kv, h_kv=h_kv, d=d, dtype=dtype, len=length, n_q=n_q,
                mass=rng.random() < 0.5)


def lens_of(case):
    """Tokens that each sequence holds: ragged down to half of `len`, the last of eight or more slots empty."""
    b, n = case["batch"], case["len"]
    if case["op"] == "evict" and n <= case["keep"] + 64:
        return [n] * b  # chats that are brought back as soon as they pass their budget by a page
    lens = [max(1, n - i * n // (2 * b) - (i % 7)) for i in range(b)]
    if case["op"] != "store" and b >= 8:
        lens[-1] = 0
    return lens


def rows_of(case):
    """Rows that each sequence writes: ragged down to half of `rows`."""
    b, n = case["batch"], case["rows"]
    return [min(t, max(1, n - i * n // (2 * b))) for i, t in enumerate(lens_of(case))]


# ---------------------------------------------------------------- the quantiser and the pages' byte order
def exponent_of(top):
    """The smallest e of a scale 2^e that holds magnitudes up to `top` (fp32): top = m 2^k, 448 = 1.75 2^8."""
    m, k = torch.frexp(top)  # m in [0.5, 1)
    return torch.where(top > 0, k - 9 + (m > 0.875).int(), LOW).clamp(LOW, HIGH).int()


def two_to(e):
    """2^e in fp32, exactly (a power function may be a unit off)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def encode(x):
    """Codes uint8 of fp32 values within +-448: e4m3, rounded to the nearest, ties to the even code."""
    a = x.abs()
    k = torch.where(a > 0, torch.frexp(a)[1] - 1, -6).clamp(min=-6)
    code = (k + 6) * 8 + torch.round(a * two_to(3 - k)).int()
    return (code + 128 * (x < 0).int()).to(torch.uint8)


def values_of():
    """The 256 codes' values in fp32."""
    c = torch.arange(256, device="cuda")
    f, m = (c >> 3) & 15, (c & 7).float()
    a = torch.where(f == 0, m * 2.0 ** -9, (8 + m) * two_to(f - 10))
    return torch.where(c >= 128, -a, a)


def cut(x):
    """Rows as the cache takes them: fp32, within +-BIG."""
    return x.float().clamp(-BIG, BIG)


def pack_keys(c):
    """Key bytes [n, 64 D] of codes [n, 64, D]: [token pair][D / 64][token of the pair][64 channels]."""
    n, _, d = c.shape
    return c.view(n, PAGE // 2, 2, d // 64, 64).transpose(2, 3).reshape(n, -1)


def unpack_keys(b, d):
    return b.reshape(-1, PAGE // 2, d // 64, 2, 64).transpose(2, 3).reshape(-1, PAGE, d)


def pack_values(c):
    """Value bytes [n, 64 D]: [8 tokens][D / 64][8 channels][token pair][channel][token of the pair]."""
    n, _, d = c.shape
    return c.view(n, 8, 4, 2, d // 64, 8, 8).permute(0, 1, 4, 5, 2, 6, 3).reshape(n, -1)


def unpack_values(b, d):
    return b.reshape(-1, 8, d // 64, 8, 4, 8, 2).permute(0, 1, 4, 6, 2, 3, 5).reshape(-1, PAGE, d)


def pack_pages(x, live, values):
    """Bytes [n, h, 64 D] and scales [n, h] of n pages of rows x [n, 64, h, D] (cut); live [n, 64]: rows that count."""
    x = x.masked_fill(~live[..., None, None], 0.0)
    e = exponent_of(x.abs().amax((1, 3)))
    c = encode(x * two_to(-e[:, None, :, None]))
    n, _, h, d = x.shape
    c = c.transpose(1, 2).reshape(n * h, PAGE, d)
    return (pack_values if values else pack_keys)(c).view(n, h, -1), two_to(e)


# ---------------------------------------------------------------- what a user's program holds
def _rows(g, n, h_kv, d, u, outlier, keys):
    """n rows [n, h_kv, D] as a model's cache sees them: normal values; keys with four outlier channels a
    head and one row in a hundred aligned with the queries' direction."""
    x = torch.randn(n, h_kv, d, generator=g, device="cuda")
    if keys:
        heavy = (torch.rand(n, h_kv, generator=g, device="cuda") < 0.01).float()
        x += (2.0 * math.sqrt(d)) * heavy[..., None] * u
        x *= outlier
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    b, h, d, dt = case["batch"], case["h_kv"], case["d"], TYPES[case["dtype"]]
    lens = lens_of(case)
    u = torch.randn(h, d, generator=g, device="cuda")
    u /= u.norm(dim=-1, keepdim=True)
    outlier = torch.ones(h, d, device="cuda")
    outlier.scatter_(1, torch.rand(h, d, generator=g, device="cuda").argsort(-1)[:, :4], 10.0)
    stride = max(1, -(-max(lens) // PAGE))
    need = [-(-n // PAGE) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(b, stride, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    pages = torch.zeros(n_pages, h, 128 * d, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n_pages, h, 2, device="cuda")
    state = dict(case=case, lens_host=lens, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), table=table,
                 pages=pages, scales=scales, stride=stride)
    if case["op"] == "store":
        rows = rows_of(case)
        start, first = [0], [t - n for t, n in zip(lens, rows)]
        for n in rows:
            start.append(start[-1] + n)
        # read back from the first written page's first token: the rows that were there may be held anew
        back = [0]
        for t, f in zip(lens, first):
            back.append(back[-1] + t - f // PAGE * PAGE)
        state.update(rows=rows, first_host=first)
        for name, x in (("row_start", start), ("back_start", back), ("back_first", [f // PAGE * PAGE for f in first])):
            state[name] = torch.tensor(x, dtype=torch.int32, device="cuda")
        state["back_host"] = [y - x for x, y in zip(back, back[1:])]
        held = [f % PAGE for f in first]  # what the rows before the written ones left in the first page
        where = [table[i, f // PAGE] for i, f in enumerate(first)]
    else:
        held, where = lens, None
    for i, n in enumerate(held):
        if n == 0:
            continue
        whole = -(-n // PAGE)
        ids = (table[i, :whole] if where is None else where[i].view(1)).long()
        live = (torch.arange(whole * PAGE, device="cuda") < n).view(whole, PAGE)
        for values in (False, True):
            x = torch.zeros(whole * PAGE, h, d, device="cuda", dtype=dt)
            x[:n] = _rows(g, n, h, d, u, outlier, not values).to(dt)
            for a in range(0, whole, 256):
                part, sc = pack_pages(cut(x[a * PAGE:(a + 256) * PAGE]).view(-1, PAGE, h, d), live[a:a + 256], values)
                pages[ids[a:a + 256], :, 64 * d * values:64 * d * (1 + values)] = part
                scales[ids[a:a + 256], :, int(values)] = sc
            del x
    if case["op"] == "store":
        state["k"] = _rows(g, start[-1], h, d, u, outlier, True).to(dt)
        state["v"] = _rows(g, start[-1], h, d, u, outlier, False).to(dt)
    else:
        # weights as some hundred steps leave them: a few keys take most, many hardly any; some take none
        w = torch.rand(b, h, stride * PAGE, generator=g, device="cuda")
        w = (10.0 * (3.0 * torch.randn(w.shape, generator=g, device="cuda") - 4.0).exp2()).masked_fill(w < 0.05, 0.0)
        past = torch.arange(stride * PAGE, device="cuda") >= state["lens"][:, None, None]
        state["weights"] = w.masked_fill(past, 0.0)
        state["mass"] = state["weights"].clone()
    if case["op"] == "attn":
        q = torch.randn(b, case["n_q"], case["h_q"], d, generator=g, device="cuda")
        q += 2.0 * u.repeat_interleave(case["h_q"] // h, 0)
        state["q"] = q.to(dt)
    if case["op"] == "evict":
        kept = [min(n, case["keep"]) for n in lens]
        start = [0]
        for n in kept:
            start.append(start[-1] + n)
        state.update(kept_host=kept, back_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    if own:
        from mixed_bit_kv_gb300 import rdkv

        state["cache"] = rdkv.Q8Cache(b, h, d, stride * PAGE, "cuda", pages=pages, scales=scales, page_table=table,
                                      lens=state["lens"])
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if op == "evict":
        # the prompt's weights, which its scorer gave, into the buffer that goes with the cache; so every pass
        # chooses among, and moves, rows of weights in no order
        state["mass"].copy_(state["weights"])
    if own:
        from mixed_bit_kv_gb300 import rdkv

        c = state["cache"]
        if op == "store":
            rdkv.rdkv_q8_write(c, state["k"], state["v"], row_start=state["row_start"], max_rows=max(state["rows"]))
            k, v = rdkv.rdkv_q8_read(c, max(state["back_host"]), row_start=state["back_start"], first=state["back_first"],
                                     n_rows=sum(state["back_host"]), dtype=state["k"].dtype)
            return dict(k=k, v=v, scales=state["scales"])
        if op == "attn":
            if not case["mass"]:
                out, lse = rdkv.rdkv_q8_attn(c, state["q"])
                return dict(out=out, lse=lse)
            out, lse = rdkv.rdkv_q8_attn(c, state["q"], mass=state["mass"])
            return dict(out=out, lse=lse, mass=state["mass"])
        kept = rdkv.rdkv_q8_evict(c, state["mass"], case["keep"], n_first=case["first"], n_last=case["last"])
        k, v = rdkv.rdkv_q8_read(c, case["keep"], row_start=state["back_start"], n_rows=sum(state["kept_host"]),
                                 dtype=TYPES[case["dtype"]])
        return dict(k=k, v=v, kept=kept, mass=state["mass"])
    return dict(store=plain_store, attn=plain_attention, evict=plain_evict)[op](state)


def plain_held(state, ids):
    """fp32 K, V [n, 64, H, D] of pages ids [n]."""
    d, h = state["case"]["d"], state["case"]["h_kv"]
    lut = values_of()
    got = []
    for j, unpack in enumerate((unpack_keys, unpack_values)):
        c = unpack(state["pages"][ids][..., 64 * d * j:64 * d * (j + 1)].flatten(0, 1), d)
        x = lut[c.int()].view(-1, h, PAGE, d) * state["scales"][ids][..., j, None, None]
        got.append(x.transpose(1, 2))
    return got


def plain_store(state):
    case = state["case"]
    h, d, dt = case["h_kv"], case["d"], state["k"].dtype
    dev = state["k"].device
    r = torch.arange(state["k"].shape[0], device=dev)
    seq = torch.searchsorted(state["row_start"][1:].long(), r, right=True)
    first = state["lens"].long() - state["row_start"].long().diff()
    pos = first[seq] + r - state["row_start"].long()[seq]
    page, slot = state["table"].long()[seq, pos // PAGE], pos % PAGE
    ids = page.unique()
    at = torch.searchsorted(ids, page)
    fresh = torch.zeros(len(ids), dtype=torch.bool, device=dev)
    fresh[at[slot == 0]] = True  # a page whose first token is written starts anew
    # rows that were in the page before, and its scale
    begun = torch.zeros(len(ids), dtype=torch.long, device=dev).scatter_reduce(0, at, slot, "amin", include_self=False)
    before = torch.arange(PAGE, device=dev) < begun[:, None]
    for j, (x, old) in enumerate(zip((state["k"], state["v"]), plain_held(state, ids))):
        rows = old.masked_fill(~before[..., None, None], 0.0)
        new = torch.zeros_like(rows)
        new[at, slot] = cut(x)
        e = exponent_of(new.abs().amax((1, 3)))
        was = torch.frexp(state["scales"][ids][..., j])[1] - 1
        e = torch.maximum(e, was.masked_fill(fresh[:, None], LOW))
        c = encode((rows + new) * two_to(-e[:, None, :, None]))
        c = c.transpose(1, 2).reshape(-1, PAGE, d)
        state["pages"][ids, :, 64 * d * j:64 * d * (j + 1)] = (pack_keys, pack_values)[j](c).view(-1, h, 64 * d)
        state["scales"][ids, :, j] = two_to(e)
    # and back
    return dict(plain_read(state, state["back_first"].long(), dt), scales=state["scales"])


def plain_read(state, first, dt):
    """The rows of sequence b from position first[b], as many as back_start says."""
    start = state["back_start"].long()
    r = torch.arange(sum(state["back_host"] if "back_host" in state else state["kept_host"]), device=start.device)
    seq = torch.searchsorted(start[1:], r, right=True)
    pos = first[seq] + r - start[seq]
    page, slot = state["table"].long()[seq, pos // PAGE], pos % PAGE
    ids = page.unique()
    k, v = (x[torch.searchsorted(ids, page), slot] for x in plain_held(state, ids))
    return dict(k=k.to(dt), v=v.to(dt))


def plain_attention(state):
    case = state["case"]
    b, h, d, n_q, g = case["batch"], case["h_kv"], case["d"], case["n_q"], case["h_q"] // case["h_kv"]
    k, v = (x.reshape(b, -1, h, d) for x in plain_held(state, state["table"].long().flatten()))
    n, dev = k.shape[1], k.device
    k, v = (x.masked_fill((torch.arange(n, device=dev) >= state["lens"][:, None])[..., None, None], 0.0) for x in (k, v))
    seen = state["lens"].long()[:, None] - n_q + 1 + torch.arange(n_q, device=dev)  # keys each query token sees
    q = state["q"].float().view(b, n_q, h, g, d)
    s = torch.einsum("bihgd,bnhd->bihgn", q, k) / math.sqrt(d)
    hide = torch.arange(n, device=dev) >= seen[..., None]  # [B, n_q, n]
    s = s.masked_fill(hide[:, :, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = p.sum(-1)
    out = torch.einsum("bihgn,bnhd->bihgd", p, v) / total.clamp(min=1e-30)[..., None]
    got = dict(out=out.reshape(b, n_q, -1, d).to(state["q"].dtype), lse=(top[..., 0] + total.log()).reshape(b, n_q, -1))
    if case["mass"]:
        state["mass"] += (p / total.clamp(min=1e-30)[..., None]).sum((1, 3))
        got["mass"] = state["mass"]
    return got


def plain_evict(state):
    case, mass, lens = state["case"], state["mass"], state["lens"].long()
    keep, h, d = case["keep"], case["h_kv"], case["d"]
    n, dev = mass.shape[-1], mass.device
    t = torch.arange(n, device=dev)
    some = lens[:, None, None]
    score = mass.masked_fill((t < case["first"]) | (t >= some - case["last"]), math.inf)
    score = score.masked_fill(t >= some, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    if n < keep:
        order = torch.nn.functional.pad(order, (0, keep - n), value=n)
    kept = order.masked_fill(order >= some, n).sort(-1).values  # behind the last: n
    source = kept.clamp(max=n - 1)
    moved = torch.zeros_like(mass)
    m = min(n, keep)
    moved[..., :m] = mass.gather(-1, source)[..., :m].masked_fill(kept[..., :m] == n, 0.0)
    mass.copy_(moved)
    # the kept rows, page by page: dequantised, and held anew in the scale that they need
    pages = -(-keep // PAGE)
    source = torch.nn.functional.pad(source, (0, pages * PAGE - keep))
    live = torch.nn.functional.pad(kept < n, (0, pages * PAGE - keep))[:, 0].reshape(-1, PAGE)  # (the same in every head)
    ids = state["table"].long()
    k, v = (x.reshape(ids.shape[0], -1, h, d) for x in plain_held(state, ids.flatten()))
    at = source.transpose(1, 2)[..., None].expand(-1, -1, -1, d)
    to = torch.nn.functional.pad(ids, (0, max(0, pages - ids.shape[1])))[:, :pages].flatten()
    real = live.any(-1)
    for j, x in enumerate((k, v)):
        new, sc = pack_pages(x.gather(1, at).reshape(-1, PAGE, h, d), live, j == 1)
        state["pages"][to[real], :, 64 * d * j:64 * d * (j + 1)] = new[real]
        state["scales"][to[real], :, j] = sc[real]
    back = plain_read(state, torch.zeros_like(lens), TYPES[case["dtype"]])
    return dict(back, kept=kept.masked_fill(kept == n, -1).to(torch.int32), mass=mass)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    h, d = case["h_kv"], case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    held = 2.0 * d  # bytes of one token and KV head
    if case["op"] == "store":
        rows = sum(rows_of(case)) * h
        # written once and read back once
        return dict(bytes=rows * (2 * held + 4 * d * size), flops=rows * 8.0 * d)
    tokens = sum(lens_of(case)) * h
    if case["op"] == "attn":
        n_q, q_rows = case["n_q"], case["h_q"] * case["batch"] * case["n_q"]
        moved = q_rows * (2 * d * size + 4) + (8 * tokens if case["mass"] else 0)
        return dict(bytes=moved + tokens * held, flops=4.0 * d * tokens * (case["h_q"] // h) * n_q)
    kept = sum(min(n, case["keep"]) for n in lens_of(case)) * h
    # the weights read, and written once where they were copied and once where they end; the kept rows read,
    # written, and read back; their indices
    return dict(bytes=16 * tokens + kept * (3 * held + 2 * d * size + 4), flops=kept * 8.0 * d)


# ---------------------------------------------------------------- the definition in 64 bits
_E4M3 = sorted([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (f - 10) for f in range(1, 16) for m in range(8) if (f, m) != (15, 7)])


def _power(e):
    """2^e in float64, out of its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(x, e):
    """x [.., D] (float64) as codes of the scales 2^e hold it: the nearest of the 127 magnitudes, halves to the even code."""
    grid = torch.tensor(_E4M3, dtype=torch.float64, device=x.device)
    scale = _power(e)
    y = x.abs() / scale
    low = (torch.searchsorted(grid, y, right=True) - 1).clamp(max=len(_E4M3) - 2)
    below, above = grid[low], grid[low + 1]
    up = (y - below > above - y) | ((y - below == above - y) & (low % 2 == 1))
    return torch.where(up, above, below) * x.sign() * scale


def _least(top):
    """The exponent of the smallest scale for magnitudes up to top (a Python number)."""
    e = LOW
    while e < HIGH and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def _exponents(x):
    """The same for every (page, head) of x [n, 64, h, D]."""
    top = x.abs().amax((1, 3))
    edges = torch.tensor([448.0 * 2.0 ** e for e in range(LOW, HIGH)], dtype=torch.float64, device=x.device)
    return (LOW + torch.searchsorted(edges, top)).double()


def _cached(s, i, first, n):
    """K, V float64 [n, H, D] of positions first.. of sequence i, byte by byte out of its pages."""
    d, h = s["case"]["d"], s["case"]["h_kv"]
    pos = torch.arange(first, first + n, device="cuda")
    page, t = s["table"][i].long()[pos // PAGE], (pos % PAGE)[:, None]
    c = torch.arange(d, device="cuda")
    where = (t // 2 * 2 * d + c // 64 * 128 + t % 2 * 64 + c % 64,
             64 * d + t // 8 * 8 * d + c // 64 * 512 + c % 64 // 8 * 64 + t % 8 // 2 * 16 + c % 8 * 2 + t % 2)
    table = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device="cuda")
    table = torch.cat([table, -table])
    got = []
    for j in (0, 1):
        x = torch.empty(n, h, d, dtype=torch.float64, device="cuda")
        for a in range(0, n, 16384):
            for m in range(h):
                b = s["pages"][page[a:a + 16384], m].gather(1, where[j][a:a + 16384])
                x[a:a + 16384, m] = table[b.long()] * s["scales"][page[a:a + 16384], m, j, None].double()
        got.append(x)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    h, d = case["h_kv"], case["d"]
    if case["op"] == "store":
        return _exact_store(s, h, d)
    if case["op"] == "attn":
        return _exact_attention(s, h, d)
    mass = s["weights"].double()
    out = dict(k=[], v=[], kept=torch.full((case["batch"], h, case["keep"]), -1, dtype=torch.int32, device="cuda"),
               mass=torch.zeros_like(mass))
    for i, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        held = _cached(s, i, 0, n)
        rows = []
        for j in range(h):
            if n <= case["keep"]:
                rows.append(list(range(n)))
                continue
            w = s["weights"][i, j, :n].tolist()
            free = range(case["first"], n - case["last"])
            best = sorted(free, key=lambda t: (-w[t], t))[:case["keep"] - case["first"] - case["last"]]
            rows.append(sorted(best) if not case["first"] + case["last"] else
                        sorted(best + list(range(case["first"])) + list(range(n - case["last"], n))))
        at = torch.tensor(rows, device="cuda")  # [h, kept]
        m = at.shape[1]
        out["kept"][i, :, :m] = at.int()
        out["mass"][i, :, :m] = mass[i].gather(1, at)
        for name, x in zip("kv", held):
            y = x.gather(0, at.t()[..., None].expand(-1, -1, d))
            whole = torch.zeros(-(-m // PAGE) * PAGE, h, d, dtype=torch.float64, device="cuda")
            whole[:m] = y
            whole = whole.view(-1, PAGE, h, d)
            e = _exponents(whole)[:, None, :, None]
            out[name].append(torch.cat([_nearest(a, b) for a, b in zip(whole.split(128), e.split(128))]).view(-1, h, d)[:m])
    return dict(out, k=torch.cat(out["k"]), v=torch.cat(out["v"]))


def _exact_store(s, h, d):
    scales = s["scales"].double()
    got = dict(k=[], v=[])
    start = 0
    for i, n in enumerate(s["rows"]):
        first = s["first_host"][i]
        part = first % PAGE
        held = _cached(s, i, first - part, part)
        for j, name in enumerate("kv"):
            x = s[name][start:start + n].double().clamp(-BIG, BIG)
            whole = torch.zeros(-(-(part + n) // PAGE) * PAGE, h, d, dtype=torch.float64, device="cuda")
            whole[part:part + n] = x
            e = _exponents(whole.view(-1, PAGE, h, d))
            if part:
                e[0] = torch.maximum(e[0], torch.log2(scales[s["table"][i, first // PAGE].long(), :, j]).round())
                whole[:part] = held[j]
            y = whole.view(-1, PAGE, h, d)
            y = torch.cat([_nearest(a, b[:, None, :, None]) for a, b in zip(y.split(128), e.split(128))])
            got[name].append(y.reshape(-1, h, d)[:part + n])
            ids = s["table"][i, first // PAGE:first // PAGE + len(e)].long()
            scales[ids, :, j] = _power(e)
        start += n
    return dict(k=torch.cat(got["k"]), v=torch.cat(got["v"]), scales=scales)


def _exact_attention(s, h, d):
    case = s["case"]
    n_q, g = case["n_q"], case["h_q"] // h
    out = torch.zeros(case["batch"], n_q, case["h_q"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], n_q, case["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    mass = s["mass"].double()
    for i, n in enumerate(s["lens_host"]):
        if not n:
            continue
        k, v = _cached(s, i, 0, n)
        for t in range(n_q):
            m = n - n_q + t + 1
            for j in range(h if m > 0 else 0):
                z = s["q"][i, t, j * g:(j + 1) * g].double() @ k[:m, j].t() * d ** -0.5
                p = torch.softmax(z, -1)
                lse[i, t, j * g:(j + 1) * g] = torch.logsumexp(z, -1)
                out[i, t, j * g:(j + 1) * g] = p @ v[:m, j]
                mass[i, j, :m] += p.sum(0)
    got = dict(out=out, lse=lse)
    if case["mass"]:
        got["mass"] = mass
    return got
