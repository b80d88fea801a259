"""The 4-bit paged cache's operators as they are measured: writing rows and reading them back, reading a
stored prefix, attention over the cache, and attention over the pages that a cheap score selects.

A page holds 64 tokens of one sequence for every KV head: per head the K codes, K scales, K zeros, V codes,
V scales, V zeros (`pack_pages` writes the byte layout with torch operations, so a packed cache can be made
without the library).  Groups of 32 channels of a token share an fp16 scale and zero:
x^ = zero + scale * code, code in 0..15.
"""
import math

import torch

own = False

PAGE = 64
GROUP = 32
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BIG = 65504.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 chats: a single new token of each is quantised and stored (latency)
        dict(name="store_step", op="store", batch=32, h_kv=8, d=128, dtype="bf16", len=2047, rows=1),
        # the prompt of the 3B-shaped layer written whole after its prefill
        dict(name="store_prompt", op="store", batch=1, h_kv=8, d=128, dtype="f16", len=32768, rows=32768),
        # a chunked prefill's ragged chunks, started inside pages, small heads in fp32
        dict(name="store_ragged", op="store", batch=8, h_kv=4, d=64, dtype="f32", len=3001, rows=777),
        # a short stored prefix read back for four sequences
        dict(name="load_short", op="load", batch=4, h_kv=1, d=64, dtype="f32", len=500, rows=333),
        # whole caches read back, to be compressed further or moved to another engine
        dict(name="load_batch", op="load", batch=8, h_kv=8, d=128, dtype="f16", len=32768, rows=32768),
        # the tiny single layer: the smallest attention call (latency)
        dict(name="attn_tiny", op="attn", batch=1, h_q=4, h_kv=1, d=64, dtype="f32", len=513, n_q=1),
        # one decode token of the 3B-shaped layer
        dict(name="attn_3b", op="attn", batch=1, h_q=24, h_kv=8, d=128, dtype="f16", len=32777, n_q=1),
        # the batched decode: eight ragged sequences, the last slot empty
        dict(name="attn_batch", op="attn", batch=8, h_q=32, h_kv=8, d=128, dtype="bf16", len=32768, n_q=1),
        # four drafted tokens of each of sixteen chats checked at once
        dict(name="attn_draft", op="attn", batch=16, h_q=32, h_kv=8, d=128, dtype="f16", len=8191, n_q=4),
        # one decode token of the 72B-shaped layer at its full length
        dict(name="attn_72b", op="attn", batch=1, h_q=64, h_kv=8, d=128, dtype="f16", len=262144, n_q=1),
        # the 8B-shaped layer's long context, a thirty-second of its pages attended
        dict(name="sparse_8b", op="sparse", batch=1, h_q=32, h_kv=8, d=128, dtype="f16", len=131072, n_q=1, keep=64),
        # eight ragged sequences of the 3B shape, pages selected for each
        dict(name="sparse_batch", op="sparse", batch=8, h_q=24, h_kv=8, d=128, dtype="bf16", len=32701, n_q=1, keep=48),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("store", "load", "attn", "attn", "sparse"))
    d, h_kv, dtype = rng.choice((64, 128, 128)), rng.choice((1, 2, 4, 8)), rng.choice(("f16", "bf16", "f32"))
    batch = _log(rng, 1, 48)
    most = 1_500_000 // (batch * h_kv)  # (tokens, heads) of the largest listed attention: 2,097,152
    if op in ("store", "load"):
        rows = _log(rng, 1, max(2, min(16384, most // 4)))
        return dict(op=op, batch=batch, h_kv=h_kv, d=d, dtype=dtype, rows=rows, len=rows + rng.randrange(0, 500))
    g = rng.randrange(1, 9)
    n_q = 1 if op == "sparse" else rng.choice((1, 1, 2, 3, 5, 8))
    length = _log(rng, 2000 if op == "sparse" else 1, max(2001, min(200_000, most // n_q)))
    case = dict(op=op, batch=batch, h_q=g * h_kv, h_kv=h_kv, d=d, dtype=dtype, len=length, n_q=n_q)
    if op == "sparse":
        case["keep"] = rng.randrange(8, 100)
    return case


def lens_of(case):
    """Tokens that each sequence holds: ragged down to half of `len`, the last of eight or more slots empty."""
    b, n = case["batch"], case["len"]
    lens = [max(1, n - i * n // (2 * b) - (i % 7)) for i in range(b)]
    if case["op"] in ("attn", "sparse") and b >= 8:
        lens[-1] = 0
    return lens


def rows_of(case):
    """Rows that each sequence writes, or reads: ragged down to half of `rows`."""
    b, n = case["batch"], case["rows"]
    return [min(t, max(1, n - i * n // (2 * b))) for i, t in enumerate(lens_of(case))]


# ---------------------------------------------------------------- the quantiser and the pages' layout
def quantise(x):
    """Codes uint8 [..., D], scale and zero fp16 [..., D / 32] of rows x [..., D]: the definition, in fp32
    (a division by a number would be taken as a product with its inverse: the one by 15 is in 64 bits)."""
    g = x.float().clamp(-BIG, BIG).unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    zero, scale = lo.half(), ((hi - lo).double() / 15).float().half()  # the fp32 quotient, rounded to fp16
    code = ((g - zero.float()) / scale.float()).round().clamp(0, 15)
    code = torch.where(scale > 0, code, 0).to(torch.uint8)
    return code.flatten(-2), scale.squeeze(-1), zero.squeeze(-1)


def dequantise(code, scale, zero):
    """fp32 values zero + scale * code."""
    c = code.float().unflatten(-1, (-1, GROUP))
    return (zero.float()[..., None] + scale.float()[..., None] * c).flatten(-2)


def pack_pages(k, v):
    """Page bytes uint8 [n, 80 D] of n whole pages of one head: k, v each (codes, scale, zero) [n, 64, ...]."""
    (kc, ks, kz), (vc, vs, vz) = k, v
    n, _, d = kc.shape
    ng = d // GROUP
    dev = kc.device
    # K word (token, q, group): channels 32 group + 8 q + e, element e at bit 16 (e mod 2) + 4 (e / 2)
    e = torch.arange(8, device=dev)
    kw = (kc.view(n, PAGE, ng, 4, 8).permute(0, 1, 3, 2, 4).long() << (16 * (e % 2) + 4 * (e // 2))).sum(-1)
    # V word (token pair, g, group): channels 32 group + 4 g + j at bit 4 j, the odd token's 16 bits above
    s = 16 * torch.arange(2, device=dev)[:, None] + 4 * torch.arange(4, device=dev)
    vw = (vc.view(n, PAGE // 2, 2, ng, 8, 4).permute(0, 1, 4, 3, 2, 5).long() << s).sum((-2, -1))

    def words(w):
        w = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
        return w.reshape(n, -1).view(torch.uint8)

    def halves(h):
        return h.contiguous().reshape(n, -1).view(torch.uint8)

    def pairs(h):  # token pair major, group, then the pair's two tokens
        return halves(h.view(n, PAGE // 2, 2, ng).transpose(2, 3))

    return torch.cat([words(kw), pairs(ks), halves(kz), words(vw), pairs(vs), pairs(vz)], 1)


def unpack_pages(b, d):
    """The inverse of pack_pages: ((codes, scale, zero) of K, the same of V), codes uint8 [n, 64, D]."""
    n, ng, dev = b.shape[0], d // GROUP, b.device
    c, m = 32 * d, 4 * d
    kw, ks, kz, vw, vs, vz = b.split([c, m, m, c, m, m], 1)

    def words(x):
        return x.contiguous().view(torch.int32).long() & 0xFFFFFFFF

    def halves(x):
        return x.contiguous().view(torch.float16)

    e = torch.arange(8, device=dev)
    kc = (words(kw).view(n, PAGE, 4, ng, 1) >> (16 * (e % 2) + 4 * (e // 2))) & 15
    kc = kc.permute(0, 1, 3, 2, 4).reshape(n, PAGE, d).to(torch.uint8)
    s = 16 * torch.arange(2, device=dev)[:, None] + 4 * torch.arange(4, device=dev)
    vc = (words(vw).view(n, PAGE // 2, 8, ng, 1, 1) >> s) & 15
    vc = vc.permute(0, 1, 4, 3, 2, 5).reshape(n, PAGE, d).to(torch.uint8)

    def pairs(x):
        return halves(x).view(n, PAGE // 2, ng, 2).transpose(2, 3).reshape(n, PAGE, ng)

    return ((kc, pairs(ks), halves(kz).view(n, PAGE, ng)), (vc, pairs(vs), pairs(vz)))


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
    pages = torch.zeros(n_pages, h, 80 * d, dtype=torch.uint8, device="cuda")
    bounds = torch.zeros(n_pages, h, 2, d, dtype=torch.float16, device="cuda")
    state = dict(case=case, lens_host=lens, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), table=table,
                 pages=pages, bounds=bounds)
    for i, n in enumerate(lens):
        if case["op"] == "store":  # what the rows before the written ones left in the first page
            first = n - rows_of(case)[i]
            part = first % PAGE
            if part:
                x = dequantise(*quantise(_rows(g, part, h, d, u, outlier, True).to(dt)))
                x = x.clamp(-BIG, BIG).half()
                bounds[table[i, first // PAGE].long()] = torch.stack([x.amin(0), x.amax(0)], 1)
            continue
        if n == 0:
            continue
        whole = -(-n // PAGE) * PAGE
        packed = []
        for keys in (True, False):
            x = torch.zeros(whole, h, d, device="cuda", dtype=dt)
            x[:n] = _rows(g, n, h, d, u, outlier, keys).to(dt)
            c, s, z = quantise(x)
            packed.append([t.view(whole // PAGE, PAGE, h, -1).transpose(1, 2).flatten(0, 1) for t in (c, s, z)])
            if keys:
                x = dequantise(c, s, z).clamp(-BIG, BIG).half()
                x = x.view(whole // PAGE, PAGE, h, d)
                top = (torch.arange(whole, device="cuda") >= n).view(-1, PAGE, 1, 1)
                lo = x.masked_fill(top, math.inf).amin(1)
                bounds[table[i, :need[i]].long()] = torch.stack([lo, x.masked_fill(top, -math.inf).amax(1)], 2)
            del x
        ids = table[i, :need[i]].long()
        for at in range(0, need[i], 256):
            part = [[t[at * h:(at + 256) * h] for t in side] for side in packed]
            pages[ids[at:at + 256]] = pack_pages(*part).view(-1, h, 80 * d)
    if case["op"] in ("store", "load"):
        rows = rows_of(case)
        start = [0]
        for n in rows:
            start.append(start[-1] + n)
        first = [t - n for t, n in zip(lens, rows)] if case["op"] == "store" else [(t - n) // 2 for t, n in zip(lens, rows)]
        state.update(rows=rows, first_host=first, row_start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                     first=torch.tensor(first, dtype=torch.int32, device="cuda"))
        if case["op"] == "store":
            state["k"] = _rows(g, start[-1], h, d, u, outlier, True).to(dt)
            state["v"] = _rows(g, start[-1], h, d, u, outlier, False).to(dt)
    else:
        q = torch.randn(b, case["n_q"], case["h_q"], d, generator=g, device="cuda")
        q += 2.0 * u.repeat_interleave(case["h_q"] // h, 0)
        state["q"] = q.to(dt)
    if own:
        from mixed_bit_kv_gb300 import rdkv

        state["cache"] = rdkv.Q4Cache(b, h, d, stride * PAGE, "cuda", pages=pages, bounds=bounds, page_table=table,
                                      lens=state["lens"])
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        from mixed_bit_kv_gb300 import rdkv

        c = state["cache"]
        if op == "store":
            rdkv.rdkv_q4_write(c, state["k"], state["v"], row_start=state["row_start"], max_rows=max(state["rows"]))
            k, v = rdkv.rdkv_q4_read(c, max(state["rows"]), row_start=state["row_start"], first=state["first"],
                                     n_rows=state["k"].shape[0], dtype=state["k"].dtype)
            return dict(k=k, v=v, bounds=state["bounds"])
        if op == "load":
            k, v = rdkv.rdkv_q4_read(c, max(state["rows"]), row_start=state["row_start"], first=state["first"],
                                     n_rows=sum(state["rows"]), dtype=TYPES[state["case"]["dtype"]])
            return dict(k=k, v=v)
        if op == "attn":
            out, lse = rdkv.rdkv_q4_attn(c, state["q"])
            return dict(out=out, lse=lse)
        sel = rdkv.rdkv_q4_select(c, state["q"], state["case"]["keep"], n_first=1, n_last=2)
        out, lse = rdkv.rdkv_q4_attn(c, state["q"], sel=sel)
        return dict(out=out, lse=lse, sel=sel)
    if op == "store":
        return plain_store(state)
    if op == "load":
        return plain_load(state)
    return plain_attention(state)


def plain_store(state):
    k = dequantise(*quantise(state["k"]))
    v = dequantise(*quantise(state["v"]))
    # each written row's page: its sequence is the number of starts at or below it
    dev = k.device
    r = torch.arange(k.shape[0], device=dev)
    seq = torch.searchsorted(state["row_start"][1:].long(), r, right=True)
    pos = state["first"].long()[seq] + r - state["row_start"].long()[seq]
    page = state["table"].long()[seq, pos // PAGE]
    x = k.clamp(-BIG, BIG).half().float()
    lo, hi = (state["bounds"][:, :, j].float() for j in (0, 1))
    fresh = torch.zeros(lo.shape[0], dtype=torch.bool, device=dev)
    fresh[page[pos % PAGE == 0]] = True  # a page whose first token is written starts anew
    lo = lo.masked_fill(fresh[:, None, None], math.inf)
    hi = hi.masked_fill(fresh[:, None, None], -math.inf)
    at = page[:, None, None].expand_as(x)
    lo = lo.scatter_reduce(0, at, x, "amin")
    hi = hi.scatter_reduce(0, at, x, "amax")
    dt = state["k"].dtype
    return dict(k=k.to(dt), v=v.to(dt), bounds=torch.stack([lo, hi], 2).half())


def plain_load(state):
    k, v = plain_values(state)
    n = k.shape[1]
    dev = k.device
    r = torch.arange(int(sum(state["rows"])), device=dev)
    seq = torch.searchsorted(state["row_start"][1:].long(), r, right=True)
    pos = state["first"].long()[seq] + r - state["row_start"].long()[seq]
    dt = TYPES[state["case"]["dtype"]]
    return dict(k=k.flatten(0, 1)[seq * n + pos].to(dt), v=v.flatten(0, 1)[seq * n + pos].to(dt))


def plain_values(state):
    """fp32 K, V [B, stride * 64, H_kv, D] of the cache (what lies past a sequence's length is arbitrary)."""
    b, h, d = (state["case"][x] for x in ("batch", "h_kv", "d"))
    p = state["pages"][state["table"].long()]  # [B, stride, H, bytes]
    sides = unpack_pages(p.flatten(0, 2), d)
    return [dequantise(*s).view(b, -1, h, PAGE, d).transpose(2, 3).flatten(1, 2) for s in sides]


def plain_attention(state):
    case = state["case"]
    b, h, d, n_q, g = case["batch"], case["h_kv"], case["d"], case["n_q"], case["h_q"] // case["h_kv"]
    k, v = plain_values(state)
    n, dev = k.shape[1], k.device
    seen = state["lens"].long()[:, None] - n_q + 1 + torch.arange(n_q, device=dev)  # keys each query token sees
    q = state["q"].float().view(b, n_q, h, g, d)
    s = torch.einsum("bihgd,bnhd->bihgn", q, k) / math.sqrt(d)
    hide = torch.arange(n, device=dev) >= seen[..., None]  # [B, n_q, n]
    sel = None
    if case["op"] == "sparse":
        sel = plain_select(state, seen)
        kept = torch.zeros(b, n_q, h, n // PAGE + 1, dtype=torch.bool, device=dev)
        kept.scatter_(-1, torch.where(sel < 0, n // PAGE, sel).long(), True)
        hide = hide[:, :, None] | ~kept[..., :-1].repeat_interleave(PAGE, -1)
        s = s.masked_fill(hide[:, :, :, None], -math.inf)
    else:
        s = s.masked_fill(hide[:, :, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = p.sum(-1)
    out = torch.einsum("bihgn,bnhd->bihgd", p, v) / total.clamp(min=1e-30)[..., None]
    got = dict(out=out.reshape(b, n_q, -1, d).to(state["q"].dtype), lse=(top[..., 0] + total.log()).reshape(b, n_q, -1))
    if sel is not None:
        got["sel"] = sel
    return got


def plain_select(state, seen):
    """Pages kept for each (sequence, query token, KV head): int32 [B, n_q, H_kv, keep], ascending, -1 behind the
    last.  A page's score bounds its logits from above; the sums are taken in 64 bits (order next to the border)."""
    case = state["case"]
    b, h, d, n_q, keep = (case[x] for x in ("batch", "h_kv", "d", "n_q", "keep"))
    dev = seen.device
    q = state["q"].double().view(b, n_q, h, -1, 1, d)
    e = state["bounds"][state["table"].long()].double().permute(0, 2, 1, 3, 4)[:, None, :, None]  # [B,1,H,1,P,2,D]
    score = torch.maximum(q * e[..., 0, :], q * e[..., 1, :]).sum(-1).amax(3)  # [B, n_q, H, P]
    n = (seen.clamp(min=0) + PAGE - 1) // PAGE  # pages with a key that the query sees
    page = torch.arange(score.shape[-1], device=dev)
    some = n[..., None, None]
    score = score.masked_fill((page < 1) | ((page >= some - 2) & (page < some)), math.inf)
    score = score.masked_fill(page >= some, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=1 << 30)
    order = order.masked_fill(order >= some, 1 << 30).sort(-1).values
    return order.masked_fill(order == 1 << 30, -1).to(torch.int32)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    h, d = case["h_kv"], case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    held = 1.25 * d  # bytes of one token and KV head
    if case["op"] in ("store", "load"):
        rows = sum(rows_of(case)) * h
        if case["op"] == "load":
            return dict(bytes=rows * (held + 2 * d * size), flops=rows * 4.0 * d)
        # written once and read back once, the bounds of the rows' pages beside them
        return dict(bytes=rows * (2 * held + 4 * d * size) + rows / PAGE * 4 * d, flops=rows * 14.0 * d)
    n_q, q_rows = case["n_q"], case["h_q"] * case["batch"] * case["n_q"]
    moved = q_rows * (2 * d * size + 4)
    if case["op"] == "attn":
        tokens = sum(lens_of(case))
        return dict(bytes=moved + tokens * h * held, flops=4.0 * d * tokens * case["h_q"] * n_q)
    pages = sum(-(-n // PAGE) for n in lens_of(case))
    kept = sum(min(n, case["keep"] * PAGE) for n in lens_of(case))
    return dict(bytes=moved + n_q * (pages * h * 4 * d + kept * h * held + case["batch"] * h * case["keep"] * 4),
                flops=n_q * case["h_q"] * (4.0 * d * pages + 4.0 * d * kept))


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d, h = case["d"], case["h_kv"]
    if case["op"] == "store":
        bounds = s["bounds"].double()
        done = []
        for name in ("k", "v"):
            done.append(torch.cat([_held(x) for x in s[name].split(8192)]))
        start = 0
        for i, n in enumerate(s["rows"]):  # the pages' bounds, page by page
            x = done[0][start:start + n].clamp(-BIG, BIG).half().double()
            at = s["first_host"][i]
            while len(x):
                m = min(len(x), PAGE - at % PAGE)
                p = int(s["table"][i, at // PAGE])
                both = torch.stack([x[:m].min(0).values, x[:m].max(0).values], 1)
                if at % PAGE:
                    both = torch.stack([torch.minimum(both[:, 0], bounds[p, :, 0]),
                                        torch.maximum(both[:, 1], bounds[p, :, 1])], 1)
                bounds[p] = both
                x, at = x[m:], at + m
            start += n
        return dict(k=done[0], v=done[1], bounds=bounds)
    if case["op"] == "load":
        k, v = [], []
        for i, n in enumerate(s["rows"]):
            a, c = _cached(s, i, s["first_host"][i], n)
            k.append(a)
            v.append(c)
        return dict(k=torch.cat(k), v=torch.cat(v))
    n_q, g = case["n_q"], case["h_q"] // h
    out = torch.zeros(case["batch"], n_q, case["h_q"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], n_q, case["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens_host"]):
        if not n:
            continue
        k, v = _cached(s, i, 0, n)
        for t in range(n_q):
            m = n - n_q + t + 1
            for j in range(h if m > 0 else 0):
                q = s["q"][i, t, j * g:(j + 1) * g].double()
                kk, vv = k[:m, j], v[:m, j]
                if case["op"] == "sparse":
                    rows = _kept_rows(s, i, j, q, m, case["keep"])
                    kk, vv = kk[rows], vv[rows]
                z = q @ kk.t() * d ** -0.5
                lse[i, t, j * g:(j + 1) * g] = torch.logsumexp(z, -1)
                out[i, t, j * g:(j + 1) * g] = torch.softmax(z, -1) @ vv
    got = dict(out=out, lse=lse)
    if case["op"] == "sparse":
        got["sel"] = None
    return got


def _held(x):
    """The values that rows x are held as.  The definition rounds the zero and the scale to fp16 and the
    difference and the quotient to fp32; the rest is in 64 bits."""
    y = x.double().clamp(-BIG, BIG).reshape(*x.shape[:-1], -1, GROUP)
    low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    zero = low.float().half().double()
    step = ((high - low).float().double() / 15).float().half().double()
    ratio = ((y - zero).float().double() / step.masked_fill(step == 0, 1)).float().double()
    code = ratio.round().clamp(0, 15).masked_fill(step == 0, 0)
    return (zero + step * code).reshape(x.shape)


def _cached(s, i, first, n):
    """K, V float64 [n, H_kv, D] of positions first.. of sequence i, byte by byte out of its pages."""
    d, h = s["case"]["d"], s["case"]["h_kv"]
    ng, half = d // GROUP, 40 * d
    pos = torch.arange(first, first + n, device="cuda")
    page, row = s["table"][i].long()[pos // PAGE], pos % PAGE
    flat = s["pages"].view(-1, 80 * d)
    c = torch.arange(d, device="cuda")
    grp, r = c // GROUP, c % GROUP
    got = []
    for v in (0, 1):
        x = torch.empty(n, h, d, dtype=torch.float64, device="cuda")
        for a in range(0, n, 16384):
            t = row[a:a + 16384, None]
            if not v:  # K: the word of (token, 8-channel run, group), the channel's four bits
                word, bit = (t * 4 + r // 8) * ng + grp, 16 * (r % 2) + 4 * (r % 8 // 2)
                at_scale, at_zero = (t // 2 * ng + grp) * 2 + t % 2, t * ng + grp
            else:  # V: the word of (token pair, 4-channel run, group)
                word, bit = (t // 2 * 8 + r // 4) * ng + grp, 16 * (t % 2) + 4 * (r % 4)
                at_scale = at_zero = (t // 2 * ng + grp) * 2 + t % 2
            at = half * v + 4 * word + bit // 8
            for j in range(h):
                b = flat[page[a:a + 16384] * h + j]
                code = (b.gather(1, at) >> (bit % 8).expand_as(at)) & 15
                hb = b.view(torch.float16)
                scale = hb.gather(1, (half * v + 32 * d) // 2 + at_scale).double()
                zero = hb.gather(1, (half * v + 36 * d) // 2 + at_zero).double()
                x[a:a + 16384, j] = (zero + scale * code.double())
        got.append(x)
    return got


def _kept_rows(s, i, j, q, m, keep):
    """The cache rows of the pages kept for head j's queries q [G, D] of sequence i, which see m keys."""
    n = -(-m // PAGE)
    if n <= keep:
        return torch.arange(m, device="cuda")
    e = s["bounds"][s["table"][i, :n].long(), j].double()  # [n, 2, D]
    score = (q.clamp(min=0) @ e[:, 1].t() + q.clamp(max=0) @ e[:, 0].t()).max(0).values.cpu().tolist()
    forced = {0, n - 2, n - 1}
    rest = sorted((p for p in range(n) if p not in forced), key=lambda p: (-score[p], p))[:keep - len(forced)]
    page = torch.tensor(sorted(forced | set(rest)), device="cuda")
    rows = (page[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
    return rows[rows < m]
