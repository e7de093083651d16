"""Measured cases of the operators that stand between the weight products of a
decode step: block tables and slot maps of a paged key-value cache, the append
to that cache with rotary positions, attention of one to six new tokens over
it, and the norms around a block with its gate and residual scale.

With ``own`` false ``run`` computes the plain forms (elementary torch
operations in 32 bits); with ``own`` true it calls the package.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    """What each case stands for is said beside it."""
    return [
        # one token of a small model early in a chat: latency counts
        attn("attention, 1 request, 700 tokens, q8_0", "q8_0", "f32", 1, 1, 16, 4, 128, 16, 700),
        # one token of a 7B-shaped model deep in a long document
        attn("attention, 1 request, 100003 tokens, f16", "f16", "f32", 1, 1, 28, 4, 128, 32, 100003),
        # a server's decode step over requests of ragged lengths
        attn("attention, 48 requests to 12001, bf16", "bf16", "bf16", 48, 1, 32, 8, 128, 64, 12001),
        # speculative decoding: five rows verified at once over a quantized cache
        attn("attention, verify 5 rows, 24577, q8_0", "q8_0", "f32", 1, 5, 40, 8, 128, 16, 24577),
        # many short requests of a small model with heads of 64
        attn("attention, 160 requests to 2500, f16", "f16", "f16", 160, 1, 14, 2, 64, 16, 2500),
        # the append of one token's keys and values
        append("append, 1 token, f16", "f16", "f32", 1, 16, 4, 128, 128, 1, False, 16, 131000),
        # a prompt's chunk into a quantized cache
        append("append, 8192 tokens, q8_0", "q8_0", "f32", 8192, 28, 4, 128, 128, 1, False, 32, 120000),
        # an image and text prompt: time, height and width positions
        append("append, 4001 tokens, 3 axes, bf16", "bf16", "bf16", 4001, 16, 4, 128, 128, 3, False, 64, 32000),
        # a decode step of 256 requests: one token each, some finished
        tables("block tables, 256 requests decode", 256, 16, 1, 9000),
        # a step that mixes prompts with decode
        tables("block tables, 1000 requests with prompts", 1000, 64, 900, 30000),
        # between two blocks of one token
        norm("norm, 1 row of 1024, f32", "f32", "f32", 1, 1024, "channel"),
        # between two blocks of a prompt, residual stream kept in 32 bits
        norm("norm, 8192 rows of 5120, bf16", "bf16", "f32", 8192, 5120, "channel"),
    ]


def attn(name, cache, q, requests, rows, heads, kv_heads, dim, page, length):
    return named(name, op="attention", cache=cache, q=q, requests=requests, rows=rows, heads=heads,
                 kv_heads=kv_heads, dim=dim, page=page, length=length)


def append(name, cache, x, tokens, heads, kv_heads, dim, rot, axes, interleaved, page, far):
    return named(name, op="append", cache=cache, x=x, tokens=tokens, heads=heads,
                 kv_heads=kv_heads, dim=dim, rot=rot, axes=axes, interleaved=interleaved, page=page,
                 far=far)


def tables(name, requests, page, grow, length):
    return named(name, op="tables", requests=requests, page=page, grow=grow, length=length)


def norm(name, x, residual, rows, width, gate):
    return named(name, op="norm", x=x, residual=residual, rows=rows, width=width, gate=gate)


def named(name, **case):
    return dict(case, name=name) if name else case


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# no drawn attention reads more cache than the largest listed one, no drawn
# append or norm moves more than the listed ones
MOST_CACHE = 48 * 7500 * 8 * 128
MOST_APPEND = 8192 * 36 * 128
MOST_NORM = 8192 * 5120


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "tables", "norm"])
    if op == "attention":
        cache = rng.choice(["f16", "bf16", "q8_0"])
        q = rng.choice(["f32", "f32", {"q8_0": "bf16"}.get(cache, cache)])
        dim = rng.choice([64, 96, 128, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.randint(1, 8)
        rows = rng.choice([1, 1, 1, rng.randint(2, 6)])
        requests = spread(rng, 1, 256)
        most = MOST_CACHE // (requests * kv_heads * dim)
        return attn(None, cache, q, requests, rows, heads, kv_heads, dim,
                    rng.choice([8, 16, 24, 32, 64, 128]), spread(rng, 12, min(most, 131072)))
    if op == "append":
        cache = rng.choice(["f16", "bf16", "q8_0"])
        x = rng.choice(["f32", {"q8_0": "bf16"}.get(cache, cache)])
        dim = rng.choice([64, 96, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.randint(1, 8)
        axes = rng.choice([1, 1, 3])
        rot = dim if rng.random() < 0.75 else dim // 2
        most = MOST_APPEND // ((heads + 2 * kv_heads) * dim)
        return append(None, cache, x, spread(rng, 1, min(most, 16384)), heads, kv_heads, dim, rot,
                      axes, axes == 1 and rng.random() < 0.3, rng.choice([8, 16, 24, 32, 64, 128]),
                      spread(rng, 20000, 1000000))
    if op == "tables":
        return tables(None, spread(rng, 1, 2000), rng.choice([8, 16, 24, 32, 64, 128]),
                      spread(rng, 1, 900), spread(rng, 100, 30000))
    x = rng.choice(["f32", "bf16", "f16"])
    width = rng.choice([896, 1000, 1024, 2047, 2048, 3584, 4096, 5120, 8192, 12345])
    return norm(None, x, rng.choice([x, "f32"]), spread(rng, 1, MOST_NORM // width), width,
                rng.choice(["none", "channel", "token"]))


def lengths(case):
    """The requests' lengths, from the case alone: the first is the longest,
    the others ragged between a tenth of it and all of it."""
    n, most = case["requests"], case["length"]
    rest = np.random.RandomState(n * 7 + most).uniform(0.1, 1.0, n)
    rest[0] = 1.0
    return np.maximum(1, (rest * most).astype(np.int64))


def growth(case):
    """Old and new lengths of a step: most requests grow by one token, some
    start with a prompt, some end and give their pages back."""
    n, most, grow = case["requests"], case["length"], case["grow"]
    r = np.random.RandomState(n * 13 + most)
    old = (np.exp(r.uniform(math.log(2.0), math.log(most), n))).astype(np.int64)
    kind = r.uniform(0, 1, n)
    new = old + 1
    if grow > 1:
        fresh = kind < 0.2
        old[fresh] = 0
        new[fresh] = 1 + (r.uniform(0.1, 1.0, n)[fresh] * (grow - 1)).astype(np.int64)
    new[kind > 0.96] = 0
    return old, new


def pages_of(n, page):
    return -(-n // page)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": case}
    {"attention": prepare_attention, "append": prepare_append, "tables": prepare_tables,
     "norm": prepare_norm}[case["op"]](case, s, g)
    return s


def normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def cache_pages(case, s, g, pages, filled):
    """A layer's cache [pages, kv heads, slots of a page, dim]: values near
    N(0, 1), in Q8_0 as codes and a scale for each 32 of them."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    for name in ("k", "v"):
        if case["cache"] == "q8_0":
            if filled:
                codes = torch.empty(shape, dtype=torch.int8, device=DEV)
                for i in range(0, pages, 8192):  # in pieces: the drawn values are four times as large
                    part = normal(g, codes[i:i + 8192].shape, torch.float16)
                    codes[i:i + 8192] = (part * 42).clamp_(-127, 127).to(torch.int8)
                scale = (0.024 + 0.002 * normal(g, shape[:3] + (shape[3] // 32,))).to(torch.float16)
            else:
                codes = torch.zeros(shape, dtype=torch.int8, device=DEV)
                scale = torch.zeros(shape[:3] + (shape[3] // 32,), dtype=torch.float16, device=DEV)
            s[name], s[name + "_scale"] = codes, scale
        else:
            dtype = DTYPES[case["cache"]]
            s[name] = normal(g, shape, dtype) if filled else torch.zeros(shape, dtype=dtype, device=DEV)
            s[name + "_scale"] = None
    if own:
        import block_quantized_weight_dequant_gb300 as bq
        s["cache"] = bq.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])


def prepare_attention(case, s, g):
    lens = lengths(case)
    need = pages_of(lens, case["page"])
    total, width = int(need.sum()), int(need.max())
    pool = total + 7
    cache_pages(case, s, g, pool, True)
    order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    need_t = torch.from_numpy(need).to(DEV)
    col = torch.arange(width, device=DEV)
    first = torch.cumsum(need_t, 0) - need_t
    at = first[:, None] + col[None, :]
    s["table"] = torch.where(col[None, :] < need_t[:, None], order[at.clamp(max=pool - 1)],
                             torch.full_like(at, -1, dtype=torch.int32))
    s["lens"] = torch.from_numpy(lens).to(DEV).to(torch.int32)
    s["q"] = normal(g, (case["requests"] * case["rows"], case["heads"], case["dim"])).to(DTYPES[case["q"]])


def sections(case):
    """Pairs of each axis: a quarter of them for time, the rest for height
    and width."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [half]
    a = half // 4
    b = (half - a) // 2
    return [a, b, half - a - b]


def prepare_append(case, s, g):
    T, page = case["tokens"], case["page"]
    pool = pages_of(T, page) + 5
    cache_pages(case, s, g, pool, False)
    heads, kv, D = case["heads"], case["kv_heads"], case["dim"]
    # q, k and v are slices of one product's rows, as the fused projection leaves them
    qkv = normal(g, (T, (heads + 2 * kv) * D)).to(DTYPES[case["x"]])
    s["q"] = qkv[:, :heads * D].view(T, heads, D)
    s["kn"] = qkv[:, heads * D:(heads + kv) * D].view(T, kv, D)
    s["vn"] = qkv[:, (heads + kv) * D:].view(T, kv, D)
    order = torch.randperm(pool, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    s["slots"] = order[t // page] * page + t % page
    start = torch.randint(0, case["far"] - T, (1,), generator=g, device=DEV)
    if case["axes"] == 1:
        s["positions"] = (start + t).to(torch.int32)[None]
    else:  # time, height, width of 32 x 32 patches
        s["positions"] = torch.stack([start + t // 1024, start + t // 32 % 32, start + t % 32]).to(torch.int32)
    half = case["rot"] // 2
    freq = 1.0e6 ** (-np.arange(half, dtype=np.float64) * 2 / case["rot"])
    s["freq"] = torch.from_numpy(freq).to(DEV)
    s["axis"] = torch.from_numpy(np.repeat(np.arange(case["axes"]), sections(case))).to(DEV)
    if own:
        import block_quantized_weight_dequant_gb300 as bq
        s["rope"] = bq.Rope(s["freq"], sections=sections(case), interleaved=case["interleaved"])
        s["q_out"] = torch.empty((T, heads, D), dtype=qkv.dtype, device=DEV)


def prepare_tables(case, s, g):
    old, new = growth(case)
    page, n = case["page"], case["requests"]
    held, wanted = pages_of(old, page), pages_of(new, page)
    width = int(max(held.max(), wanted.max())) + 1
    pool = int(held.sum()) + int(np.maximum(wanted - held, 0).sum()) + 11
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    held_t = torch.from_numpy(held).to(DEV)
    col = torch.arange(width, device=DEV)
    at = (torch.cumsum(held_t, 0) - held_t)[:, None] + col[None, :]
    s["table"] = torch.where(col[None, :] < held_t[:, None], order[at.clamp(max=pool - 1)],
                             torch.full_like(at, -1, dtype=torch.int32))
    used = int(held.sum())
    s["free"] = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
    s["free"][:pool - used] = order[used:]
    s["free_count"] = torch.tensor([pool - used], dtype=torch.int32, device=DEV)
    s["old"] = torch.from_numpy(old).to(DEV).to(torch.int32)
    s["new"] = torch.from_numpy(new).to(DEV).to(torch.int32)
    room = int(np.maximum(new - old, 0).sum()) + 3  # a few rows behind the last token
    s["slots"] = torch.zeros(room, dtype=torch.int64, device=DEV)
    s["positions"] = torch.zeros(room, dtype=torch.int32, device=DEV)
    s["starts"] = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    s["lens_out"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    s["count_out"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    s["refused"] = torch.zeros(1, dtype=torch.int32, device=DEV)


def prepare_norm(case, s, g):
    T, H = case["rows"], case["width"]
    x, r = DTYPES[case["x"]], DTYPES[case["residual"]]
    s["y"] = (0.5 * normal(g, (T, H))).to(x)
    s["h"] = normal(g, (T, H)).to(r)
    s["post"] = 1 + 0.1 * normal(g, (H,))
    s["pre"] = 1 + 0.1 * normal(g, (H,))
    s["gate"] = {"none": lambda: None, "channel": lambda: (0.3 * normal(g, (H,))).to(x),
                 "token": lambda: (0.3 * normal(g, (T, H))).to(x)}[case["gate"]]()
    s["alpha"], s["beta"], s["eps"] = 0.9375, 1.25, 1e-6
    s["h_out"], s["x_out"] = torch.empty_like(s["h"]), torch.empty_like(s["y"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import block_quantized_weight_dequant_gb300 as bq
        if op == "attention":
            return bq.paged_attention(s["cache"], s["q"], s["table"], s["lens"], rows=s["case"]["rows"])
        if op == "append":
            bq.kv_append(s["cache"], s["kn"], s["vn"], s["slots"], q=s["q"], q_out=s["q_out"],
                         rope=s["rope"], positions=s["positions"])
            return [s["q_out"]] + held_values(s)
        if op == "tables":
            bq.kv_block_tables(s["old"], s["new"], s["table"], s["free"], s["free_count"],
                               s["case"]["page"], s["slots"], s["positions"], s["starts"],
                               lens_out=s["lens_out"], free_count_out=s["count_out"], refused=s["refused"])
            return [s["table"], s["free"], s["slots"], s["positions"], s["starts"], s["lens_out"],
                    s["count_out"], s["refused"]]
        return list(bq.sandwich_norm(s["y"], s["h"], pre_gain=s["pre"], post_gain=s["post"], gate=s["gate"],
                                     alpha=s["alpha"], beta=s["beta"], eps=s["eps"],
                                     h_out=s["h_out"], x_out=s["x_out"]))
    return {"attention": plain_attention, "append": plain_append, "tables": plain_tables,
            "norm": plain_norm}[op](s)


def held_values(s):
    """The cache itself; of a quantized one the values its blocks stand for."""
    if s["case"]["cache"] != "q8_0":
        return [s["k"], s["v"]]
    return [(codes.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
            for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))]


def gathered(values, scale, table):
    """[requests, kv heads, positions, dim] in 32 bits."""
    x = values[table].float()
    if scale is not None:
        x = (x.unflatten(-1, (-1, 32)) * scale[table].float()[..., None]).flatten(-2)
    return x.transpose(1, 2).flatten(2, 3)


def plain_attention(s):
    c = s["case"]
    B, R, H, KV, D = c["requests"], c["rows"], c["heads"], c["kv_heads"], c["dim"]
    table = s["table"].clamp(min=0).long()
    k = gathered(s["k"], s["k_scale"], table)
    q = s["q"].float().view(B, R, KV, H // KV, D).permute(0, 2, 1, 3, 4).reshape(B, KV, R * (H // KV), D)
    scores = torch.matmul(q, k.transpose(2, 3)).div_(math.sqrt(D)).unflatten(2, (R, H // KV))
    seen = s["lens"].long()[:, None] - R + 1 + torch.arange(R, device=DEV)
    hidden = torch.arange(k.shape[2], device=DEV) >= seen[:, :, None]
    del k
    scores.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = gathered(s["v"], s["v_scale"], table)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (R, H // KV)) / total
    o = torch.where((seen <= 0)[:, None, :, None, None], torch.zeros_like(o), o)
    return o.permute(0, 2, 1, 3, 4).reshape(B * R, H, D).to(s["q"].dtype)


def turned(x, cos, sin, rot, interleaved):
    """The first `rot` values of each head turned by their angles."""
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        e, o = a[..., 0::2], a[..., 1::2]
        a = torch.stack([e * cos - o * sin, o * cos + e * sin], -1).flatten(-2)
    else:
        e, o = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat([e * cos - o * sin, o * cos + e * sin], -1)
    return torch.cat([a, rest], -1)


def plain_append(s):
    c = s["case"]
    # angles of far positions, and values next to a rounding border, in 64 bits
    angle = s["positions"].double()[s["axis"]].t() * s["freq"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    q = turned(s["q"].double(), cos, sin, c["rot"], c["interleaved"])
    k = turned(s["kn"].double(), cos, sin, c["rot"], c["interleaved"])
    page, slot = s["slots"] // c["page"], s["slots"] % c["page"]
    for name, x in (("k", k), ("v", s["vn"])):
        if c["cache"] == "q8_0":
            x = x.float().unflatten(-1, (-1, 32))
            d = (x.abs().amax(-1) / 127).to(torch.float16)
            f = d.float()[..., None]
            r = x / torch.where(f == 0, torch.ones_like(f), f)
            r = torch.sign(r) * torch.floor(r.abs() + 0.5)  # halves away from zero
            r = torch.where(f == 0, torch.zeros_like(r), r).clamp(-127, 127)
            s[name][page, :, slot] = r.flatten(-2).to(torch.int8)
            s[name + "_scale"][page, :, slot] = d
        else:
            s[name][page, :, slot] = x.to(s[name].dtype)
    return [q.to(s["q"].dtype)] + held_values(s)


def plain_tables(s):
    page = s["case"]["page"]
    old, new = s["old"].long(), s["new"].long()
    table, n = s["table"], old.numel()
    held, wanted = (old + page - 1) // page, (new + page - 1) // page
    freed, asked = (held - wanted).clamp(min=0), (wanted - held).clamp(min=0)
    tokens = (new - old).clamp(min=0)
    ends = torch.cumsum(tokens, 0)
    count = s["free_count"].long()
    freed_ends, asked_ends = torch.cumsum(freed, 0), torch.cumsum(asked, 0)
    served = ((asked == 0) | (asked_ends <= count + freed_ends[-1])) & ((tokens == 0) | (ends <= s["slots"].numel()))
    given = torch.where(served, asked, 0).sum()
    # the stack of free pages: the released ones on top, in the requests' order
    col = torch.arange(table.shape[1], device=DEV)
    leaving = (col >= wanted[:, None]) & (col < held[:, None])
    free = s["free"].clone()
    place = torch.where(leaving, count + (freed_ends - freed)[:, None] + col - wanted[:, None], free.numel())
    free = torch.cat([free, free.new_zeros(1)]).index_put((place.flatten().clamp(max=free.numel()),), table.flatten())[:-1]
    top = count + freed_ends[-1]
    coming = (col >= held[:, None]) & (col < wanted[:, None]) & served[:, None]
    pick = top - 1 - ((asked_ends - asked)[:, None] + col - held[:, None])
    table.copy_(torch.where(coming, free[pick.clamp(0, free.numel() - 1)], table))
    left = top - given
    # what is above the stack's new top is left as it was
    slot = torch.arange(free.numel(), device=DEV)
    free = torch.where(slot < left, free, s["free"])
    t = torch.arange(s["slots"].numel(), device=DEV)
    request = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    live = (t < ends[-1]) & served[request]
    position = old[request] + t - (ends - tokens)[request]
    row = table[request, (position // page).clamp(0, table.shape[1] - 1)].long()
    s["slots"].copy_(torch.where(live, row * page + position % page, -1))
    s["positions"].copy_(torch.where(live, position, 0))
    s["free"].copy_(free)
    starts = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    return [table, s["free"], s["slots"], s["positions"], starts, torch.where(served, new, old).to(torch.int32),
            left.to(torch.int32), (~served).sum()[None].to(torch.int32)]


def plain_norm(s):
    b = s["y"].float()
    b = b * torch.rsqrt((b * b).mean(-1, keepdim=True) + s["eps"]) * s["post"]
    if s["gate"] is not None:
        b = b * s["gate"].float()
    h = s["alpha"] * s["h"].float() + s["beta"] * b
    x = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["pre"]
    return [h.to(s["h"].dtype), x.to(s["y"].dtype)]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def size_of(name):
    return {"f32": 4, "f16": 2, "bf16": 2}[name]


def cache_bytes(case, values):
    return values * (34 / 32 if case["cache"] == "q8_0" else 2)


def work(case):
    if case["op"] == "attention":
        lens, R = lengths(case), case["rows"]
        tokens, pages = int(lens.sum()), int(pages_of(lens, case["page"]).sum())
        q = case["requests"] * R * case["heads"] * case["dim"]
        seen = sum(int(np.maximum(lens - R + r + 1, 0).sum()) for r in range(R))
        return {"bytes": cache_bytes(case, 2 * tokens * case["kv_heads"] * case["dim"])
                + 2 * q * size_of(case["q"]) + 4 * pages + 4 * case["requests"],
                "flops": 4.0 * seen * case["heads"] * case["dim"]}
    if case["op"] == "append":
        T, D, x = case["tokens"], case["dim"], size_of(case["x"])
        return {"bytes": T * D * (case["heads"] * 2 * x + 2 * case["kv_heads"] * x)
                + cache_bytes(case, 2 * T * case["kv_heads"] * D) + T * (8 + 4 * case["axes"]),
                "flops": 3.0 * T * case["rot"] * (case["heads"] + case["kv_heads"])}
    if case["op"] == "tables":
        old, new = growth(case)
        tokens = int(np.maximum(new - old, 0).sum())
        moved = int(np.abs(pages_of(old, case["page"]) - pages_of(new, case["page"])).sum())
        return {"bytes": 16.0 * case["requests"] + 8 * moved + 12 * tokens, "flops": 0.0}
    n = case["rows"] * case["width"]
    x, r = size_of(case["x"]), size_of(case["residual"])
    gate = {"none": 0, "channel": case["width"], "token": n}[case["gate"]]
    return {"bytes": 2 * n * x + 2 * n * r + gate * x + 8 * case["width"], "flops": 10.0 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": exact_attention, "append": exact_append, "tables": exact_tables,
            "norm": exact_norm}[case["op"]](case, s)


def exact_attention(case, s):
    page, R, D = case["page"], case["rows"], case["dim"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()

    def history(name, ids, h, n):
        x = s[name][ids, h].reshape(-1, D)[:n].double()
        if s[name + "_scale"] is not None:
            d = s[name + "_scale"][ids, h].reshape(-1, D // 32)[:n].double()
            x = x * d.repeat_interleave(32, dim=1)
        return x

    for b, n in enumerate(lens):
        ids = torch.from_numpy(table[b, :-(-n // page)].astype(np.int64)).to(DEV)
        for h in range(case["kv_heads"]):
            k, v = history("k", ids, h, n), history("v", ids, h, n)
            for r in range(R):
                m = n - R + r + 1
                if m > 0:
                    q = s["q"][b * R + r, h * group:(h + 1) * group].double()
                    out[b * R + r, h * group:(h + 1) * group] = torch.softmax(q @ k[:m].t() * D ** -0.5, -1) @ v[:m]
    return out


def exact_append(case, s):
    # the kept values of a quantized cache are whole multiples of their scale: only q and, in 16 bits, the
    # rotated keys have a value in 64 bits
    T, rot = case["tokens"], case["rot"]
    half = rot // 2
    angle = torch.empty((T, half), dtype=torch.float64, device=DEV)
    for p in range(half):
        angle[:, p] = s["positions"][int(s["axis"][p])].double() * float(s["freq"][p])
    both = []
    for x in (s["q"], s["kn"]):
        z = x.double().clone()
        if case["interleaved"]:
            pair = torch.view_as_complex(x[..., :rot].double().reshape(x.shape[:2] + (half, 2)).contiguous())
        else:
            pair = torch.complex(x[..., :half].double(), x[..., half:rot].double())
        pair = pair * torch.polar(torch.ones_like(angle), angle)[:, None]
        if case["interleaved"]:
            z[..., :rot] = torch.view_as_real(pair).flatten(-2)
        else:
            z[..., :half], z[..., half:rot] = pair.real, pair.imag
        both.append(z)
    if case["cache"] == "q8_0":
        return [both[0], None, None]
    kept = []
    for name, x in (("k", both[1]), ("v", s["vn"].double())):
        pages, kv, page, D = s[name].shape
        flat = torch.zeros((pages * page, kv, D), dtype=torch.float64, device=DEV)
        flat[s["slots"]] = x
        kept.append(flat.view(pages, page, kv, D).transpose(1, 2).contiguous())
    return [both[0]] + kept


def exact_tables(case, s):
    """The step told request by request on the host."""
    page = case["page"]
    old, new = s["old"].tolist(), s["new"].tolist()
    table = s["table"].cpu().numpy().copy()
    count = int(s["free_count"])
    free = s["free"].cpu().numpy().copy()
    stack = free[:count].tolist()
    for b, (a, z) in enumerate(zip(old, new)):
        stack += table[b, -(-z // page):-(-a // page)].tolist() if z < a else []
    slots = np.full(s["slots"].numel(), -1, np.int64)
    positions = np.zeros(slots.size, np.int32)
    starts, lens = [0], []
    for b, (a, z) in enumerate(zip(old, new)):  # the prepared steps have pages and rows enough for all
        for j in range(-(-a // page), -(-z // page)):
            table[b, j] = stack.pop()
        where = np.arange(a, z)
        slots[starts[-1]:starts[-1] + where.size] = table[b, where // page].astype(np.int64) * page + where % page
        positions[starts[-1]:starts[-1] + where.size] = where
        starts.append(starts[-1] + where.size)
        lens.append(z)
    free[:len(stack)] = stack
    i32 = np.int32
    return [table, free, slots, positions, np.array(starts, i32), np.array(lens, i32),
            np.array([len(stack)], i32), np.array([0], i32)]


def exact_norm(case, s):
    y, h = s["y"].double(), s["h"].double()
    g = 1.0 if s["gate"] is None else s["gate"].double()
    h = s["alpha"] * h + s["beta"] * g * (y / (y.square().mean(1, keepdim=True) + s["eps"]).sqrt() * s["post"].double())
    return [h, h / (h.square().mean(1, keepdim=True) + s["eps"]).sqrt() * s["pre"].double()]
