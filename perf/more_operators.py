"""Measured cases of what requests that share their beginning need of a paged
key-value cache: keys and queries normed per head, turned and appended in one
pass; attention of a batch over a long prefix that its requests hold in common;
and the pages themselves: forking, freeing, copying and compacting.

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
        # one token of a small model whose layers norm queries and keys: latency counts
        append("normed append 1 token f16", "f16", "f32", 1, 16, 8, 128, 128, 1, False, 16, 131000),
        # a prompt's chunk
        append("normed append 8192 tokens f16", "f16", "f32", 8192, 28, 4, 128, 128, 1, False, 32, 120000),
        # four answers to one short prompt
        prefix("prefix attention 4 requests 700 shared f16", "f16", "f32", 4, 1, 1, 16, 8, 128, 16, 700, 90),
        # a server whose requests all begin with the same long document
        prefix("prefix attention 96 requests 32801 shared bf16", "bf16", "bf16", 96, 1, 1, 32, 8, 128, 64, 32801, 400),
        # many requests of a small model under three system prompts
        prefix("prefix attention 200 requests 3 groups of 9001 f16", "f16", "f16", 200, 3, 1, 14, 2, 64, 16, 9001, 300),
        # samples of one long conversation over a quantized cache
        prefix("prefix attention 16 requests 30011 shared q8_0", "q8_0", "f32", 16, 1, 1, 16, 8, 128, 32, 30011, 500),
        # a prompt forked into fifteen samples beside a few other requests
        tables("page tables 24 requests 15 forks", 24, 16, 15, 1, 3000),
        # a busy server's step: prompts, decode, forks, rollbacks, ended requests
        tables("page tables 1000 requests 120 forks", 1000, 16, 120, 200, 20000),
        # the pages that a few forks of one step must have for themselves, in every layer
        copy("page copy 6 pages of 28 layers f16", "f16", 28, 64, 6, 8, 128, 16),
        # what a compaction moves
        copy("page copy 200 pages of 28 layers bf16", "bf16", 28, 450, 200, 8, 128, 16),
        # a small server's pool before it gives memory back
        compact("compaction 3000 pages", 40, 16, 3000, 0.4),
        # a large one's
        compact("compaction 200000 pages", 600, 16, 200000, 0.5),
    ]


def append(name, cache, x, tokens, heads, kv_heads, dim, rot, axes, interleaved, page, far):
    return named(name, op="append", cache=cache, x=x, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                 axes=axes, interleaved=interleaved, page=page, far=far)


def prefix(name, cache, q, requests, groups, rows, heads, kv_heads, dim, page, shared, alone):
    return named(name, op="prefix", cache=cache, q=q, requests=requests, groups=groups, rows=rows, heads=heads,
                 kv_heads=kv_heads, dim=dim, page=page, shared=shared, alone=alone)


def tables(name, requests, page, forks, grow, length):
    return named(name, op="tables", requests=requests, page=page, forks=forks, grow=grow, length=length)


def copy(name, cache, layers, pool, moves, kv_heads, dim, page):
    return named(name, op="copy", cache=cache, layers=layers, pool=pool, moves=moves, kv_heads=kv_heads, dim=dim,
                 page=page)


def compact(name, requests, page, pool, used):
    return named(name, op="compact", requests=requests, page=page, pool=pool, used=used)


def named(name, **case):
    return dict(case, name=name) if name else case


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# no drawn case costs more than the largest listed one of its operator
MOST_APPEND = 8192 * 36 * 128
MOST_PREFIX = 96 * 32801 * 32 * 128  # products of a query with a shared position
MOST_CACHE = 8 * 128 * (32801 + 96 * 400)  # cached values of all requests
MOST_COPY = 200 * 28 * 8 * 128 * 16
MOST_POOL = 450 * 28 * 8 * 128 * 16


def draw(rng):
    op = rng.choice(["append", "prefix", "prefix", "prefix", "tables", "copy", "compact"])
    if op == "append":
        cache = rng.choice(["f16", "bf16", "q8_0"])
        x = rng.choice(["f32", {"q8_0": "bf16"}.get(cache, cache)])
        dim = rng.choice([64, 96, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.randint(1, 8)
        axes = rng.choice([1, 1, 3])
        rot = dim if rng.random() < 0.75 else dim // 2
        most = MOST_APPEND // ((heads + 2 * kv_heads) * dim)
        return append(None, cache, x, spread(rng, 1, min(most, 16384)), heads, kv_heads, dim, rot, axes,
                      axes == 1 and rng.random() < 0.3, rng.choice([8, 16, 24, 32, 64, 128]), spread(rng, 20000, 1000000))
    if op == "prefix":
        cache = rng.choice(["f16", "f16", "bf16", "bf16", "q8_0"])
        q = rng.choice(["f32", {"q8_0": "bf16"}.get(cache, cache)])
        dim = rng.choice([64, 96, 128, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.randint(1, 8)
        rows = rng.choice([1, 1, 1, rng.randint(2, 6)])
        requests = spread(rng, 2, 256)
        groups = 1 if requests < 6 else rng.choice([1, 1, rng.randint(2, 3)])
        most = min(MOST_PREFIX // (requests * rows * heads * dim), MOST_CACHE // (kv_heads * dim) // (2 * groups))
        alone = min(spread(rng, 2, 1500), MOST_CACHE // (kv_heads * dim) // (2 * requests))
        return prefix(None, cache, q, requests, groups, rows, heads, kv_heads, dim, rng.choice([8, 16, 24, 32, 64, 128]),
                      spread(rng, 40, max(41, min(most, 65536))), max(rows, alone))
    if op == "tables":
        requests = spread(rng, 2, 1000)
        return tables(None, requests, rng.choice([16, 24, 32, 64, 128]), spread(rng, 1, min(120, max(1, requests // 2))),
                      spread(rng, 1, 200), spread(rng, 100, 20000))
    if op == "copy":
        kv_heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256]), rng.choice([8, 16, 24, 32, 64])
        layers = spread(rng, 1, 64)
        one = layers * kv_heads * dim * page
        moves = spread(rng, 1, min(400, MOST_COPY // one))
        return copy(None, rng.choice(["f16", "bf16"]), layers, min(2 * moves + spread(rng, 1, 60), MOST_POOL // one),
                    moves, kv_heads, dim, page)
    requests = spread(rng, 1, 600)
    return compact(None, requests, rng.choice([8, 16, 24, 32, 64]), spread(rng, 40 * requests, 200000),
                   rng.uniform(0.05, 0.95))


def pages_of(n, page):
    return -(-n // page)


def group_sizes(case):
    """Requests of each group and the positions that they share: the first
    group is the one of the full length."""
    n, g = case["requests"], case["groups"]
    each = [n // g + (i < n % g) for i in range(g)]
    return [(m, max(1, case["shared"] - i * (case["shared"] // 5))) for i, m in enumerate(each)]


def lengths(case):
    """The requests' lengths, from the case alone: the shared part, then ragged
    parts of their own; the last of eight or more requests has ended."""
    r = np.random.RandomState(case["requests"] * 7 + case["shared"])
    alone = case["rows"] + (r.uniform(0.0, 1.0, case["requests"]) * (case["alone"] - case["rows"] + 1)).astype(np.int64)
    shared = np.repeat([s for _, s in group_sizes(case)], [m for m, _ in group_sizes(case)])
    lens = shared + np.minimum(alone, case["alone"])
    if case["requests"] >= 8:
        lens[-1] = 0
    return lens, shared


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": case}
    {"append": prepare_append, "prefix": prepare_prefix, "tables": prepare_tables, "copy": prepare_copy,
     "compact": prepare_compact}[case["op"]](case, s, g)
    return s


def normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def cache_pages(case, s, g, pages, filled):
    """A layer's cache [pages, kv heads, slots of a page, dim]: values near
    N(0, 1), in Q8_0 as codes and a scale for each 32 of them."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    for name in ("k", "v"):
        if case["cache"] == "q8_0":
            codes = torch.zeros(shape, dtype=torch.int8, device=DEV)
            scale = torch.zeros(shape[:3] + (shape[3] // 32,), dtype=torch.float16, device=DEV)
            if filled:
                codes = (normal(g, shape, torch.float16) * 42).clamp_(-127, 127).to(torch.int8)
                scale = (0.024 + 0.002 * normal(g, scale.shape)).to(torch.float16)
            s[name], s[name + "_scale"] = codes, scale
        else:
            dtype = DTYPES[case["cache"]]
            s[name] = normal(g, shape, dtype) if filled else torch.zeros(shape, dtype=dtype, device=DEV)
            s[name + "_scale"] = None
    if own:
        import block_quantized_weight_dequant_gb300 as bq
        s["cache"] = bq.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])


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
    qkv = (0.7 * normal(g, (T, (heads + 2 * kv) * D))).to(DTYPES[case["x"]])
    s["q"] = qkv[:, :heads * D].view(T, heads, D)
    s["kn"] = qkv[:, heads * D:(heads + kv) * D].view(T, kv, D)
    s["vn"] = qkv[:, (heads + kv) * D:].view(T, kv, D)
    s["q_gain"] = 1 + 0.2 * normal(g, (D,))
    s["k_gain"] = 1 + 0.2 * normal(g, (D,))
    s["eps"] = 1e-6
    order = torch.randperm(pool, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    s["slots"] = order[t // page] * page + t % page
    start = torch.randint(0, case["far"] - T, (1,), generator=g, device=DEV)
    if case["axes"] == 1:
        s["positions"] = (start + t).to(torch.int32)[None]
    else:  # time, height, width of 32 x 32 patches
        s["positions"] = torch.stack([start + t // 1024, start + t // 32 % 32, start + t % 32]).to(torch.int32)
    freq = 1.0e6 ** (-np.arange(case["rot"] // 2, dtype=np.float64) * 2 / case["rot"])
    s["freq"] = torch.from_numpy(freq).to(DEV)
    s["axis"] = torch.from_numpy(np.repeat(np.arange(case["axes"]), sections(case))).to(DEV)
    if own:
        import block_quantized_weight_dequant_gb300 as bq
        s["rope"] = bq.Rope(s["freq"], sections=sections(case), interleaved=case["interleaved"])
        s["q_out"] = torch.empty((T, heads, D), dtype=qkv.dtype, device=DEV)


def prepare_prefix(case, s, g):
    page, n = case["page"], case["requests"]
    lens, shared = lengths(case)
    common = [m // page for m in shared]  # whole pages that a request has in common with its group
    need = pages_of(lens, page)
    first = np.cumsum([0] + [m for m, _ in group_sizes(case)])[:-1]
    heads_of = np.repeat(first, [m for m, _ in group_sizes(case)])
    width = int(need.max())
    total = int(sum(common[f] for f in first) + sum(max(0, need[b] - common[b]) for b in range(n)))
    pool = total + 7
    cache_pages(case, s, g, pool, True)
    order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).to(torch.int32).cpu().numpy()
    table = np.full((n, width), -1, np.int32)
    at = 0
    for b in range(n):
        if b in first:
            table[b, :common[b]] = order[at:at + common[b]]
            at += common[b]
        if lens[b]:
            table[b, :common[b]] = table[heads_of[b], :common[b]]
            table[b, common[b]:need[b]] = order[at:at + need[b] - common[b]]
            at += need[b] - common[b]
    s["table"] = torch.from_numpy(table).to(DEV)
    s["lens"] = torch.from_numpy(lens).to(DEV).to(torch.int32)
    s["groups"] = group_sizes(case)
    # the shared part is the same in every request: of a page that each has for itself, too
    for b in range(n):
        rest = int(shared[b]) - int(common[b]) * page
        if lens[b] and rest and b not in first:
            to, of = int(table[b, common[b]]), int(table[heads_of[b], common[b]])
            for name in ("k", "v", "k_scale", "v_scale"):
                if s[name] is not None:
                    s[name][to, :, :rest] = s[name][of, :, :rest]
    s["q"] = normal(g, (n * case["rows"], case["heads"], case["dim"])).to(DTYPES[case["q"]])


def holdings(case):
    """A server's requests before and after a step: (old lengths, new lengths,
    parents, pages of each request as indices of a list, how many pages)."""
    n, page = case["requests"], case["page"]
    r = np.random.RandomState(n * 13 + case["length"])
    forks = min(case["forks"], n - 1)
    old = np.exp(r.uniform(math.log(2.0), math.log(case["length"]), n)).astype(np.int64)
    old[0] = case["length"]
    kind = r.uniform(0, 1, n)
    child = np.zeros(n, bool)
    child[1 + r.permutation(n - 1)[:forks]] = True
    fresh = ~child & (kind < 0.1) & (case["grow"] > 1)
    fresh[0] = False
    old[child | fresh] = 0
    parents = np.full(n, -1, np.int64)
    grown = np.flatnonzero(old > 0)
    parents[child] = np.where(r.uniform(0, 1, forks) < 0.5, 0, grown[r.randint(0, grown.size, forks)])
    new = old + 1
    new[fresh] = 1 + r.randint(0, case["grow"], int(fresh.sum()))
    new[child] = np.maximum(1, old[parents[child]] + r.randint(-1, 2, forks) * r.randint(0, 5, forks))
    back = ~child & ~fresh & (kind > 0.85) & (kind < 0.95)
    new[back] = np.maximum(0, old[back] - r.randint(0, 3 * page, int(back.sum())))
    ended = ~child & ~fresh & (kind > 0.95)
    ended[0] = False
    new[ended] = 0
    # pages: some requests came from an earlier fork and hold another's first pages too
    rows, count = [], 0
    like = r.uniform(0, 1, n)
    for b in range(n):
        need = int(pages_of(old[b], page))
        row = np.empty(0, np.int64)
        if b and like[b] < 0.35:
            row = rows[r.randint(0, b)][:need]
        row = np.concatenate([row, np.arange(count, count + need - row.size)])
        count = max(count, int(row.max()) + 1) if need else count
        rows.append(row)
    return old, new, parents, rows, count


def state_of(s, pool, pages, rows, width, order):
    """refs, the stack of free pages and the table in one buffer, so that one copy sets the step's start."""
    n = len(rows)
    table = np.full((n, width), -1, np.int32)
    refs = np.zeros(pool, np.int32)
    for b, row in enumerate(rows):
        table[b, :row.size] = order[row]
        refs[order[row]] += 1
    free = np.full(pool, -1, np.int32)
    free[:pool - pages] = order[pages:]
    s["start"] = torch.from_numpy(np.concatenate([refs, free, table.ravel()]).astype(np.int32)).to(DEV)
    s["state"] = s["start"].clone()
    s["refs"], s["free"] = s["state"][:pool], s["state"][pool:2 * pool]
    s["table"] = s["state"][2 * pool:].view(n, width)
    s["free_count"] = torch.tensor([pool - pages], dtype=torch.int32, device=DEV)
    s["count_out"] = torch.zeros(1, dtype=torch.int32, device=DEV)


def shuffled(g, pool):
    return torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).cpu().numpy()


def prepare_tables(case, s, g):
    old, new, parents, rows, used = holdings(case)
    page, n = case["page"], case["requests"]
    width = int(max(pages_of(old, page).max(), pages_of(new, page).max())) + 1
    asked = np.maximum(pages_of(new, page) - np.where(parents >= 0, 0, pages_of(old, page)), 0).sum() + n
    pool = used + int(asked) + 11
    state_of(s, pool, used, rows, width, shuffled(g, pool))
    for name, x in (("old", old), ("new", new), ("parents", parents)):
        s[name] = torch.from_numpy(x).to(DEV).to(torch.int32)
    base = np.where(parents >= 0, np.minimum(old[parents], new), old)
    room = int(np.maximum(new - base, 0).sum()) + 3  # a few rows behind the last token
    i32 = dict(dtype=torch.int32, device=DEV)
    s["slots"] = torch.zeros(room, dtype=torch.int64, device=DEV)
    s["positions"], s["starts"] = torch.zeros(room, **i32), torch.zeros(n + 1, **i32)
    s["lens_out"], s["refused"] = torch.zeros(n, **i32), torch.zeros(1, **i32)
    s["copy_src"], s["copy_dst"], s["copy_count"] = torch.zeros(n, **i32), torch.zeros(n, **i32), torch.zeros(1, **i32)


def prepare_copy(case, s, g):
    shape = (case["pool"], case["kv_heads"], case["page"], case["dim"])
    s["layers"] = [(normal(g, shape, DTYPES[case["cache"]]), normal(g, shape, DTYPES[case["cache"]]))
                   for _ in range(case["layers"])]
    order = torch.randperm(case["pool"], generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    m = case["moves"]
    s["src"], s["dst"] = order[:m].contiguous(), order[m:2 * m].contiguous()
    if own:
        import block_quantized_weight_dequant_gb300 as bq
        s["caches"] = [bq.PagedKVCache(k, v) for k, v in s["layers"]]


def prepare_compact(case, s, g):
    """Requests of ragged lengths, their pages spread over the pool."""
    n, page, pool = case["requests"], case["page"], case["pool"]
    r = np.random.RandomState(n * 5 + pool)
    part = r.uniform(0.2, 1.0, n)
    need = np.maximum(1, (part / part.sum() * case["used"] * pool).astype(np.int64))
    lens = need * page - r.randint(0, page, n)
    rows, count = [], 0
    for b in range(n):
        held = rows[b - 1][:int(need[b]) // 3] if b % 4 == 3 else np.empty(0, np.int64)  # a fork of the one before
        row = np.concatenate([held, np.arange(count, count + need[b] - held.size)])
        count += int(need[b] - held.size)
        rows.append(row)
    state_of(s, pool, count, rows, int(need.max()) + 1, shuffled(g, pool))
    s["lens"] = torch.from_numpy(lens).to(DEV).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=DEV)
    room = max(1, pool // 2)
    s["copy_src"], s["copy_dst"], s["copy_count"] = torch.zeros(room, **i32), torch.zeros(room, **i32), torch.zeros(1, **i32)
    s["moved"] = torch.zeros(pool, **i32)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op, page = s["case"]["op"], s["case"].get("page")
    if op in ("tables", "compact"):
        s["state"].copy_(s["start"])  # the step is made in place: each pass starts from the same state
    if not own:
        return {"append": plain_append, "prefix": plain_prefix, "tables": plain_tables, "copy": plain_copy,
                "compact": plain_compact}[op](s)
    import block_quantized_weight_dequant_gb300 as bq
    if op == "append":
        bq.kv_append(s["cache"], s["kn"], s["vn"], s["slots"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                     positions=s["positions"], q_norm=s["q_gain"], k_norm=s["k_gain"], eps=s["eps"])
        return [s["q_out"]] + held_values(s)
    if op == "prefix":
        return bq.paged_prefix_attention(s["cache"], s["q"], s["table"], s["lens"], s["groups"], rows=s["case"]["rows"])
    if op == "tables":
        bq.kv_shared_tables(s["old"], s["new"], s["table"], s["free"], s["free_count"], s["refs"], page, s["slots"],
                            s["positions"], s["starts"], s["copy_src"], s["copy_dst"], s["copy_count"],
                            parents=s["parents"], lens_out=s["lens_out"], free_count_out=s["count_out"],
                            refused=s["refused"])
        return [s["table"], s["free"], s["refs"], s["slots"], s["positions"], s["starts"], s["lens_out"],
                s["count_out"], s["refused"], s["copy_src"], s["copy_dst"], s["copy_count"]]
    if op == "copy":
        bq.kv_copy_pages(s["caches"], s["src"], s["dst"])
        return [t for layer in s["layers"] for t in layer]
    bq.kv_compact(s["lens"], s["table"], s["free"], s["free_count"], s["refs"], page, s["copy_src"], s["copy_dst"],
                  s["copy_count"], s["moved"], free_count_out=s["count_out"])
    return [s["table"], s["free"], s["refs"], s["count_out"], s["copy_src"], s["copy_dst"], s["copy_count"], s["moved"]]


def held_values(s):
    """The cache itself; of a quantized one the values its blocks stand for."""
    if s["case"]["cache"] != "q8_0":
        return [s["k"], s["v"]]
    return [(codes.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
            for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))]


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

    def normed(x, gain):
        x = x.double()
        return turned(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * gain.double(), cos, sin, c["rot"],
                      c["interleaved"])

    q, k = normed(s["q"], s["q_gain"]), normed(s["kn"], s["k_gain"])
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


def gathered(values, scale, table, head):
    """[..., positions, dim] of one head in 32 bits, for tables [..., pages]."""
    x = values[:, head][table].float()
    if scale is not None:
        x = (x.unflatten(-1, (-1, 32)) * scale[:, head][table].float()[..., None]).flatten(-2)
    return x.flatten(-3, -2)


def plain_prefix(s):
    c = s["case"]
    R, H, KV, D, page = c["rows"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    G = H // KV
    out = torch.empty(s["q"].shape, dtype=torch.float32, device=DEV)
    first = 0
    for n, shared in s["groups"]:
        table = s["table"][first:first + n].clamp(min=0).long()
        lens = s["lens"][first:first + n].long()
        pre = table[0, :pages_of(shared, page)]
        after = table[:, shared // page:]  # the pages with positions behind the shared ones
        col = shared // page * page + torch.arange(after.shape[1] * page, device=DEV)
        seen = lens[:, None] - R + 1 + torch.arange(R, device=DEV)  # [n, R]
        hidden = (col >= seen[:, :, None]) | (col < shared)
        empty = (seen <= 0).view(n, R, 1).expand(n, R, G).reshape(n * R * G, 1)
        for h in range(KV):
            q = s["q"][first * R:(first + n) * R, h * G:(h + 1) * G].float() / math.sqrt(D)
            a = q.reshape(n * R * G, D) @ gathered(s["k"], s["k_scale"], pre, h)[:shared].t()
            b = q.reshape(n, R * G, D) @ gathered(s["k"], s["k_scale"], after, h).transpose(1, 2)
            b = b.view(n, R, G, -1).masked_fill_(hidden[:, :, None], -math.inf).view(n * R * G, -1)
            top = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
            a, b = a.sub_(top).exp_(), b.sub_(top).exp_()
            total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
            o = (b.view(n, R * G, -1) @ gathered(s["v"], s["v_scale"], after, h)).view(n * R * G, D)
            o = (o + a @ gathered(s["v"], s["v_scale"], pre, h)[:shared]) / total
            out[first * R:(first + n) * R, h * G:(h + 1) * G] = o.masked_fill_(empty, 0.0).view(n * R, G, D)
        first += n
    return out.to(s["q"].dtype)


def plain_tables(s):
    page = s["case"]["page"]
    old, new, parents, table = s["old"].long(), s["new"].long(), s["parents"].long(), s["table"]
    n, width, pool = old.numel(), table.shape[1], s["refs"].numel()
    child = parents >= 0
    of = torch.where(child, parents, torch.arange(n, device=DEV))
    base = torch.where(child, torch.minimum(old[of], new), old)
    held, wanted = (base + page - 1) // page, (new + page - 1) // page
    rows = table[of]
    last = rows.gather(1, (held - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0).long()
    parted = (base % page != 0) & (new > base) & (child | (s["refs"][last] > 1))  # its last page becomes its own
    cut = held - parted.long()
    asked, tokens = (wanted - cut).clamp(min=0), (new - base).clamp(min=0)
    ends, asked_ends, count = torch.cumsum(tokens, 0), torch.cumsum(asked, 0), s["free_count"].long()
    served = ((asked == 0) | (asked_ends <= count)) & ((tokens == 0) | (ends <= s["slots"].numel()))
    given = torch.where(served, asked, 0).sum()
    col = torch.arange(width, device=DEV)
    one = torch.ones(n * width, dtype=torch.int32, device=DEV)

    def counted(mask, pages):  # how often each page stands under the mask
        at = torch.where(mask, pages.long(), pool).flatten()
        return torch.zeros(pool + 1, dtype=torch.int32, device=DEV).index_add_(0, at, one)[:pool]

    joins = (child & served)[:, None] & (col < cut[:, None])
    leaves = served[:, None] & ~child[:, None] & (col >= torch.minimum(wanted, cut)[:, None]) & (col < held[:, None])
    comes = (served & (asked > 0))[:, None] & (col >= cut[:, None]) & (col < wanted[:, None])
    pick = (count - 1)[:, None] - ((asked_ends - asked)[:, None] + col - cut[:, None])
    fresh = s["free"][pick.clamp(0, pool - 1)]
    before = table.clone()
    table.copy_(torch.where(comes, fresh, torch.where(joins, rows, table)))
    refs = s["refs"] + counted(joins, rows) - counted(leaves, before) + counted(comes, fresh)
    # given back: pages that nobody holds any more, in the order of their first release
    index = torch.arange(n * width, device=DEV)
    where = torch.where(leaves, before.long(), pool).flatten()
    first = torch.full((pool + 1,), n * width, device=DEV).scatter_reduce_(0, where, index, "amin")
    back = leaves.flatten() & (torch.cat([refs, refs.new_ones(1)])[where] == 0) & (first[where] == index)
    place = torch.where(back, count - given + torch.cumsum(back.long(), 0) - 1, pool)
    s["free"].copy_(torch.cat([s["free"], s["free"].new_zeros(1)]).index_put((place,), before.flatten())[:-1])
    s["refs"].copy_(refs)
    copied = parted & served
    at = torch.where(copied, torch.cumsum(copied.long(), 0) - 1, n)
    empty = torch.full((n + 1,), -1, dtype=torch.int32, device=DEV)
    copy_src = empty.index_put((at,), last.to(torch.int32))[:n]
    copy_dst = empty.index_put((at,), table.gather(1, (held - 1).clamp(min=0)[:, None])[:, 0])[:n]
    t = torch.arange(s["slots"].numel(), device=DEV)
    request = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    live = (t < ends[-1]) & served[request]
    position = base[request] + t - (ends - tokens)[request]
    row = table[request, (position // page).clamp(0, width - 1)].long()
    i32 = torch.int32
    return [table, s["free"], s["refs"], torch.where(live, row * page + position % page, -1),
            torch.where(live, position, 0).to(i32), torch.cat([ends.new_zeros(1), ends]).to(i32),
            torch.where(served, new, old).to(i32), (count - given + back.sum()).to(i32),
            (~served).sum()[None].to(i32), copy_src, copy_dst, copied.sum()[None].to(i32)]


def plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for k, v in s["layers"]:
        k[dst] = k[src]
        v[dst] = v[src]
    return [t for layer in s["layers"] for t in layer]


def plain_compact(s):
    refs, table, page = s["refs"], s["table"], s["case"]["page"]
    pool, room = refs.numel(), s["copy_src"].numel()
    p = torch.arange(pool, device=DEV)
    live = refs > 0
    upto = torch.cumsum(live.long(), 0)
    many, below = upto[-1], upto - live.long()
    # the highest page in use goes to the lowest free one, and so on
    from_rank, to_rank = many - 1 - below, p - below
    goes, takes = live & (p >= many) & (from_rank < room), ~live & (p < many) & (to_rank < room)
    empty = torch.full((room + 1,), -1, dtype=torch.int64, device=DEV)
    src = empty.index_put((torch.where(goes, from_rank, room),), p)[:room]
    dst = empty.index_put((torch.where(takes, to_rank, room),), p)[:room]
    moved = torch.where(goes, dst[from_rank.clamp(0, room - 1)], p)
    refs.copy_(torch.zeros_like(refs).index_add_(0, moved, torch.where(live, refs, 0)))
    held = torch.arange(table.shape[1], device=DEV) < ((s["lens"].long() + page - 1) // page)[:, None]
    table.copy_(torch.where(held, moved[table.clamp(min=0).long()].to(torch.int32), table))
    free = refs == 0
    place = torch.where(free, free.sum() - torch.cumsum(free.long(), 0), pool)
    s["free"].copy_(torch.cat([s["free"], s["free"].new_zeros(1)]).index_put((place,), p.to(torch.int32))[:-1])
    i32 = torch.int32
    return [table, s["free"], refs, (pool - many)[None].to(i32), src.to(i32), dst.to(i32), goes.sum()[None].to(i32),
            moved.to(i32)]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def size_of(name):
    return {"f32": 4, "f16": 2, "bf16": 2}[name]


def cache_bytes(case, values):
    return values * (34 / 32 if case["cache"] == "q8_0" else 2)


def work(case):
    op = case["op"]
    if op == "append":
        T, D, x = case["tokens"], case["dim"], size_of(case["x"])
        heads = case["heads"] + case["kv_heads"]
        return {"bytes": T * D * (case["heads"] * 2 * x + 2 * case["kv_heads"] * x)
                + cache_bytes(case, 2 * T * case["kv_heads"] * D) + T * (8 + 4 * case["axes"]) + 8 * D,
                "flops": T * heads * (3.0 * case["rot"] + 4.0 * D)}
    if op == "prefix":
        lens, shared = lengths(case)
        R, page = case["rows"], case["page"]
        alone = int(np.maximum(lens - shared, 0).sum())
        tokens = sum(m for _, m in group_sizes(case)) + alone
        pages = sum(int(pages_of(m, page)) for _, m in group_sizes(case)) + int(pages_of(np.maximum(lens - shared, 0), page).sum())
        q = case["requests"] * R * case["heads"] * case["dim"]
        seen = sum(int(np.maximum(lens - R + r + 1, 0).sum()) for r in range(R))
        return {"bytes": cache_bytes(case, 2 * tokens * case["kv_heads"] * case["dim"]) + 2 * q * size_of(case["q"])
                + 4 * pages + 4 * case["requests"], "flops": 4.0 * seen * case["heads"] * case["dim"]}
    if op == "tables":
        old, new, parents, _, _ = holdings(case)
        page = case["page"]
        base = np.where(parents >= 0, np.minimum(old[parents], new), old)
        tokens = int(np.maximum(new - base, 0).sum())
        # a fork's entries are read, written and counted; pages that come or go are moved and counted
        joined = int(pages_of(base, page)[parents >= 0].sum())
        moved = int(np.abs(pages_of(base, page) - pages_of(new, page)).sum())
        return {"bytes": 24.0 * case["requests"] + 16 * joined + 16 * moved + 12 * tokens, "flops": 0.0}
    if op == "copy":
        return {"bytes": 2.0 * case["layers"] * case["moves"] * 2 * case["kv_heads"] * case["page"] * case["dim"] * 2
                + 8 * case["moves"], "flops": 0.0}
    # counts read, numbers written, table entries read, stack written
    used = case["used"] * case["pool"]
    return {"bytes": 4.0 * (2 * case["pool"] + used + (case["pool"] - used)), "flops": 0.0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": exact_append, "prefix": exact_prefix, "tables": exact_tables, "copy": exact_copy,
            "compact": exact_compact}[case["op"]](case, s)


def exact_append(case, s):
    # the kept values of a quantized cache are whole multiples of their scale: only q and, in 16 bits, the
    # rotated keys have a value in 64 bits
    T, rot = case["tokens"], case["rot"]
    half = rot // 2
    angle = torch.empty((T, half), dtype=torch.float64, device=DEV)
    for p in range(half):
        angle[:, p] = s["positions"][int(s["axis"][p])].double() * float(s["freq"][p])
    both = []
    for x, gain in ((s["q"], s["q_gain"]), (s["kn"], s["k_gain"])):
        x = x.double()
        z = x / (x.square().sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt() * gain.double()
        if case["interleaved"]:
            pair = torch.view_as_complex(z[..., :rot].reshape(x.shape[:2] + (half, 2)).contiguous())
        else:
            pair = torch.complex(z[..., :half].contiguous(), z[..., half:rot].contiguous())
        pair = pair * torch.polar(torch.ones_like(angle), angle)[:, None]
        z = z.clone()
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


def exact_prefix(case, s):
    """Each request by itself over its own table, as if nothing were shared."""
    page, R, D = case["page"], case["rows"], case["dim"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()

    def history(name, ids, h, n):
        x = s[name][ids, h].reshape(-1, D)[:n].double()
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"][ids, h].reshape(-1, D // 32)[:n].double().repeat_interleave(32, dim=1)
        return x

    for b, n in enumerate(lens):
        ids = torch.from_numpy(table[b, :-(-n // page)].astype(np.int64)).to(DEV)
        for h in range(case["kv_heads"]):
            if not n:
                continue
            k, v = history("k", ids, h, n), history("v", ids, h, n)
            for r in range(R):
                m = n - R + r + 1
                if m > 0:
                    q = s["q"][b * R + r, h * group:(h + 1) * group].double()
                    out[b * R + r, h * group:(h + 1) * group] = torch.softmax(q @ k[:m].t() * D ** -0.5, -1) @ v[:m]
    return out


def exact_tables(case, s):
    """The step told request by request on the host."""
    page, i32 = case["page"], np.int32
    old, new, parents = s["old"].tolist(), s["new"].tolist(), s["parents"].tolist()
    was = s["table"].cpu().numpy()
    table, free, refs = was.copy(), s["free"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    held_by = refs.copy()  # before the step
    stack = free[:int(s["free_count"])].tolist()
    slots = np.full(s["slots"].numel(), -1, np.int64)
    positions = np.zeros(slots.size, i32)
    starts, copies, gone = [0], [], []
    for b, z in enumerate(new):  # the prepared steps have pages and rows enough for all
        p = parents[b]
        a = old[b] if p < 0 else min(old[p], z)
        row = was[b if p < 0 else p]
        have = -(-a // page)
        if p >= 0:
            table[b, :have] = row[:have]
            np.add.at(refs, row[:have], 1)
        if z > a and a % page and (p >= 0 or held_by[row[have - 1]] > 1):
            table[b, have - 1] = stack.pop()
            refs[table[b, have - 1]] += 1
            refs[row[have - 1]] -= 1
            copies.append((row[have - 1], table[b, have - 1]))
            if p < 0:
                gone.append(row[have - 1])
        for j in range(have, -(-z // page)):
            table[b, j] = stack.pop()
            refs[table[b, j]] += 1
        for j in range(-(-z // page), have):
            refs[row[j]] -= 1
            gone.append(row[j])
        where = np.arange(a, z)
        slots[starts[-1]:starts[-1] + where.size] = table[b, where // page].astype(np.int64) * page + where % page
        positions[starts[-1]:starts[-1] + where.size] = where
        starts.append(starts[-1] + where.size)
    for page_ in dict.fromkeys(gone):
        if refs[page_] == 0:
            stack.append(page_)
    free[:len(stack)] = stack
    src, dst = np.full(len(old), -1, i32), np.full(len(old), -1, i32)
    for i, (x, y) in enumerate(copies):
        src[i], dst[i] = x, y
    return [table, free, refs, slots, positions, np.array(starts, i32), np.array(new, i32),
            np.array([len(stack)], i32), np.array([0], i32), src, dst, np.array([len(copies)], i32)]


def exact_copy(case, s):
    out = []
    for layer in s["layers"]:
        for x in layer:
            y = x.clone()
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                y[b].copy_(x[a])
            out.append(y)
    return out


def exact_compact(case, s):
    page, pool, i32 = case["page"], case["pool"], np.int32
    table, free, refs = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    used = np.flatnonzero(refs)
    room = s["copy_src"].numel()
    src, dst, moved = np.full(room, -1, i32), np.full(room, -1, i32), np.arange(pool, dtype=i32)
    high, low = used[used >= used.size][::-1], np.setdiff1d(np.arange(used.size), used)
    for i, (a, b) in enumerate(zip(high[:room], low[:room])):
        src[i], dst[i], moved[a] = a, b, b
        refs[b], refs[a] = refs[a], 0
    for b, n in enumerate(s["lens"].tolist()):
        table[b, :-(-n // page)] = moved[table[b, :-(-n // page)]]
    rest = np.flatnonzero(refs == 0)[::-1]
    free[:rest.size] = rest
    return [table, free, refs, np.array([rest.size], i32), src, dst, np.array([min(room, high.size)], i32), moved]
