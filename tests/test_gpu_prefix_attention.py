"""Attention of requests that share their first pages (paged_prefix_attention)
against a plain 64-bit form that knows nothing of sharing."""
import ctypes

import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import _lib

import paged_plain as plain
from test_gpu_cache import BF16, DEV, F16, F32, KINDS, filled_cache, healthy, normal, poison, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["shared", "by size"])
def limit(request):
    """Calls that would read little again are served in one pass over whole requests:
    every test runs with the shared pages gone through once whatever their size, and
    with the choice as it is."""
    _lib.lib.bq_internal_prefix_whole_limit.restype = ctypes.c_int64
    _lib.lib.bq_internal_prefix_whole_limit.argtypes = [ctypes.c_int64]
    _lib.lib.bq_internal_prefix_whole_limit(0 if request.param == "shared" else -1)
    yield request.param
    _lib.lib.bq_internal_prefix_whole_limit(-1)


def shared_table(g, lens, shared, page, pages, width=None, junk=-1):
    """A table whose requests have their group's first pages in common: shared is a
    list of (requests, positions); a request of length 0 has a row of junk."""
    width = width or max(1, max(-(-n // page) for n in lens))
    order = g.permutation(pages)
    table, at, b = np.full((len(lens), width), junk, np.int32), 0, 0
    for count, positions in shared:
        common = order[at:at + positions // page]
        at += common.size
        for _ in range(count):
            need = -(-lens[b] // page)
            if lens[b]:
                table[b, :common.size] = common
                table[b, common.size:need] = order[at:at + need - common.size]
                at += max(0, need - common.size)
            b += 1
    assert at <= pages and b == len(lens)
    return torch.from_numpy(table).to(DEV)


def pages_needed(lens, shared, page):
    b, n = 0, 3
    for count, positions in shared:
        n += positions // page + sum(max(0, -(-m // page) - positions // page) for m in lens[b:b + count])
        b += count
    return n


def bound_of(want, mag, top, dtype, kind):
    """paged_plain's bound, and what is carried here in fewer bits: over a bf16 cache
    the weights as two bf16 parts (each leaves half a unit of 2^-8 of the rest:
    2^-17 of a weight) and the products of a 128-position tile summed by the tensor
    cores, up to 2 * 32 * 8 additions of the running sum between the fp32 joins,
    each off by 2^-23 of a sum of magnitudes: 2^-14."""
    extra = (2.0 ** -17 + 2.0 ** -14) * mag
    return plain.attention_bound(want, mag, top, dtype, False) + extra * (1 + plain.EPS[dtype])


def check(cache, q, table, lens, shared, rows=1, scale=None, out=None, **more):
    n = len(lens)
    got = bq.paged_prefix_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), shared, rows=rows,
                                    scale=scale, out=out, **more)
    k, v = plain.values(cache)
    s = cache.head_dim ** -0.5 if scale is None else scale
    want, mag, top = plain.attention(k, v, q.cpu(), table.cpu(), lens, rows, s)
    bound = bound_of(want, mag, top, q.dtype, cache.kind)
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside the bound; worst {err[bad].max()} at "
                           f"{bad.nonzero()[0].tolist()}")
    assert n == lens.__len__()
    return got


def case(g, kind, dtype, lens, shared, page, heads, kv, D, rows=1, layout="hs", width=None, hurt=True, **more):
    groups = [(len(lens), shared)] if isinstance(shared, int) else shared
    pages = pages_needed(lens, groups, page)
    cache = filled_cache(g, kind, pages, page, kv, D, layout)
    table = shared_table(g, lens, groups, page, pages, width)
    if hurt:
        poison(cache, table, lens)
    q = normal(g, (len(lens) * rows, heads, D), dtype)
    return check(cache, q, table, lens, shared, rows=rows, **more), cache, q, table


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("D,heads,kv", [(128, 16, 4), (64, 14, 2), (96, 6, 3), (256, 4, 1), (32, 5, 5), (160, 2, 2)])
def test_types_and_heads(kind, dtype, D, heads, kv):
    """Ragged rests, one of them empty, one request that has ended."""
    lens = [300, 289, 288, 0, 417, 305]
    case(rng("p", kind, str(dtype), D), kind, dtype, lens, 288, 16, heads, kv, D)


@pytest.mark.parametrize("kind,dtype", [("f16", F16), ("f16", F32), ("bf16", BF16), ("bf16", F32)])
@pytest.mark.parametrize("D,page", [(8, 8), (24, 16), (40, 40), (72, 5), (120, 24)])
def test_odd_heads(kind, dtype, D, page):
    """Heads that are no whole steps or blocks of the tensor cores, one kv head and three."""
    for kv in (1, 3):
        g = rng("odd", kind, str(dtype), D, kv)
        case(g, kind, dtype, [650, 641, 699, 0, 640], 640, page, 4 * kv, kv, D, layout=("hs", "sh")[kv == 3])


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", F32)])
def test_pages_beyond_32_bits(kind, dtype):
    """Pages whose offset is above 2^31 elements (2^32 bytes in 16 bits), copied there
    from the front first."""
    g = rng("far", kind)
    D, kv, page, pool, requests, shared = 128, 8, 16, 140000, 12, 700
    small = filled_cache(g, kind, 160, page, kv, D)
    lens = [shared + 1 + int(n) for n in g.integers(0, 20, requests)]
    near = shared_table(g, lens, [(requests, shared)], page, 160)
    planes = [torch.empty((pool,) + t.shape[1:], dtype=t.dtype, device=DEV) for t in
              (small.k, small.v) + (() if small.k_scale is None else (small.k_scale, small.v_scale))]
    for big, t in zip(planes, (small.k, small.v, small.k_scale, small.v_scale)):
        big[:160] = t
    cache = bq.PagedKVCache(*planes)
    assert cache.k.stride(0) * (pool - 200) > 2 ** 31
    src = torch.arange(160, dtype=torch.int32, device=DEV)
    bq.kv_copy_pages(cache, src, pool - 1 - src)
    q = normal(g, (requests, 16, D), dtype)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = bq.paged_prefix_attention(small, q, near, at, shared)
    far = torch.where(near >= 0, pool - 1 - near, near)
    assert torch.equal(bq.paged_prefix_attention(cache, q, far, at, shared), want)
    assert torch.equal(bq.paged_attention(cache, q, far, at), bq.paged_attention(small, q, near, at))


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", F32)])
@pytest.mark.parametrize("shared", [0, 1, 15, 16, 17, 127, 128, 129, 255, 257, 640, 1000])
def test_shared_lengths(kind, dtype, shared):
    """From nothing to beyond tiles and chunks; what is not a whole page is each request's own."""
    lens = [shared + 1, shared + 40, shared + 2]
    case(rng("s", kind, shared), kind, dtype, lens, shared, 16, 8, 2, 128)


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("f16", F16), ("bf16", BF16), ("bf16", F32), ("q8_0", BF16)])
@pytest.mark.parametrize("requests,heads,kv", [(1, 1, 1), (33, 8, 2), (130, 4, 4), (64, 16, 4), (300, 7, 1)])
def test_many_rows(kind, dtype, requests, heads, kv):
    """Tiles of query rows, the last one ragged."""
    g = rng("r", kind, requests)
    lens = [200 + int(n) for n in g.integers(1, 60, requests)]
    case(g, kind, dtype, lens, 200, 8, heads, kv, 64)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D,page,layout", [(32, 16, "hs"), (96, 24, "sh"), (128, 7, "kv"), (128, 64, "hs"), (64, 16, "sh")])
def test_many_rows_over_q8_0(dtype, D, page, layout):
    """Enough rows that codes are put into parts for the tensor cores, ragged tiles of
    positions, a page outside the pool among them (masked)."""
    g = rng("q8", str(dtype), D, page)
    lens = [n + 1 for n in g.integers(700, 760, 29)] + [0]
    case(g, "q8_0", dtype, lens, 700, page, 6, 3, D, layout=layout)
    shared = [(20, 700), (10, 333)]
    lens = [701 + int(n) for n in g.integers(0, 40, 20)] + [334 + int(n) for n in g.integers(0, 40, 10)]
    out, cache, q, table = case(g, "q8_0", dtype, lens, shared, page, 6, 3, D, layout=layout, hurt=False)
    bad = 333 // page // 2
    table[:, bad] = cache.pages + 3
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    hurt = bq.paged_prefix_attention(cache, q, table, at, shared)
    assert bq.device_status(clear=True) == 0x100
    keep = [i for i in range(table.shape[1]) if i != bad]
    want, mag, top = plain.attention(*plain.values(cache), q.cpu(), table.cpu()[:, keep], [n - page for n in lens], 1,
                                     D ** -0.5)
    assert ((hurt.cpu().double() - want).abs() <= bound_of(want, mag, top, dtype, "q8_0")).all()


@pytest.mark.parametrize("D,dtype,layout", [(64, F16, "hs"), (128, F32, "kv")])
@pytest.mark.parametrize("rows", [33, 64, 65, 97, 161])
def test_tiles_partly_filled_over_q8_0(D, dtype, layout, rows):
    """Rows that fill one to four of a tile's quarters, and a second tile's first: the
    warps of the others put codes into parts."""
    g = rng("quarters", str(dtype), D, rows)
    case(g, "q8_0", dtype, [400 + int(n) for n in g.integers(0, 20, rows)], 400, 16, 1, 1, D, layout=layout)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** -12, 1.0, 3.0e4])
def test_scales_of_any_size_over_q8_0(dtype, size):
    """All scales small or large, and a few blocks far above the others.  A value of a
    block far below the largest of its chunk is off by 2^-39 of what the largest scale's
    codes reach (127 times it), a score by that much of each of its D products."""
    g = rng("scales", str(dtype), str(size))
    D, page, n, requests = 64, 16, 512, 20
    pages = n // page + requests + 2
    lens = [n + 3 + b % 9 for b in range(requests)]
    table = shared_table(g, lens, [(requests, n)], page, pages)
    for far in (False, True):
        cache = filled_cache(g, "q8_0", pages, page, 2, D)
        cache.k_scale.mul_(30 * size).clamp_(max=6.0e4)
        cache.v_scale.mul_(30 * size).clamp_(max=6.0e4)
        if far:
            cache.k_scale[table[0, 5].long(), :, 3, 1] = 6.0e4
            cache.v_scale[table[0, 7].long(), :, 9, 0] = 6.0e4
        # scores of a few units whatever the keys' size; with a far block that block decides
        q = (normal(g, (requests, 4, D)) / max(float(cache.k_scale.max()) * 60, 2.0 ** -30)).to(dtype)
        out = bq.paged_prefix_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), n)
        k, v = plain.values(cache)
        want, mag, top = plain.attention(k, v, q.cpu(), table.cpu(), lens, 1, D ** -0.5)
        kt, vt = (127.0 * float(s.max()) for s in (cache.k_scale, cache.v_scale))
        score = D ** -0.5 * D * float(q.abs().max()) * 2.0 ** -38 * kt
        extra = 2.0 ** -38 * vt + 2 * score * mag
        bound = bound_of(want, mag, top, dtype, "q8_0") + extra * (1 + plain.EPS[dtype])
        assert ((out.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", F32)])
def test_a_long_prefix(kind, dtype):
    lens = [9003, 9100, 9003, 0, 9777]
    case(rng("long", kind), kind, dtype, lens, 9003, 24, 8, 2, 128, hurt=False)


@pytest.mark.parametrize("kind,dtype,D", [("f16", F32, 64), ("f16", F16, 128), ("bf16", BF16, 64), ("bf16", F32, 64),
                                          ("q8_0", F32, 64), ("q8_0", BF16, 128)])
@pytest.mark.parametrize("shared", [1111, 4100])
def test_long_chunks(kind, dtype, D, shared):
    """Row tiles and heads enough for the whole GPU, so that a chunk is many tiles of
    positions long and O is added up several times; the maximum grows late in some rows.
    Against the ordinary kernel, whose own error is within its bound."""
    g = rng("chunks", kind, str(dtype), shared)
    requests, heads, kv, page = 200, 32, 16, 32
    lens = [shared + 5 + int(n) for n in g.integers(0, 30, requests)]
    pages = pages_needed(lens, [(requests, shared)], page)
    cache = filled_cache(g, kind, pages, page, kv, D)
    table = shared_table(g, lens, [(requests, shared)], page, pages)
    late = table[0, shared // page - 2].long()
    if kind == "q8_0":
        cache.k_scale[late] *= 3
    else:
        cache.k[late] *= 3
    q = normal(g, (requests * 5, heads, D), dtype)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = bq.paged_attention(cache, q, table, at, rows=5).double()
    got = bq.paged_prefix_attention(cache, q, table, at, shared, rows=5).double()
    # values N(0, 1) (Q8_0: rms 2.2, at most 3.81): outputs below 4, mean magnitudes below 4.
    # Scores below 60 of magnitude 200: both forms are off by at most twice 2^-17 of that in
    # the weights, 2^-14 in the sums, 2^-17 in bf16 weights, and half a unit of the output.
    rel = 2 * (2.0 ** -17 * 200 + 2.0 ** -20) + 2.0 ** -14 + 2.0 ** -17
    assert float((got - want).abs().max()) <= 2 * (rel * 4 + plain.EPS[dtype] / 2 * 4)
    # and over all of them, where the errors are of both signs: a hundredth of that bound
    # beside the output's rounding (fp32: sums of thousands of terms, 2^-24 * 64 of them)
    assert float((got - want).norm() / want.norm()) <= plain.EPS[dtype] + 2.0 ** -16


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", F32)])
@pytest.mark.parametrize("rows", [2, 5, 6])
def test_verify_rows(kind, dtype, rows):
    """Row r of a request sees rows - 1 - r positions fewer; the first one sees the
    whole prefix and maybe nothing else."""
    lens = [256 + rows - 1, 256 + rows, 300, 0, 271]
    case(rng("v", kind, rows), kind, dtype, lens, 256, 16, 8, 2, 128, rows=rows)


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", F32)])
def test_groups(kind, dtype):
    """Groups of several lengths, one that shares nothing, an empty one, one whose
    first request has ended, one that has ended whole."""
    shared = [(3, 700), (2, 0), (0, 500), (4, 129), (2, 64), (1, 2000)]
    lens = [710, 900, 701, 5, 333, 0, 140, 131, 600, 0, 0, 2004]
    case(rng("g", kind), kind, dtype, lens, shared, 16, 8, 2, 64)


def test_groups_of_one():
    shared = [(1, 10 * i) for i in range(64)]
    case(rng("g1"), "f16", F16, [10 * i + 7 for i in range(64)], shared, 8, 4, 2, 64)


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", BF16)])
@pytest.mark.parametrize("page,layout", [(1, "hs"), (7, "sh"), (24, "kv"), (128, "sh"), (200, "hs")])
def test_pages_and_layouts(kind, dtype, page, layout):
    lens = [500, 433, 470]
    case(rng("l", kind, page), kind, dtype, lens, 431, page, 6, 2, 64, layout=layout)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    for kind, dtype in (("f16", F32), ("bf16", BF16), ("q8_0", F32)):
        case(rng("scale", kind), kind, dtype, [400, 390, 385], 384, 16, 8, 2, 128, scale=scale)


def test_strided_queries_outputs_in_place_and_a_workspace():
    g = rng("strides")
    for kind, dtype in (("f16", F32), ("bf16", BF16), ("q8_0", F32)):
        lens, page = [400, 390, 385], 16
        cache = filled_cache(g, kind, 90, page, 2, 64)
        table = shared_table(g, lens, [(3, 384)], page, 90, width=40)
        wide = normal(g, (3, 8 + 2, 64 + 1), dtype)
        q = wide[:, 1:9, 1:]
        first = check(cache, q, table, lens, 384)
        again = bq.paged_prefix_attention(cache, q.contiguous(), table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                          384)
        assert torch.equal(first, again)
        room = torch.empty(bq.paged_prefix_attention_workspace(cache, 3, 1, 8, 40, 384, dtype) + 5, dtype=torch.uint8,
                           device=DEV)
        room.fill_(255)
        out = normal(g, (3, 10, 80), dtype)
        kept = out.clone()
        view = out[:, 2:, 3:67]
        bq.paged_prefix_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), [(3, 384)], out=view,
                                  workspace=room)
        assert torch.equal(view, first)
        kept[:, 2:, 3:67] = view
        assert torch.equal(out, kept)  # and nothing else
        same = q.clone()
        assert torch.equal(bq.paged_prefix_attention(cache, same, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                                     384, out=same), first)
        assert torch.equal(same, first)


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", F32)])
def test_large_scores_and_growing_maxima(kind, dtype):
    """Scores of hundreds, rising and falling over the positions: the running maximum
    is replaced again and again, or never after the first tile."""
    g = rng("grow", kind)
    page, n = 16, 2048
    for order in (1, -1):
        cache = filled_cache(g, kind, n // page + 12, page, 1, 64)
        table = shared_table(g, [n + 20, n + 9], [(2, n)], page, n // page + 12)
        ramp = torch.linspace(0.05, 12.0, n, device=DEV)[::order].contiguous() if order == 1 else torch.linspace(
            12.0, 0.05, n, device=DEV)
        ids = table[0, :n // page].long()
        k = ramp.view(-1, 1, page, 1) * (0.5 + 0.5 * torch.rand(n // page, 1, page, 64, device=DEV))
        if kind == "q8_0":
            cache.k_scale[ids] = (k.abs().amax(-1, keepdim=True) / 127).to(F16).expand(-1, -1, -1, 2)
            cache.k[ids] = (k / cache.k_scale[ids].float().repeat_interleave(32, -1)).round().clamp(-127, 127).to(torch.int8)
        else:
            cache.k[ids] = k.to(cache.k.dtype)
        q = (0.5 + normal(g, (2, 4, 64)).abs()).to(dtype)
        check(cache, q, table, [n + 20, n + 9], n)


def test_scales_that_are_not_finite_over_q8_0():
    """A NaN or infinite scale of a shared value or key reaches the rows of its head and
    where it lies, and nothing else."""
    g = rng("nans")
    lens, page = [300 + b % 5 for b in range(25)], 16
    out, cache, q, table = case(g, "q8_0", F32, lens, 288, page, 8, 2, 64)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for bad in (float("nan"), float("inf")):
        kept = cache.v_scale.clone()
        cache.v_scale[int(table[0, 4]), 1, 6, 1] = bad  # values 32 to 63 of head 1
        hurt = bq.paged_prefix_attention(cache, q, table, at, 288)
        same = torch.ones_like(out, dtype=torch.bool)
        same[:, 4:, 32:] = False
        assert torch.equal(hurt[same], out[same]) and not hurt[:, 4:, 32:].isfinite().any()
        cache.v_scale.copy_(kept)
        kept = cache.k_scale.clone()
        cache.k_scale[int(table[0, 4]), 0, 6, 0] = float("nan")
        hurt = bq.paged_prefix_attention(cache, q, table, at, 288)
        assert hurt[:, :4].isnan().all() and torch.equal(hurt[:, 4:], out[:, 4:])
        cache.k_scale.copy_(kept)


def test_values_that_are_not_finite_reach_only_their_rows_and_heads():
    g = rng("inf")
    for kind, dtype in (("f16", F32), ("bf16", BF16)):
        lens, page = [300, 290, 289], 16
        out, cache, q, table = case(g, kind, dtype, lens, 288, page, 4, 2, 64)
        own = int(table[1, 18])
        cache.v[own, 1, 0, 3] = float("nan")  # of request 1's own page, head 1
        hurt = bq.paged_prefix_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), 288)
        same = torch.ones_like(out, dtype=torch.bool)
        same[1, 2:, 3] = False
        assert torch.equal(out[same], hurt[same]) and hurt[1, 2:, 3].isnan().all()
        cache.k[int(table[0, 3]), 0, 5, 7] = float("nan")  # of the shared pages, head 0
        hurt = bq.paged_prefix_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), 288)
        assert hurt[:, :2].isnan().all() and torch.equal(hurt[:, 2:][same[:, 2:]], out[:, 2:][same[:, 2:]])
        qq = q.clone()
        cache.k[int(table[0, 3]), 0, 5, 7] = 0.0
        cache.v[own, 1, 0, 3] = 0.0
        want = bq.paged_prefix_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), 288)
        qq[2, 3, 0] = float("inf")  # one row's query
        hurt = bq.paged_prefix_attention(cache, qq, table, torch.tensor(lens, dtype=torch.int32, device=DEV), 288)
        keep = torch.ones(3, 4, dtype=torch.bool, device=DEV)
        keep[2, 3] = False
        assert torch.equal(hurt[keep], want[keep]) and not hurt[2, 3].isfinite().all()


def test_a_row_has_its_bits_whatever_is_beside_it():
    """Other queries and other requests' own pages do not move a row."""
    for kind, dtype in (("f16", F32), ("bf16", BF16), ("q8_0", F32)):
        g = rng("beside", kind)
        lens = [1100, 1050, 1029, 1033]
        out, cache, q, table = case(g, kind, dtype, lens, 1024, 16, 8, 2, 128, hurt=False)
        q2 = q * 3
        q2[1] = q[1]
        for b in (0, 2, 3):
            own = table[b, 64:-(-lens[b] // 16)].long()
            if cache.k_scale is None:
                cache.k[own] = -cache.k[own]
            else:
                cache.k_scale[own] = cache.k_scale[own] * 2
        again = bq.paged_prefix_attention(cache, q2, table, torch.tensor(lens, dtype=torch.int32, device=DEV), 1024)
        assert torch.equal(again[1], out[1])


def test_bad_pages_and_short_requests_are_reported():
    g = rng("bad")
    for kind, dtype in (("f16", F32), ("bf16", BF16), ("q8_0", F32)):
        lens, page, pages = [300, 290, 200, 289], 16, 60
        cache = filled_cache(g, kind, pages, page, 2, 64)
        table = shared_table(g, [300, 290, 300, 289], [(4, 288)], page, pages)
        q = normal(g, (4, 4, 64), dtype)
        at = torch.tensor(lens, dtype=torch.int32, device=DEV)
        out = bq.paged_prefix_attention(cache, q, table, at, 288)
        assert bq.device_status(clear=True) == 0x200  # request 2 does not see its prefix
        assert (out[2] == 0).all() and (out[[0, 1, 3]] != 0).any(-1).all()
        table[:, 3] = pages + 5  # a shared page outside the pool: masked
        at[2] = 0
        hurt = bq.paged_prefix_attention(cache, q, table, at, 288)
        assert bq.device_status(clear=True) == 0x100
        k, v = plain.values(cache)
        t = table.cpu().clone()
        keep = [i for i in range(t.shape[1]) if i != 3]
        cut = t[:, keep]
        want, mag, top = plain.attention(k, v, q.cpu(), cut, [n - 16 if n else 0 for n in at.tolist()], 1, 64 ** -0.5)
        assert ((hurt.cpu().double() - want).abs() <= bound_of(want, mag, top, dtype, kind)).all()


def test_captured_and_replayed_with_other_lengths_beside_another_graph():
    g = rng("graph")
    page, pages = 16, 200
    caches = [filled_cache(g, kind, pages, page, 2, 128) for kind in ("f16", "q8_0")]
    table = shared_table(g, [900, 900, 900], [(3, 640)], page, pages)
    q = normal(g, (3, 8, 128))
    lens = torch.tensor([641, 650, 700], dtype=torch.int32, device=DEV)
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for cache in caches:
        bq.paged_prefix_attention(cache, q, table, lens, 640)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = bq.paged_prefix_attention(cache, q, table, lens, 640)
        graphs.append((graph, out))
    for step in range(4):
        lens += 13
        torch.cuda.synchronize()
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for cache, (_, out) in zip(caches, graphs):
            assert torch.equal(out, bq.paged_prefix_attention(cache, q, table, lens, 640))


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("requests,shared,heads,kv,D", [(40, 2049, 16, 4, 128), (9, 1030, 14, 2, 64)])
def test_steps_back_to_back(kind, requests, shared, heads, kv, D):
    """A token appended and attended, step after step with nothing between the launches,
    eager and replayed, has the bits of the steps that are waited for."""
    g, page, own, steps = rng("steps", kind, requests), 16, 4, 12
    whole = shared // page
    at = whole * page + 3
    first = filled_cache(g, kind, whole + requests * own, page, kv, D)
    planes = [t for t in (first.k, first.v, first.k_scale, first.v_scale) if t is not None]
    table = torch.arange(whole, dtype=torch.int32).expand(requests, -1)
    table = torch.cat([table, whole + torch.arange(requests * own, dtype=torch.int32).view(requests, own)], 1).to(DEV)
    k, v = (normal(g, (steps, requests, kv, D), F16) for _ in range(2))
    q = normal(g, (steps, requests, heads, D), F16)
    slots = [table[:, (at + i) // page].long() * page + (at + i) % page for i in range(steps)]
    lens = [torch.full((requests,), at + i + 1, dtype=torch.int32, device=DEV) for i in range(steps)]

    def run(cache, wait):
        out = []
        for i in range(steps):
            bq.kv_append(cache, k[i], v[i], slots[i])
            wait()
            out.append(bq.paged_prefix_attention(cache, q[i], table, lens[i], shared))
            wait()
        return out

    def fresh():
        return bq.PagedKVCache(*[t.clone() for t in planes])

    want = run(fresh(), torch.cuda.synchronize)
    for _ in range(4):
        got = run(fresh(), lambda: None)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    cache = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(cache, lambda: None)
    for _ in range(4):
        for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), planes):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_it_agrees_with_ordinary_attention_at_a_servers_size():
    """Both forms of one call lie within their bounds of one another."""
    g = rng("both")
    requests, page = 40, 32
    lens = [6000 + int(n) for n in g.integers(1, 300, requests)]
    pages = pages_needed(lens, [(requests, 6000)], page)
    for kind, dtype in (("f16", F16), ("bf16", BF16), ("q8_0", F32)):
        cache = filled_cache(g, kind, pages, page, 4, 128)
        table = shared_table(g, lens, [(requests, 6000)], page, pages)
        q = normal(g, (requests, 16, 128), dtype)
        at = torch.tensor(lens, dtype=torch.int32, device=DEV)
        a = bq.paged_attention(cache, q, table, at).double()
        b = bq.paged_prefix_attention(cache, q, table, at, 6000).double()
        # outputs are means of thousands of N(0, 1) values (a Q8_0 value's rms is 2.2): below 0.5.
        # Each is off by half a unit of its type and 2^-13 of the mean magnitude (below 2).
        assert float((a - b).abs().max()) <= 2 * (plain.EPS[dtype] / 2 * 0.5 + 2.0 ** -13 * 2)


def test_nothing_to_do_and_refusals(limit):
    cache = bq.PagedKVCache.zeros(8, 16, 2, 64)
    i32 = dict(dtype=torch.int32, device=DEV)
    q, table, lens = torch.zeros(2, 4, 64, device=DEV), torch.zeros(2, 4, **i32), torch.full((2,), 20, **i32)
    none = bq.paged_prefix_attention(cache, q[:0], table[:0], lens[:0], 16)
    assert none.shape == (0, 4, 64)
    for bad in (-1, 65, [(1, 16)], [(3, 16)], [(3, 16), (-1, 16)], [], [(1, 8)] * 65):
        with pytest.raises((ValueError, bq.BQError)):
            bq.paged_prefix_attention(cache, q, table, lens, bad)
    with pytest.raises(ValueError):
        bq.paged_prefix_attention(cache, q, table, lens, 16, rows=7)
    with pytest.raises(TypeError):
        bq.paged_prefix_attention(cache, q, table, lens.long(), 16)
    with pytest.raises(ValueError):
        bq.paged_prefix_attention(cache, q, table[:1], lens, 16)
    if limit == "shared":  # (the one pass needs no workspace here)
        with pytest.raises(bq.BQError):
            bq.paged_prefix_attention(cache, q, table, lens, 16, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(bq.BQError):
        bq.paged_prefix_attention(cache, q, table, lens, 16, scale=float("nan"))
