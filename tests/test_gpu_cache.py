"""The paged key-value cache on the GPU: block tables, append with rotary
positions and attention, each against a plain 64-bit form at the sizes and masks
where it can go wrong, and a run of them together as a server would use them."""
import os
import re
import subprocess
import sys
import threading
import zlib

import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import _lib

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def healthy():
    bq.device_status(clear=True)
    yield
    assert bq.device_status(clear=True) == 0


def rng(*key):
    return np.random.default_rng([zlib.crc32(k.encode()) if isinstance(k, str) else int(k) for k in key])


def normal(g, shape, dtype=F32):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(dtype).to(DEV)


def filled_cache(g, kind, pages, page, kv, D, layout="hs"):
    """A cache of N(0, 1) values; layout "sh": slots before heads in memory,
    "kv": k and v slices of one tensor."""
    shape = (pages, kv, page, D)
    if kind == "q8_0":
        def codes():
            return torch.from_numpy(g.integers(-127, 128, shape).astype(np.int8)).to(DEV)

        def scales():
            return torch.from_numpy((0.02 + 0.01 * g.random(shape[:3] + (D // 32,))).astype(np.float16)).to(DEV)

        parts = [codes(), codes(), scales(), scales()]
    else:
        parts = [normal(g, shape, {"f16": F16, "bf16": BF16}[kind]) for _ in range(2)]
    if layout == "sh":
        parts = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in parts]
    elif layout == "kv":
        def together(a, b):
            both = torch.stack([a, b], 1)
            return [both[:, 0], both[:, 1]]
        parts = [t for i in range(0, len(parts), 2) for t in together(parts[i], parts[i + 1])]
    return bq.PagedKVCache(*parts)


def request_tables(g, lens, page, pages, width=None, junk=-1):
    """A table over distinct random pages; entries behind a request's pages are junk."""
    need = [-(-n // page) for n in lens]
    width = width or max(need + [1])
    order = g.permutation(pages)
    table = np.full((len(lens), width), junk, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    assert at <= pages
    return torch.from_numpy(table).to(DEV)


def poison(cache, table, lens):
    """NaN (or the largest scale, for codes) in every slot that no request holds."""
    page = cache.page_size
    live = torch.zeros(cache.pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            live[int(table[b, t // page]), t % page] = True
    dead = (~live).to(DEV)[:, None, :, None]
    for t in (cache.k, cache.v) if cache.k_scale is None else (cache.k_scale, cache.v_scale):
        t.masked_fill_(dead, float("nan"))


def check_attention(cache, q, table, lens, rows=1, scale=None, out=None, **more):
    got = bq.paged_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), rows=rows, scale=scale,
                             out=out, **more)
    k, v = plain.values(cache)
    s = cache.head_dim ** -0.5 if scale is None else scale
    want, mag, top = plain.attention(k, v, q.cpu(), table.cpu(), lens, rows, s)
    bound = plain.attention_bound(want, mag, top, q.dtype, cache.kind == "q8_0" and q.dtype == BF16)
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside the bound; worst {err[bad].max()} at "
                           f"{bad.nonzero()[0].tolist()}")
    return got


# lengths: none, one, around a tile of 16 and 32, around a page, around chunks of 128
LENS = [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 300]
KINDS = [("f16", F16), ("f16", F32), ("bf16", BF16), ("bf16", F32), ("q8_0", F32), ("q8_0", BF16), ("q8_0", F16),
         ("f16", BF16), ("bf16", F16)]


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("D,heads,kv", [(128, 16, 4), (64, 14, 2), (96, 6, 3), (256, 4, 1), (32, 5, 5)])
def test_attention_types_and_heads(kind, dtype, D, heads, kv):
    g = rng(kind, D)
    page = 16
    pages = sum(-(-n // page) for n in LENS) + 3
    cache = filled_cache(g, kind, pages, page, kv, D)
    table = request_tables(g, LENS, page, pages)
    poison(cache, table, LENS)
    q = normal(g, (len(LENS), heads, D), dtype)
    out = check_attention(cache, q, table, LENS)
    assert (out[0] == 0).all()  # an empty row


@pytest.mark.parametrize("page", [1, 3, 8, 24, 100, 128])
@pytest.mark.parametrize("layout", ["hs", "sh", "kv"])
@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_attention_pages_and_layouts(page, layout, kind):
    """Pages that end inside a tile, and other orders in memory."""
    g = rng(page, layout)
    lens = [47, 1, 200, 0, 130]
    pages = sum(-(-n // page) for n in lens) + 2
    cache = filled_cache(g, kind, pages, page, 2, 64, layout)
    table = request_tables(g, lens, page, pages, junk=1 << 30)
    poison(cache, table, lens)
    check_attention(cache, normal(g, (5, 8, 64)), table, lens)


@pytest.mark.parametrize("kind,dtype,D,heads,kv", [
    ("f16", F32, 128, 28, 4), ("q8_0", F32, 128, 40, 8), ("bf16", BF16, 64, 8, 1), ("f16", F16, 80, 6, 2),
    ("q8_0", BF16, 160, 12, 2), ("q8_0", F16, 96, 7, 1), ("bf16", F32, 256, 16, 2)])
def test_verify_rows_are_the_one_row_calls(kind, dtype, D, heads, kv):
    """Every number of rows: within the bound, and each row's bits are those of
    the one-row call at the length that it sees."""
    g = rng(kind, D, heads)
    page = 16
    lens = [3, 1, 40, 133, 700, 6]
    pages = sum(-(-n // page) for n in lens) + 1
    cache = filled_cache(g, kind, pages, page, kv, D)
    table = request_tables(g, lens, page, pages)
    poison(cache, table, lens)
    for rows in (2, 3, 6):
        q = normal(g, (len(lens) * rows, heads, D), dtype)
        out = check_attention(cache, q, table, lens, rows=rows).view(len(lens), rows, heads, D)
        for r in range(rows):
            seen = torch.tensor([max(0, n - rows + r + 1) for n in lens], dtype=torch.int32, device=DEV)
            one = bq.paged_attention(cache, q.view(len(lens), rows, heads, D)[:, r].contiguous(), table, seen)
            assert torch.equal(one, out[:, r]), (rows, r)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("n", [5, 130, 2000])
def test_a_draft_token_does_not_reach_the_rows_before_it(kind, n):
    """NaN and infinities in the last draft token's key, value and scales."""
    g = rng(kind, n)
    rows, page = 4, 16
    pages = -(-n // page) + 1
    cache = filled_cache(g, kind, pages, page, 2, 64)
    table = request_tables(g, [n], page, pages)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = normal(g, (rows, 8, 64))
    clean = bq.paged_attention(cache, q, table, lens, rows=rows)
    at = (int(table[0, (n - 1) // page]), slice(None), (n - 1) % page)
    if kind == "q8_0":
        cache.k_scale[at], cache.v_scale[at] = float("nan"), float("inf")
    else:
        cache.k[at], cache.v[at] = float("nan"), float("inf")
    out = bq.paged_attention(cache, q, table, lens, rows=rows)
    assert torch.equal(out[:-1], clean[:-1])
    assert not torch.isfinite(out[-1]).any()
    if kind != "q8_0":
        cache.k[at], cache.v[at] = 0, float("nan")
        out = bq.paged_attention(cache, q, table, lens, rows=rows)
        assert torch.equal(out[:-1], clean[:-1]) and torch.isnan(out[-1]).all()


@pytest.mark.parametrize("lens,width", [([5000], 400), ([9000, 10, 4097], 600), ([70000], None), ([2500] * 40, None)])
def test_attention_of_long_caches(lens, width):
    """Chunks joined by a second kernel, one and several per request, more units
    than fit the GPU at once, and a table wider than the requests need."""
    g = rng(len(lens), lens[0])
    page = 16
    pages = sum(-(-n // page) for n in lens)
    cache = filled_cache(g, "f16", pages, page, 2, 64)
    table = request_tables(g, lens, page, pages, width)
    q = normal(g, (len(lens), 6, 64))
    a = check_attention(cache, q, table, lens)
    assert torch.equal(a, bq.paged_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV)))
    rows = 3
    check_attention(cache, normal(g, (len(lens) * rows, 6, 64)), table, lens, rows=rows)


def test_attention_of_short_requests_in_a_wide_table():
    """Many more units than the requests fill: live ones are found by a scan."""
    g = rng(42)
    lens = [int(n) for n in g.integers(0, 60, 300)]
    lens[7], lens[200] = 5000, 2049
    page = 16
    pages = sum(-(-n // page) for n in lens)
    cache = filled_cache(g, "bf16", pages, page, 2, 64)
    table = request_tables(g, lens, page, pages, width=1000)
    check_attention(cache, normal(g, (300, 4, 64), BF16), table, lens)
    check_attention(cache, normal(g, (600, 4, 64)), table, lens, rows=2)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 104, 200])
def test_odd_head_sizes(D):
    g = rng(D, 43)
    lens, page = [0, 5, 33, 400], 8
    pages = sum(-(-n // page) for n in lens) + 1
    cache = filled_cache(g, "f16", pages, page, 3, D)
    table = request_tables(g, lens, page, pages)
    poison(cache, table, lens)
    check_attention(cache, normal(g, (4, 6, D)), table, lens)
    check_attention(cache, normal(g, (8, 3, D), BF16), table, lens, rows=2)
    check_append(g, "f16", F32, 9, 4, 3, D, 16 if D >= 16 else 0, None, False, 8, 300)
    check_append(g, "bf16", F16, 9, 4, 3, D, D // 16 * 16, None, True, 8, 300)


def test_first_calls_of_a_process_inside_a_capture():
    """A process whose first call of each kernel is captured."""
    code = """
import torch, sys
sys.path.insert(0, {root!r})
import block_quantized_weight_dequant_gb300 as bq
dev = "cuda"
cache = bq.PagedKVCache.zeros(40, 16, 2, 64, "q8_0")
t = bq.BlockTables(2, 20, 40, 16, 8)
goal = torch.tensor([3, 4], dtype=torch.int32, device=dev)
k, q = torch.randn(8, 2, 64, device=dev), torch.randn(8, 4, 64, device=dev)
rope = bq.Rope.from_theta(64)
ws = torch.empty(1 << 24, dtype=torch.uint8, device=dev)
out, turned, x = torch.empty(2, 4, 64, device=dev), torch.empty_like(q), torch.empty(8, 256, device=dev)
gain = torch.ones(256, device=dev)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    t.resize(goal)
    bq.kv_append(cache, k, k, t.slots, q=q, q_out=turned, rope=rope, positions=t.positions)
    bq.paged_attention(cache, turned[:2], t.table, t.lens, out=out, workspace=ws)
    bq.sandwich_norm(turned.view(8, 256), turned.view(8, 256), gain, h_out=x, x_out=torch.empty_like(x))
graph.replay()
torch.cuda.synchronize()
assert t.lens.tolist() == [3, 4] and torch.isfinite(out).all() and bool(out.abs().sum() > 0)
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_scores_and_scales_of_any_size(kind):
    """Large scores (weights down to 0), tiny and huge queries, values and scales."""
    g = rng(7)
    lens, page = [300, 77], 16
    cache = filled_cache(g, kind, 30, page, 2, 64)
    if kind == "q8_0":
        cache.v_scale[::3] *= 2000.0
        cache.v_scale[1::3] *= 1e-4
        cache.k_scale[::2] *= 30.0
    else:
        cache.v[::3] *= 3000.0
        cache.k[1::2] *= 0.001
    table = request_tables(g, lens, page, 30)
    q = normal(g, (2, 8, 64))
    for factor in (1.0, 1e-12, 3e-39, 50.0, 1e6):
        check_attention(cache, q * factor, table, lens)
    check_attention(cache, q, table, lens, scale=-0.3)
    check_attention(cache, q, table, lens, scale=0.0)
    check_attention(cache, torch.zeros_like(q), table, lens)


WEIGHT_KINDS = [("f16", F16), ("f16", F32), ("f16", BF16), ("bf16", BF16), ("bf16", F32), ("bf16", F16)]


def check_weights(kind, dtype, heads, kv):
    """Weights to fp32 rounding, whatever type the queries have.  Three positions a
    head: the first of score 0 and value 0; the others, of scores a < 0 and a +
    2^-17 and values 1 and -1, leave the difference of two weights w next to each
    other.  Scores are exact sums.  A weight's error: half a step of its argument
    beside the shift of 15 (2^-21, times ln 2), two ulp of the power of two (2^-22),
    the scale's and the products' rounding (2^-23 of at most 1) and the parts' 2^-23:
    below 2^-20 of it.  The difference is off by that of both weights, over their sum
    and 1, and by the tensor core's sum of three products, 2^-23 each: below 2^-20
    in all; then the output's own rounding."""
    D, page = 64, 16
    shape = (1, kv, page, D)
    k, v = torch.zeros(shape), torch.zeros(shape)
    k[..., 1:3, 0], k[..., 2, 1] = 1.0, 1.0
    v[..., 1, :], v[..., 2, :] = 1.0, -1.0
    if kind == "q8_0":
        scale = torch.full((1, kv, page, D // 32), 2.0 ** -6, dtype=F16, device=DEV)
        cache = bq.PagedKVCache((k * 64).to(torch.int8).to(DEV), (v * 64).to(torch.int8).to(DEV), scale, scale.clone())
    else:
        t = {"f16": F16, "bf16": BF16}[kind]
        cache = bq.PagedKVCache(k.to(t).to(DEV), v.to(t).to(DEV))
    q = torch.zeros((1, heads, D), dtype=torch.float64)
    q[0, :, 0] = -(torch.arange(heads) + 40.0) / 128  # 8 bits or fewer: exact in every type
    q[0, :, 1] = 2.0 ** -17
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    lens = torch.tensor([3], dtype=torch.int32, device=DEV)
    got = bq.paged_attention(cache, q.to(dtype).to(DEV), table, lens, scale=1.0).cpu().double()
    w1, w2 = torch.exp(q[0, :, 0]), torch.exp(q[0, :, 0] + q[0, :, 1])
    want = ((w1 - w2) / (1 + w1 + w2))[None, :, None].expand_as(got)
    bound = 2.0 ** -20 + plain.EPS[dtype] / 2 * (want.abs() + 2.0 ** -20) + (2.0 ** -25 if dtype is F16 else 0.0)
    assert ((got - want).abs() <= bound).all(), float((got - want).abs().max())


@pytest.mark.parametrize("kind,dtype", WEIGHT_KINDS)
@pytest.mark.parametrize("heads,kv", [(48, 48), (48, 6), (48, 4), (48, 1)])
def test_weights_are_good_to_fp32_rounding(kind, dtype, heads, kv):
    check_weights(kind, dtype, heads, kv)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,kv", [(48, 48), (48, 6), (48, 4), (48, 1)])
def test_weights_over_a_q8_0_cache_are_good_to_fp32_rounding(dtype, heads, kv):
    check_weights("q8_0", dtype, heads, kv)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("small", [-2, -8, -14])
def test_small_value_scales_beside_large_ones(dtype, small):
    """A value of a small scale that has nearly all the weight, beside one of scale
    2^10 with a weight of e^-40: off by 2^-23 of itself, and by 2^-39 of the largest
    scale for each of the two codes; then a few fp32 roundings and the output's."""
    D, page = 64, 16
    codes = torch.zeros((1, 1, page, D), dtype=torch.int8, device=DEV)
    k, v = codes.clone(), torch.from_numpy(rng(51).integers(-127, 128, codes.shape).astype(np.int8)).to(DEV)
    k[0, 0, 1, 0] = 40
    scale = torch.ones((1, 1, page, D // 32), dtype=F16, device=DEV)
    v_scale = scale * 2.0 ** 10
    v_scale[0, 0, 1] = 2.0 ** small
    cache = bq.PagedKVCache(k, v, scale, v_scale)
    q = torch.zeros((1, 4, D), dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    out = bq.paged_attention(cache, q, torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                             torch.tensor([2], dtype=torch.int32, device=DEV), scale=1.0).cpu().double()
    x = v[0, 0, :2].cpu().double() * torch.tensor([[2.0 ** 10], [2.0 ** small]], dtype=torch.float64)
    want = (x[0] * np.exp(-40.0) + x[1]) / (1 + np.exp(-40.0))
    off = 2.0 ** -21 * want.abs() + 2.0 ** -39 * 2.0 ** 10 * 2 * 127
    bound = off + plain.EPS[dtype] / 2 * (want.abs() + off) + (2.0 ** -25 if dtype is F16 else 0.0)
    assert ((out - want).abs() <= bound).all(), float((out - want).abs().max())


def test_strided_queries_and_outputs():
    g = rng(8)
    lens, page = [130, 20, 5], 16
    cache = filled_cache(g, "bf16", 16, page, 2, 64)
    table = request_tables(g, lens, page, 16, width=20)[:, :9]  # rows 20 apart
    big = normal(g, (3, 8 * 64 + 100))
    q = big[:, 100:].view(3, 8, 64)
    room = torch.full((3, 9, 80), 7.0, device=DEV)
    out = room[:, 1:, 8:72]
    check_attention(cache, q, table, lens, out=out)
    room[:, 1:, 8:72] = 7.0
    assert (room == 7.0).all()
    heads_apart = normal(g, (8, 3, 64)).transpose(0, 1)
    check_attention(cache, heads_apart, table, lens)


def test_bad_pages_and_lengths_are_masked_and_reported():
    g = rng(9)
    lens, page = [100, 40], 16
    cache = filled_cache(g, "f16", 12, page, 1, 64)
    table = request_tables(g, lens, page, 12)
    q = normal(g, (2, 4, 64))
    clean = bq.paged_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    for entry in (-1, 12, 1 << 30):
        broken = table.clone()
        broken[0, 2] = entry
        out = bq.paged_attention(cache, q, broken, torch.tensor(lens, dtype=torch.int32, device=DEV))
        assert bq.device_status(clear=True) == _lib.BQ_DEVERR_PAGE
        assert torch.equal(out[1], clean[1])
        # positions 32 .. 47 are masked: the same as a request without them
        k, v = plain.values(cache)
        keep = [i for i in range(7) if i != 2]
        want, mag, top = plain.attention(k, v, q[:1].cpu(), table[:1, keep].cpu(), [84], 1, 64 ** -0.5)
        assert ((out[:1].cpu().double() - want).abs() <= plain.attention_bound(want, mag, top, F32, False)).all()
    short = torch.tensor([-3, 40], dtype=torch.int32, device=DEV)
    out = bq.paged_attention(cache, q, table, short)
    assert bq.device_status(clear=True) == _lib.BQ_DEVERR_LENGTH
    assert (out[0] == 0).all() and torch.equal(out[1], clean[1])
    table[0, :] = table[0, 0]  # every entry of the row valid
    out = bq.paged_attention(cache, q, table, torch.tensor([10 ** 6, 40], dtype=torch.int32, device=DEV))
    assert bq.device_status(clear=True) == _lib.BQ_DEVERR_LENGTH
    full = bq.paged_attention(cache, q, table, torch.tensor([table.shape[1] * page, 40], dtype=torch.int32, device=DEV))
    assert torch.equal(out, full)


@pytest.mark.parametrize("kind,dtype,rows", [("f16", F32, 1), ("q8_0", BF16, 3)])
@pytest.mark.parametrize("lens,width", [([40, 70], 8),       # a chunk each
                                        ([1000, 300], 64),   # a cluster's chunks
                                        ([5000, 700], 320),  # many chunks
                                        ([5000] + [900] * 39, 320)])  # few chunks of many requests
def test_a_request_of_bad_pages_alone_gives_zeros(kind, dtype, rows, lens, width):
    """Every position masked: the row sees nothing.  The same with the positions
    after the first 16 valid: the softmax is over those alone."""
    g = rng(kind, rows, width, len(lens))
    page, D, kv, n = 16, 64, 2, len(lens)
    pages = sum(-(-x // page) for x in lens)
    cache = filled_cache(g, kind, pages, page, kv, D)
    table = request_tables(g, lens, page, pages, width)
    q = normal(g, (n * rows, 2 * kv, D), dtype)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean = bq.paged_attention(cache, q, table, at, rows=rows)
    broken = table.clone()
    broken[0] = pages
    out = bq.paged_attention(cache, q, broken, at, rows=rows)
    assert bq.device_status(clear=True) == _lib.BQ_DEVERR_PAGE
    assert (out[:rows] == 0).all() and torch.equal(out[rows:], clean[rows:])
    broken[0] = table[0]
    broken[0, 0] = -1
    out = bq.paged_attention(cache, q, broken, at, rows=rows)
    assert bq.device_status(clear=True) == _lib.BQ_DEVERR_PAGE
    k, v = plain.values(cache)
    want, mag, top = plain.attention(k, v, q[:rows].cpu(), table[:1, 1:].cpu(), [lens[0] - page], rows, D ** -0.5)
    bound = plain.attention_bound(want, mag, top, dtype, kind == "q8_0" and dtype == BF16)
    assert ((out[:rows].cpu().double() - want).abs() <= bound).all()
    assert torch.equal(out[rows:], clean[rows:])


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("lens,page,width,heads,kv,D,rows", [
    ([0, 1, 40, 17] * 1024, 16, 4, 2, 1, 32, 6),     # the most requests and rows
    ([5, 700] * 2048, 64, 40, 1, 1, 32, 1),          # more units than wait for a CTA each
    ([70, 3], 16, 5, 4096, 1024, 32, 1),             # the most heads
    ([200], 65536, 128, 2, 1, 64, 2),                # the widest table, the largest page
    ([200, 4], 1, 1 << 20, 2, 1, 64, 1),             # pages of one position in a wide table
    ([90], 16, 6, 640, 1, 64, 6)])                   # 3840 query rows of one kv head
def test_attention_at_its_limits(kind, lens, page, width, heads, kv, D, rows):
    g = rng(kind, page, width, heads)
    pages = sum(-(-x // page) for x in lens) + 1
    cache = filled_cache(g, kind, pages, page, kv, D)
    table = request_tables(g, lens, page, pages, width)
    check_attention(cache, normal(g, (len(lens) * rows, heads, D)), table, lens, rows=rows)


def test_append_at_its_limits():
    g = rng(25)
    check_append(g, "f16", F16, 3, 4096, 1024, 8, 0, None, False, 65536, 10)
    check_append(g, "q8_0", F32, 2, 4096, 1024, 32, 32, None, False, 1, 10)
    check_append(g, "bf16", F32, 700, 40, 8, 256, 256, [0, 0, 128], True, 16, 10)


def test_a_cache_of_more_than_2_to_31_elements():
    """Offsets that pass 32 bits: the pages in use lie at the end of a 10 GB cache."""
    page, D, pages = 256, 128, 80000
    k = torch.empty((pages, 1, page, D), dtype=F16, device=DEV)
    v = torch.empty_like(k)
    g = rng(10)
    for i in (pages - 1, pages - 3):
        k[i], v[i] = normal(g, (1, page, D), F16), normal(g, (1, page, D), F16)
    cache = bq.PagedKVCache(k, v)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=DEV)
    q = normal(g, (1, 4, D))
    lens = torch.tensor([301], dtype=torch.int32, device=DEV)
    # appended through the same far slots
    new_k, new_v = normal(g, (1, 1, D)), normal(g, (1, 1, D))
    slot = torch.tensor([(pages - 3) * page + 44], dtype=torch.int64, device=DEV)
    assert int(slot) * D > 2 ** 31
    bq.kv_append(cache, new_k, new_v, slot)
    assert torch.equal(k[pages - 3, 0, 44], new_k[0, 0].half())
    out = bq.paged_attention(cache, q, table, lens)
    small = bq.PagedKVCache(k[[pages - 1, pages - 3]], v[[pages - 1, pages - 3]])
    again = bq.paged_attention(small, q, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), lens)
    assert torch.equal(out, again)
    check_attention(small, q, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), [301])


def test_attention_on_a_side_stream_and_in_graphs():
    """A captured call replayed with other lengths, tables and cache contents, two
    graphs with workspaces of their own, and a call on another stream."""
    g = rng(11)
    page, width = 16, 400
    cache = filled_cache(g, "q8_0", 900, page, 2, 64)
    lens_now = [6000, 900]
    table = request_tables(g, lens_now, page, 900, width)
    lens = torch.tensor(lens_now, dtype=torch.int32, device=DEV)
    q = normal(g, (2, 8, 64))
    need = bq.paged_attention_workspace(cache, 2, 1, 8, width)
    assert need > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = bq.paged_attention(cache, q, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(there, bq.paged_attention(cache, q, table, lens))
    graphs = []
    for i in range(2):
        out = torch.empty_like(q)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bq.paged_attention(cache, q, table, lens, out=out, workspace=ws)
        graphs.append((graph, out))
    for n in ([6000, 900], [17, 6400], [0, 5]):
        fresh = request_tables(g, n, page, 900, width)
        table.copy_(fresh)
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        q.copy_(normal(g, (2, 8, 64)))
        torch.cuda.synchronize()
        s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
        for (graph, out), s in zip(graphs, (s0, s1)):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        want = check_attention(cache, q, table, n)
        for _, out in graphs:
            assert torch.equal(out, want)


def test_two_threads_on_one_stream():
    """Calls of two kernels each, launched by two host threads in turn on the
    default stream: each thread's results are those of its calls alone."""
    g = rng(14)
    cache = filled_cache(g, "f16", 400, 16, 2, 64)
    calls = []
    for lens in ([5000, 60], [1000, 5100]):
        table, at = request_tables(g, lens, 16, 400, 320), torch.tensor(lens, dtype=torch.int32, device=DEV)
        q = normal(g, (2, 8, 64))
        calls.append((q, table, at, bq.paged_attention(cache, q, table, at)))
    wrong = [0, 0]

    def work(i):
        q, table, at, want = calls[i]
        got = [bq.paged_attention(cache, q, table, at) for _ in range(300)]
        wrong[i] = sum(not torch.equal(x, want) for x in got)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


@pytest.mark.parametrize("lens,width", [([40, 70], 8), ([1000, 300], 64), ([5000, 700], 320)])
def test_the_output_may_be_the_queries(lens, width):
    g = rng(12, width)
    cache = filled_cache(g, "f16", 400, 16, 2, 64)
    table = request_tables(g, lens, 16, 400, width)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = normal(g, (4, 8, 64), F16)
    want = bq.paged_attention(cache, q, table, at, rows=2)
    assert bq.paged_attention(cache, q, table, at, rows=2, out=q) is q
    assert torch.equal(q, want)


def test_a_capture_that_forks_and_joins():
    """Append and norm on a forked stream, attention after the join (two layers'
    caches), replayed with other inputs: the eager calls' bits."""
    g = rng(13)
    page, width = 16, 320
    caches = [filled_cache(g, "f16", 330, page, 2, 64) for _ in range(2)]
    table = request_tables(g, [5000], page, 330, width)
    lens = torch.tensor([5000], dtype=torch.int32, device=DEV)
    slots = (table[0, 4999 // page].long() * page + 4999 % page).view(1)
    k, v, q, gain = normal(g, (1, 2, 64)), normal(g, (1, 2, 64)), normal(g, (1, 8, 64)), torch.ones(512, device=DEV)

    def step(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            bq.kv_append(caches[0], k, v, slots)
            h, x = bq.sandwich_norm(q.view(1, 512), q.view(1, 512), gain)
        bq.kv_append(caches[1], v, k, slots)
        second = bq.paged_attention(caches[1], q, table, lens)
        main.wait_stream(side)
        first = bq.paged_attention(caches[0], x.view(1, 8, 64), table, lens)
        return h, x, first, second

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        captured = step(side)
    for _ in range(2):
        for t in (k, v, q):
            t.copy_(normal(g, t.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, step(side)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_attention_refusals():
    cache = bq.PagedKVCache.zeros(4, 16, 2, 64)
    table = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 4, 64), device=DEV)
    with pytest.raises(TypeError):
        bq.paged_attention(cache, q.double(), table, lens)
    with pytest.raises(TypeError):
        bq.paged_attention(cache, q, table.long(), lens)
    with pytest.raises(ValueError):
        bq.paged_attention(cache, q, table, lens, rows=2)
    with pytest.raises(ValueError):
        bq.paged_attention(cache, q, table, lens, rows=7)
    with pytest.raises(ValueError):
        bq.paged_attention(cache, q[..., :32], table, lens)
    with pytest.raises(ValueError):
        bq.paged_attention(cache, q.transpose(1, 2).contiguous().transpose(1, 2), table, lens)
    with pytest.raises(ValueError):
        bq.paged_attention(cache, q, table[:, :0], lens)
    with pytest.raises(bq.BQError):
        bq.paged_attention(cache, torch.zeros((1, 3, 64), device=DEV), table, lens)
    with pytest.raises(bq.BQError):
        bq.paged_attention(cache, q, table, lens, scale=float("inf"))
    with pytest.raises(ValueError):
        bq.paged_attention(cache, q, table, lens, out=torch.zeros((2, 4, 64), device=DEV))
    with pytest.raises(ValueError):
        bq.PagedKVCache(cache.k, cache.v[:2])
    with pytest.raises(ValueError):
        bq.PagedKVCache(cache.k, cache.v.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        bq.PagedKVCache(cache.k, cache.v, torch.zeros(1, device=DEV), None)
    with pytest.raises(TypeError):
        bq.PagedKVCache(cache.k.float(), cache.v.float())
    with pytest.raises(ValueError, match="overlaps"):
        bq.PagedKVCache(cache.k[:1].expand(4, -1, -1, -1), cache.v[:1].expand(4, -1, -1, -1))
    with pytest.raises(ValueError, match="overlaps"):
        bq.paged_attention(cache, q, table, lens, out=torch.zeros((1, 1, 64), device=DEV).expand(1, 4, 64))
    # no requests: nothing happens
    assert bq.paged_attention(cache, q[:0], table[:0], lens[:0]).shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def check_append(g, kind, dtype, T, heads, kv, D, rot, sections, interleaved, page, far, layout="hs", fused=True,
                 in_place=False, skip=()):
    pages = -(-T // page) + 3
    cache = bq.PagedKVCache.zeros(pages, page, kv, D, kind)
    if layout != "hs":
        cache = filled_cache(g, kind, pages, page, kv, D, layout)
        for t in (cache.k, cache.v) + (() if cache.k_scale is None else (cache.k_scale, cache.v_scale)):
            t.zero_()
    order = g.permutation(pages * page)[:T].astype(np.int64)
    order[list(skip)] = -1 - np.arange(len(skip))
    slots = torch.from_numpy(order).to(DEV)
    if fused:
        qkv = normal(g, (T, (heads + 2 * kv) * D), dtype)
        q, k, v = (t.view(T, -1, D) for t in qkv.split([heads * D, kv * D, kv * D], dim=1))
    else:
        q, k, v = (normal(g, (T, n, D), dtype) for n in (heads, kv, kv))
    rope = positions = None
    if rot:
        freq = torch.from_numpy(1e4 ** (-np.arange(rot // 2) * 2.0 / rot))
        rope = bq.Rope(freq.to(DEV), sections, interleaved)
        positions = torch.from_numpy(g.integers(0, far, (rope.axes, T)).astype(np.int32))
        positions[:, 0] = far - 1
        positions[:, -1] = -positions[:, -1]
    q0, k0, v0 = q.cpu().clone(), k.cpu().clone(), v.cpu().clone()
    out = bq.kv_append(cache, k, v, slots, q=q, q_out=q if in_place else None, rope=rope,
                       positions=None if rope is None else positions.to(DEV))
    if rot:
        wq, bqd = plain.turn(q0, freq, rope.sections, positions, interleaved)
        wk, bkd = plain.turn(k0, freq, rope.sections, positions, interleaved)
    else:
        wq, wk = q0.double(), k0.double()
        bqd, bkd = torch.zeros_like(wq), torch.zeros_like(wk)
    err = (out.cpu().double() - wq).abs()
    # halves of a unit of the output's type, and of fp16's smallest subnormal
    assert (err <= bqd + plain.EPS[dtype] / 2 * (wq.abs() + bqd) + 2.0 ** -25).all(), float(err.max())
    gk, gv = plain.values(cache)
    flat = [t.transpose(1, 2).reshape(-1, kv, D) for t in (gk, gv)]
    stored = [t for t in range(T) if order[t] >= 0]
    at = torch.from_numpy(order[stored])
    for got, want, bound in ((flat[0][at], wk[stored], bkd[stored]), (flat[1][at], v0.double()[stored], 0.0)):
        err = (got - want).abs()
        if kind == "q8_0":
            # a code is off by half a step at most, the scale by half an fp16 unit of max / 127
            top = want.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
            step = top / 127 * (1 + 2.0 ** -10) + 2.0 ** -24
            assert (err <= bound + step * (0.5 + 127 * 2.0 ** -10)).all()
        else:
            eps = plain.EPS[F16 if kind == "f16" else BF16]
            assert (err <= bound + eps / 2 * (want.abs() + bound) + 2.0 ** -25).all()
    if kind == "q8_0":  # values are not rotated: their blocks are bq_quantize_pack's
        codes, scale = plain.q8(v0.float().numpy()[stored])
        gc = cache.v.cpu().transpose(1, 2).reshape(-1, kv, D)[at].numpy()
        gs = cache.v_scale.cpu().transpose(1, 2).reshape(-1, kv, D // 32)[at].numpy()
        assert np.array_equal(gc, codes) and np.array_equal(gs.view(np.uint16), scale.view(np.uint16))
        packed = bq.quantize_pack(v0.float()[stored].reshape(-1, D).to(DEV), "q8_0").cpu().numpy().reshape(-1, D // 32, 34)
        assert np.array_equal(packed[..., 2:].view(np.int8).reshape(codes.shape), codes)
        assert np.array_equal(packed[..., :2].copy().view(np.uint16).reshape(scale.shape), scale.view(np.uint16))
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[at] = False
    assert (flat[0][rest] == 0).all() and (flat[1][rest] == 0).all()
    return cache


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,heads,kv,D,rot,sections,interleaved", [
    (1, 16, 4, 128, 128, None, False), (7, 14, 2, 64, 64, [8, 12, 12], False), (33, 6, 2, 96, 96, None, False),
    (5, 3, 1, 256, 256, [32, 48, 48], False), (9, 4, 4, 128, 64, None, True), (3, 5, 5, 32, 32, [16], True),
    (600, 8, 2, 64, 32, None, False), (2, 2, 1, 160, 96, [0, 48], False), (4, 2, 2, 64, 0, None, False)])
def test_append(kind, dtype, T, heads, kv, D, rot, sections, interleaved):
    g = rng(kind, str(dtype), T, D)
    check_append(g, kind, dtype, T, heads, kv, D, rot, sections, interleaved, 16, 5000)


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("q8_0", BF16)])
def test_append_far_positions_layouts_and_skipped_tokens(kind, dtype):
    g = rng(kind, 21)
    check_append(g, kind, dtype, 40, 4, 2, 64, 64, None, False, 24, 2 ** 31 - 1)
    check_append(g, kind, dtype, 40, 4, 2, 64, 64, None, False, 7, 10 ** 6, layout="sh", fused=False)
    check_append(g, kind, dtype, 40, 4, 2, 64, 64, None, True, 1, 100, layout="kv", in_place=True)
    check_append(g, kind, dtype, 40, 4, 2, 64, 64, None, False, 16, 100, skip=(0, 5, 39))
    check_append(g, kind, dtype, 5000, 4, 2, 64, 64, None, False, 16, 100, fused=False)


@pytest.mark.parametrize("far", [2 ** 24 + 3, 2 ** 26, 2 ** 31 - 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_many_far_positions(far, interleaved):
    """Enough positions to meet the ones whose remainder beyond 24 bits is largest."""
    check_append(rng(far, 26), "f16", F32, 4000, 4, 2, 64, 64, [8, 24], interleaved, 16, far)


def test_append_odd_alignment_and_no_queries():
    g = rng(22)
    cache = bq.PagedKVCache.zeros(4, 16, 2, 64)
    room = normal(g, (10, 2 * 64 + 3), F16)
    k = room[:, 3:].view(10, 2, 64)  # rows start at odd elements
    v = normal(g, (10, 2, 64), F16)
    slots = torch.arange(10, device=DEV) + 20
    assert bq.kv_append(cache, k, v, slots) is None
    flat = cache.k.transpose(1, 2).reshape(64, 2, 64)
    assert torch.equal(flat[20:30], k) and torch.equal(cache.v.transpose(1, 2).reshape(64, 2, 64)[20:30], v)
    assert (flat[:20] == 0).all() and (flat[30:] == 0).all()
    bq.kv_append(cache, k[:0], v[:0], slots[:0])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D", [32, 96, 128, 256])
def test_append_of_any_value_packs_as_the_weights_do(dtype, D):
    """Q8_0 blocks with NaN (of either sign), infinities, zeros, values too small
    for an fp16 scale and halfway values: bq_quantize_pack's blocks, bit for bit."""
    g = rng(24, D, str(dtype))
    T, kv = 40, 2
    x = normal(g, (T, kv, D), dtype)
    x[0] = float("nan")
    x[1, :, ::5], x[2, :, ::7], x[3, :, 1::9] = float("nan"), float("inf"), float("-inf")
    x[4, :, ::3] = -x[0, :, ::3]
    x[5] = 0
    x[6], x[7, :, 3] = 0, float("nan")
    x[6, :, 0] = float("nan")
    x[8] *= 1e-7
    x[9] = torch.arange(D, device=DEV) % 32 - 15.5
    x[10, :, ::32] = 127
    x[10, :, 1::32] = 0.5
    if dtype is not F16:
        x[11] *= 1e9  # the scale is infinite
        x[12] *= 1e-30
    cache = bq.PagedKVCache.zeros(3, 16, kv, D, "q8_0")
    bq.kv_append(cache, x, x.flip(0), torch.arange(T, device=DEV))
    for codes, scales, want in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, x.flip(0))):
        packed = bq.quantize_pack(want.float().reshape(-1, D).contiguous(), "q8_0").cpu().numpy().reshape(T, kv, D // 32, 34)
        got = codes.transpose(1, 2).reshape(48, kv, D)[:T].cpu().numpy()
        scale = scales.transpose(1, 2).reshape(48, kv, D // 32)[:T].cpu().numpy()
        assert np.array_equal(scale.view(np.uint16), packed[..., :2].copy().view(np.uint16)[..., 0])
        assert np.array_equal(got, packed[..., 2:].view(np.int8).reshape(got.shape))


def test_append_slots_beyond_the_pool_are_reported():
    g = rng(23)
    cache = bq.PagedKVCache.zeros(2, 16, 1, 64)
    k = normal(g, (3, 1, 64))
    slots = torch.tensor([32, 5, 2 ** 40], dtype=torch.int64, device=DEV)
    q = normal(g, (3, 2, 64))
    out = bq.kv_append(cache, k, k, slots, q=q)
    assert bq.device_status(clear=True) == _lib.BQ_DEVERR_SLOT
    assert torch.equal(out, q)
    assert torch.equal(cache.k[0, 0, 5], k[1, 0].half())
    cache.k[0, 0, 5] = 0
    assert (cache.k == 0).all()


def test_append_refusals():
    cache = bq.PagedKVCache.zeros(2, 16, 1, 64)
    k, slots = torch.zeros((2, 1, 64), device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    rope = bq.Rope.from_theta(64, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k[:1], slots)
    with pytest.raises(TypeError):
        bq.kv_append(cache, k, k.half(), slots)
    with pytest.raises(TypeError):
        bq.kv_append(cache, k, k, slots.int())
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k, slots, q_out=k)
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k, slots, positions=pos)
    with pytest.raises(TypeError):
        bq.kv_append(cache, k, k, slots, rope=rope)
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k, slots, rope=rope, positions=pos[:1])
    with pytest.raises(bq.BQError):  # more rotated values than a head has
        bq.kv_append(cache, k, k, slots, rope=bq.Rope.from_theta(128, device=DEV), positions=pos)
    with pytest.raises(ValueError):
        bq.Rope.from_theta(24, device=DEV)
    with pytest.raises(ValueError):
        bq.Rope.from_theta(64, sections=[16, 8], device=DEV)


# ---------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------
def check_tables(lens, new, page, width, pool, room, g, count=None, in_place=False, free=None, table=None):
    lens, new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
    held = [-(-int(n) // page) if 0 <= n <= width * page else 0 for n in lens]
    order = g.permutation(pool).astype(np.int32)
    if table is None:
        table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        assert at <= pool
        free = np.full(pool, -9, np.int32)
        free[:pool - at] = order[at:]
        count = pool - at if count is None else count
    want = plain.block_tables(lens, new, table, free, count, page, room)
    d = {n: torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for n, x in dict(
        lens=lens, new=new, table=table, free=free, count=np.array([count], np.int32)).items()}
    slots = torch.full((room,), 99, dtype=torch.int64, device=DEV)
    positions = torch.full((room,), 99, dtype=torch.int32, device=DEV)
    starts = torch.full((len(lens) + 1,), 99, dtype=torch.int32, device=DEV)
    outs = {} if in_place else dict(lens_out=torch.empty_like(d["lens"]), free_count_out=torch.empty_like(d["count"]))
    refused = bq.kv_block_tables(d["lens"], d["new"], d["table"], d["free"], d["count"], page, slots, positions, starts,
                                 **outs)
    got = (d["table"], d["free"], slots, positions, starts, outs.get("lens_out", d["lens"]),
           outs.get("free_count_out", d["count"]), refused)
    names = ("table", "free", "slots", "positions", "starts", "lens", "count", "refused")
    for name, a, b in zip(names, got, want):
        assert np.array_equal(a.cpu().numpy().reshape(np.shape(b)), b), name
    if not in_place:
        assert np.array_equal(d["lens"].cpu().numpy(), lens) and int(d["count"]) == count
    return want


@pytest.mark.parametrize("n", [0, 1, 2, 31, 33, 513, 1500, 4096])
@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("in_place", [False, True])
def test_block_tables(n, page, in_place):
    """Requests that grow by one token, start with a prompt, shrink or end, with
    few token rows (one launch) and many (two)."""
    g = rng(n, page)
    old = g.integers(0, 200, n)
    new = np.where(g.random(n) < 0.2, g.integers(0, 200, n), old + 1)
    new[g.random(n) < 0.1] = 0
    width = -(-202 // page) + 1
    pool = int(sum(-(-int(max(a, z)) // page) for a, z in zip(old, new))) + 5
    rows = int(np.maximum(new - old, 0).sum())
    want = check_tables(old, new, page, width, pool, rows + 9, g, in_place=in_place)
    assert want[-1] == 0
    check_tables(old, new, page, width, pool, rows + 6000, g, in_place=in_place)


def test_block_tables_of_every_shared_memory_size():
    """Around the request counts whose shared memory passes 48 KB (with the kernel's
    static part, 2437 and more), in a process that has made no larger call."""
    code = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
import test_gpu_cache as t
g = t.rng(34)
for n in (2405, 2406, 2407, 2436, 2437, 2440, 2456, 2457, 2458):
    old = g.integers(0, 40, n)
    new = np.where(g.random(n) < 0.9, old + 1, 0)
    t.check_tables(old, new, 16, 4, 4 * n, n, g)
print("fine")
"""
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code.format(root=os.path.dirname(tests), tests=tests)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("seed", range(6))
def test_block_tables_refuse_what_does_not_fit(seed):
    g = rng(seed, 31)
    n, page, width = 40, 8, 12
    old = g.integers(0, 60, n)
    new = np.clip(old + g.integers(-30, 60, n), 0, width * page + 20)
    old[3], new[5], new[7] = -2, -1, width * page + 1  # lengths out of range
    held = sum(-(-int(a) // page) for a in old if 0 <= a <= width * page)
    pool = held + [0, 5, 20, 100, 100, 40][seed]
    rows = int(np.maximum(new - old, 0).sum())
    want = check_tables(old, new, page, width, pool, [rows, rows, rows, rows // 3, 0, 7][seed], g)
    assert want[-1] > 0


def test_block_tables_of_a_broken_stack():
    """A free count outside the pool counts as the nearest, a push beyond the pool
    is dropped, and both are reported."""
    i32 = dict(dtype=torch.int32, device=DEV)
    for count, left, stack in ((-3, 2, [4, 5, 8, 8]), (99, 4, [8, 8, 8, 8]), (3, 4, [8, 8, 8, 4])):
        lens = torch.tensor([17, 5], **i32)
        free, out = torch.full((4,), 8, **i32), torch.tensor([count], **i32)
        slots, positions, starts = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(2, **i32), torch.zeros(3, **i32)
        table = torch.tensor([[4, 5], [6, 7]], **i32)
        refused = bq.kv_block_tables(lens, torch.tensor([0, 6], **i32), table, free, out, 16, slots, positions, starts)
        assert bq.device_status(clear=True) == _lib.BQ_DEVERR_POOL
        assert int(refused) == 0 and lens.tolist() == [0, 6] and int(out) == left and free.tolist() == stack
        assert slots.tolist() == [6 * 16 + 5, -1] and positions.tolist() == [5, 0] and starts.tolist() == [0, 0, 1]


def test_block_tables_step_by_step_keep_every_page():
    """Many steps of a server in a captured graph: no page is lost or held twice."""
    g = rng(33)
    requests, pages, page = 24, 90, 8
    t = bq.BlockTables(requests, 30, pages, page, 64)
    goal = torch.zeros(requests, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    t.resize(goal)
    with torch.cuda.graph(graph):
        t.resize(goal)
    refused = 0
    for step in range(60):
        lens = t.lens.cpu().numpy()
        want = lens + (g.random(requests) < 0.8)
        fresh = (lens == 0) & (g.random(requests) < 0.3)
        want[fresh] = g.integers(1, 40, fresh.sum())
        want[g.random(requests) < 0.05] = 0
        goal.copy_(torch.from_numpy(want.astype(np.int32)))
        before = (lens, want, t.table.cpu().numpy(), t.free_pages.cpu().numpy(), int(t.free_count))
        graph.replay()
        told = plain.block_tables(before[0], before[1], before[2], before[3], before[4], page, 64)
        for a, b in zip((t.table, t.free_pages, t.slots, t.positions, t.starts, t.lens), told):
            assert np.array_equal(a.cpu().numpy(), b)
        assert int(t.free_count) == told[6] and int(t.refused) == told[7]
        refused += told[7]
        now = t.lens.cpu().numpy()
        used = [p for b in range(requests) for p in t.table[b, :-(-int(now[b]) // page)].tolist()]
        used += t.free_pages[:int(t.free_count)].tolist()
        assert sorted(used) == list(range(pages))
    assert refused > 0


def test_lengths_may_not_be_written_over_the_lengths_asked():
    i32 = dict(dtype=torch.int32, device=DEV)
    new = torch.zeros(2, **i32)
    with pytest.raises(bq.BQError):
        bq.kv_block_tables(torch.zeros(2, **i32), new, torch.zeros((2, 4), **i32), torch.zeros(8, **i32),
                           torch.zeros(1, **i32), 16, torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, **i32),
                           torch.zeros(3, **i32), lens_out=new)


def test_block_table_refusals():
    i32 = dict(dtype=torch.int32, device=DEV)
    good = dict(lens=torch.zeros(2, **i32), new_lens=torch.zeros(2, **i32), table=torch.zeros((2, 4), **i32),
                free_pages=torch.zeros(8, **i32), free_count=torch.zeros(1, **i32), page_size=16,
                slots=torch.zeros(4, dtype=torch.int64, device=DEV), positions=torch.zeros(4, **i32),
                starts=torch.zeros(3, **i32))
    bq.kv_block_tables(**good)
    for name, value, error in (("new_lens", torch.zeros(3, **i32), ValueError), ("lens", torch.zeros(2, device=DEV), TypeError),
                               ("table", torch.zeros((3, 4), **i32), ValueError),
                               ("starts", torch.zeros(2, **i32), ValueError),
                               ("positions", torch.zeros(5, **i32), ValueError), ("page_size", 0, bq.BQError),
                               ("free_count", torch.zeros(2, **i32), ValueError),
                               ("slots", torch.zeros(4, **i32), TypeError)):
        with pytest.raises(error):
            bq.kv_block_tables(**{**good, name: value})


def test_a_page_size_beyond_32_bits_is_refused():
    t = bq.BlockTables(2, 4, 8, (1 << 32) + 16, 8)
    with pytest.raises(bq.BQError):
        t.resize(torch.ones(2, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_a_server_step_by_step(kind):
    """Prompts, decode steps and an ending request through block tables, append
    and attention; every step's attention against a plain history that each
    request keeps outside the pages."""
    g = rng(kind, 41)
    requests, heads, kv, D, page = 3, 8, 2, 64, 16
    t = bq.BlockTables(requests, 12, 24, page, 128)
    cache = bq.PagedKVCache.zeros(24, page, kv, D, kind)
    rope = bq.Rope.from_theta(D, device=DEV)
    told = [[] for _ in range(requests)]
    for goal in ([20, 0, 3], [21, 50, 4], [22, 51, 0], [23, 52, 30], [0, 53, 31], [100, 54, 32]):
        lens = t.lens.cpu().tolist()
        assert int(t.resize(torch.tensor(goal, dtype=torch.int32, device=DEV))) == 0
        n = int(t.starts[-1])
        room = t.slots.numel()  # rows behind the last token are skipped by their slots
        k, v, q = normal(g, (room, kv, D)), normal(g, (room, kv, D)), normal(g, (room, heads, D))
        turned = bq.kv_append(cache, k, v, t.slots, q=q, rope=rope, positions=t.positions)
        gk, gv = plain.values(cache)
        wk, _ = plain.turn(k.cpu(), rope.freq.cpu(), rope.sections, t.positions.cpu()[None], False)
        for b in range(requests):
            told[b] = told[b][:goal[b]]
            for i in range(int(t.starts[b]), int(t.starts[b + 1])):
                told[b].append((wk[i], v[i].cpu().double()))
            assert len(told[b]) == goal[b] == int(t.lens[b])
            for p, (a, z) in enumerate(told[b]):  # the cache holds each request's history
                at = (int(t.table[b, p // page]), slice(None), p % page)
                tol = 2.0 ** -10 if kind == "f16" else 1.0 / 120
                assert ((gk[at] - a).abs() <= tol * a.abs().amax() + 1e-5).all()
                assert ((gv[at] - z).abs() <= tol * z.abs().amax() + 1e-5).all()
        last = (t.starts[1:].long() - 1).clamp(min=0)
        check_attention(cache, turned[last].contiguous(), t.table, t.lens.tolist())
        assert lens is not None and n == sum(max(0, z - a) for a, z in zip(lens, goal))


def test_the_example_of_the_readme():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        code = re.search(r"```python\n(.*?)```", f.read(), flags=re.S).group(1)
    said = {}
    exec(code, said)
    n = said["requests"]
    assert said["tables"].lens.tolist() == [1] * n and int(said["refused"]) == 0
    # one position: its value, as the cache holds it
    v = plain.values(said["cache"])[1]
    for b in range(n):
        row = v[int(said["tables"].table[b, 0]), :, 0].repeat_interleave(said["heads"] // said["kv_heads"], 0)
        assert ((said["out"][b].cpu().double() - row).abs() <= 2.0 ** -20 * row.abs()).all()
    assert torch.isfinite(said["h"]).all() and torch.isfinite(said["x"]).all()
