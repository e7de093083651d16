"""How exactly paged_prefix_attention computes what its requests share: weights that
nearly cancel, and sums of thousands of positions next to a rounding border of the
output, against the 64-bit form."""
import ctypes

import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import _lib

import paged_plain as plain
from test_gpu_cache import BF16, DEV, F16, F32, healthy, normal, rng  # noqa: F401

pytestmark = pytest.mark.gpu

# what the shared pages go through the tensor cores for, whatever the caller's types
PATHS = [("f16", F16), ("f16", F32), ("bf16", BF16), ("bf16", F32), ("q8_0", F32), ("q8_0", BF16)]


@pytest.fixture(autouse=True)
def shared_always():
    hook = _lib.lib.bq_internal_prefix_whole_limit
    hook.restype, hook.argtypes = ctypes.c_int64, [ctypes.c_int64]
    hook(0)
    yield
    hook(-1)


def cache_of(kind, k, v):
    """Float64 pages of values, each on the type's grid (Q8_0: a scale of 2^-6)."""
    if kind != "q8_0":
        return bq.PagedKVCache(*[torch.from_numpy(x).to({"f16": F16, "bf16": BF16}[kind]).to(DEV) for x in (k, v)])
    codes = [torch.from_numpy(np.rint(x * 64).astype(np.int8)).to(DEV) for x in (k, v)]
    scales = [torch.full(c.shape[:3] + (c.shape[3] // 32,), 2.0 ** -6, dtype=F16, device=DEV) for c in codes]
    return bq.PagedKVCache(*codes, *scales)


def half_step(x, dtype):
    """Half the distance of the type's numbers at x: what one rounding is off by."""
    return plain.EPS[dtype] / 2 * 2.0 ** torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14)))


def held(got, want, dtype, off):
    err = (got.double() - want).abs()
    bound = off + half_step(want.abs() + off, dtype)
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside the bound; the worst at {float((err / bound).max())} of it"


@pytest.mark.parametrize("kind,dtype", PATHS)
def test_weights_that_nearly_cancel(kind, dtype):
    """Request b gives the odd positions a weight w_b beside the even ones' 1, and value d
    is 1 at even ones and -1 / w_d on average at odd ones (two neighbours of the type's
    grid): so output d of request d is next to nothing but the error of w_d."""
    g = rng("cancel", kind, str(dtype))
    D, page, n = 64, 16, 2048
    pages = n // page + D
    a = torch.from_numpy(0.1 + 0.55 * (np.arange(D) + g.random(D)) / D).to(dtype)
    target = -np.exp(a.double().numpy())
    step = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7, "q8_0": 2.0 ** -6}[kind]
    k, v = np.zeros((n, D)), np.ones((n, D))
    k[1::2, 0] = 1.0
    for d in range(D):
        low = np.floor(target[d] / step) * step
        v[1::2, d] = low + step * (g.permutation(n // 2) < round((target[d] - low) / step * (n // 2)))
    order = g.permutation(pages)
    table = np.empty((D, n // page + 1), np.int32)
    table[:, :-1] = order[:n // page]
    table[:, -1] = order[n // page:]
    both = []
    for x in (k, v):
        whole = np.zeros((pages, 1, page, D))  # (each request's own position: key and value 0)
        whole[order[:n // page], 0] = x.reshape(-1, page, D)
        both.append(whole)
    cache = cache_of(kind, *both)
    q = torch.zeros(D, 1, D, dtype=dtype, device=DEV)
    q[:, 0, 0] = -a.to(DEV)
    table = torch.from_numpy(table).to(DEV)
    out = bq.paged_prefix_attention(cache, q, table, torch.full((D,), n + 1, dtype=torch.int32, device=DEV), n, scale=1.0)
    want, mag, _ = plain.attention(*plain.values(cache), q.cpu(), table.cpu(), [n + 1] * D, 1, 1.0)
    assert float(want[range(D), 0, range(D)].abs().max()) < 2.0 ** -14
    # A weight: its exponent, below 8, rounded (2^-22), from scores below 1 whose queries and
    # factor are right to 2^-22 and 2^-24, times ln 2; the power's 2^-22; its parts' 2^-23.
    # In all 2^-20.7; the sums, which stay small, 2^-23 of the magnitudes.
    held(out.cpu(), want, dtype, 2.0 ** -20 * mag)


@pytest.mark.parametrize("kind,dtype", PATHS)
def test_long_sums_next_to_a_border_of_the_output(kind, dtype):
    """Values 1 and one step of the grid above, half of them (a quarter): the outputs lie
    about a border between two of the type's numbers, and a sum that loses a little is
    seen. As many rows as give chunks of the most positions."""
    g = rng("border", kind, str(dtype))
    D, page, n, requests, kv, G = 64, 32, 8192, 100, 16, 20
    whole = n // page
    pages = whole + requests
    step = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7, "q8_0": 2.0 ** -6}[kind]
    v = 1.0 + step * (g.random((pages, kv, page, D)) < (0.25 if kind == "q8_0" else 0.5))
    k = g.standard_normal((pages, kv, page, D)).clip(-1.9, 1.9)
    if kind == "q8_0":
        k = np.rint(k * 64) / 64
    cache = cache_of(kind, k, v)
    table = torch.arange(whole, dtype=torch.int32).expand(requests, -1)
    table = torch.cat([table, whole + torch.arange(requests, dtype=torch.int32)[:, None]], 1).to(DEV)
    q = normal(g, (requests, kv * G, D), dtype)
    lens = [n + 1 + b % page for b in range(requests)]
    out = bq.paged_prefix_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV), n)
    kk, vv = (x.to(DEV) for x in plain.values(cache))
    want, mag, _ = plain.attention(kk, vv, q, table, lens, 1, D ** -0.5)
    # O is added up in fp32 every 256 positions, every 512 for 16-bit queries over fp16 or
    # Q8_0; until then the tensor cores add 16 positions' products of each part of the weights
    # (two, three of bf16; over Q8_0 three products): the sum of the products and the running
    # sum, half of the last one on average, lose a unit of 2^-23 each. The weights' own sum
    # and the joins: under 32 roundings of 2^-24.
    adds = (256 if dtype == F32 or kind == "bf16" else 512) // 16 * (2 if kind == "f16" else 3)
    held(out, want, dtype, (adds * 2.0 ** -23 + 2.0 ** -19) * mag)


@pytest.mark.parametrize("kind,dtype", PATHS)
def test_weights_far_below_the_largest(kind, dtype):
    """One position of each request's row takes e^9 to e^12 times the weight of any other
    and has value 0, so that the outputs are what the small weights make of it. As many kv
    heads as the GPU has places: all positions are one chunk."""
    g = rng("sink", kind, str(dtype))
    D, page, n, kv, requests = 64, 16, 2048, 152, 40
    whole = n // page
    k, v = np.zeros((whole + requests, kv, page, D)), np.ones((whole + requests, kv, page, D))
    k[1, :, 5, 0], v[1, :, 5] = 1.0, 0.0
    cache = cache_of(kind, k, v)
    table = torch.arange(whole, dtype=torch.int32).expand(requests, -1)
    table = torch.cat([table, whole + torch.arange(requests, dtype=torch.int32)[:, None]], 1).to(DEV)
    q = torch.zeros(requests, kv, D, dtype=dtype, device=DEV)
    q[:, :, 0] = torch.from_numpy(9.0 + 3.0 * g.random((requests, kv))).to(dtype).to(DEV)
    out = bq.paged_prefix_attention(cache, q, table, torch.full((requests,), n + 1, dtype=torch.int32, device=DEV), n,
                                    scale=1.0)
    want = ((n - 1 + 1) / (q[:, :, :1].double().exp() + n)).expand(-1, -1, D)
    # A small weight beside the large one: an exponent of at most 18 of a factor right to
    # 2^-23 and rounded twice at 2^-21, times ln 2; two powers of 2^-22; parts of 2^-23, and
    # for fp32 queries at most 2^-36 of the largest weight, of which it is 2^-17.4 or more
    # (2^-32 for others). Sums: under 32 roundings of 2^-24, and 2^-18 for what the tensor
    # cores lose of them (the reckoning of the test above, of 48 additions).
    rel = np.log(2.0) * (18 * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -21 + 2.0 ** -23 + 2.0 ** -19
    rel += (48 if dtype == F32 or kind == "bf16" else 96) * 2.0 ** -23
    rel += 0.0 if kind == "bf16" else 2.0 ** (17.4 - (36 if dtype == F32 else 32))
    held(out, want, dtype, rel * want)
