"""The append with norms of queries and keys per head (kv_append's q_norm and
k_norm) against a plain 64-bit form, and its relation to the append without."""
import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import workloads as wl

import paged_plain as plain
from test_gpu_cache import BF16, DEV, F16, F32, filled_cache, healthy, normal, rng  # noqa: F401
from test_gpu_paged_decode import D as DEC_D, decoder, run as decode

pytestmark = pytest.mark.gpu


def normed(x, gain, eps):
    """x [tokens, heads, D] normed per head in float64 and the error of the fp32
    form: the sum of squares takes 8 roundings in a lane and 5 in the butterfly
    (13 * 2^-24 of a sum of one sign), the mean and eps 2; the root halves them:
    2^-20.  The reciprocal root is off by 2^-22, the two products by 2^-23 in all:
    below 2^-19 of the result."""
    x = x.double()
    if gain is None:
        return x, torch.zeros_like(x)
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double()
    return y, 2.0 ** -19 * y.abs()


def turned(x, off, freq, sections, positions, interleaved):
    """normed heads turned, and their bound: an error of a pair moves both of its
    values by at most its magnitudes' sum."""
    if freq is None:
        return x, off
    y, bound = plain.turn(x, freq, sections, positions, interleaved)
    moved = off.clone()
    half = freq.numel()
    e, o = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    moved[..., e] = moved[..., o] = off[..., e] + off[..., o]
    return y, bound + moved


def check(g, kind, dtype, T, heads, kv, D, rot, sections, interleaved, which="qk", eps=1e-6, page=16, layout="hs",
          fused=True, in_place=False, far=5000, scale=1.0, x=None):
    pages = -(-T // page) + 2
    cache = bq.PagedKVCache.zeros(pages, page, kv, D, kind)
    if layout != "hs":
        cache = filled_cache(g, kind, pages, page, kv, D, layout)
        for t in (cache.k, cache.v) + (() if cache.k_scale is None else (cache.k_scale, cache.v_scale)):
            t.zero_()
    order = g.permutation(pages * page)[:T].astype(np.int64)
    slots = torch.from_numpy(order).to(DEV)
    if fused:
        qkv = normal(g, (T, (heads + 2 * kv) * D)).mul(scale).to(dtype)
        if x is not None:
            qkv.fill_(x)
        q, k, v = (t.view(T, -1, D) for t in qkv.split([heads * D, kv * D, kv * D], dim=1))
    else:
        q, k, v = (normal(g, (T, n, D)).mul(scale).to(dtype) for n in (heads, kv, kv))
    gains = [1 + 0.3 * normal(g, (D,)) if n in which else None for n in "qk"]
    rope = positions = freq = None
    if rot:
        freq = torch.from_numpy(1e4 ** (-np.arange(rot // 2) * 2.0 / rot))
        rope = bq.Rope(freq.to(DEV), sections, interleaved)
        positions = torch.from_numpy(g.integers(0, far, (rope.axes, T)).astype(np.int32))
    q0, k0, v0 = q.cpu().clone(), k.cpu().clone(), v.cpu().clone()
    out = bq.kv_append(cache, k, v, slots, q=q, q_out=q if in_place else None, rope=rope,
                       positions=None if rope is None else positions.to(DEV), q_norm=gains[0], k_norm=gains[1], eps=eps)
    sec = None if rope is None else rope.sections
    cpu = [None if t is None else t.cpu() for t in gains]
    wq, oq = turned(*normed(q0, cpu[0], eps), freq, sec, positions, interleaved)
    wk, ok = turned(*normed(k0, cpu[1], eps), freq, sec, positions, interleaved)
    err = (out.cpu().double() - wq).abs()
    assert (err <= oq + plain.EPS[dtype] / 2 * (wq.abs() + oq) + 2.0 ** -25).all(), float(err.max())
    gk, gv = plain.values(cache)
    flat = [t.transpose(1, 2).reshape(-1, kv, D) for t in (gk, gv)]
    at = torch.from_numpy(order)
    for got, want, bound in ((flat[0][at], wk, ok), (flat[1][at], v0.double(), 0.0)):
        err = (got - want).abs()
        if kind == "q8_0":
            top = want.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
            step = top / 127 * (1 + 2.0 ** -10) + 2.0 ** -24
            assert (err <= bound + step * (0.5 + 127 * 2.0 ** -10)).all()
        else:
            half = plain.EPS[F16 if kind == "f16" else BF16] / 2
            assert (err <= bound + half * (want.abs() + bound) + 2.0 ** -25).all()
    return out, cache


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,heads,kv,D,rot,sections,interleaved", [
    (1, 16, 8, 128, 128, None, False), (7, 14, 2, 64, 64, [8, 12, 12], False), (33, 6, 2, 96, 96, None, False),
    (5, 3, 1, 256, 256, [32, 48, 48], False), (9, 4, 4, 128, 64, None, True), (3, 5, 5, 32, 32, [16], True),
    (600, 8, 2, 64, 32, None, False), (2, 2, 1, 160, 96, [0, 48], False), (4, 2, 2, 64, 0, None, False)])
def test_norm_and_append(kind, dtype, T, heads, kv, D, rot, sections, interleaved):
    check(rng("n", kind, str(dtype), T, D), kind, dtype, T, heads, kv, D, rot, sections, interleaved)


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("q8_0", BF16)])
@pytest.mark.parametrize("which", ["q", "k"])
def test_one_norm_alone(kind, dtype, which):
    check(rng("one", kind, which), kind, dtype, 19, 6, 3, 64, 64, None, False, which=which)


@pytest.mark.parametrize("kind,dtype", [("f16", F32), ("bf16", BF16), ("q8_0", F32)])
def test_layouts_places_and_sizes(kind, dtype):
    g = rng("lay", kind)
    check(g, kind, dtype, 40, 4, 2, 64, 64, None, False, page=7, layout="sh", fused=False)
    check(g, kind, dtype, 40, 4, 2, 64, 64, None, True, page=1, layout="kv", in_place=True)
    check(g, kind, dtype, 5000, 4, 2, 64, 64, None, False, fused=False)
    check(g, kind, dtype, 3, 700, 300, 32, 32, None, False, page=24)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_small_values_zeros_and_a_large_eps(dtype):
    """eps decides where a head is small: zeros stay zeros, and with eps 0 a head of
    small values is still normed."""
    g = rng("small")
    check(g, "f16", dtype, 9, 4, 2, 64, 64, None, False, scale=2.0 ** -12)
    check(g, "f16", dtype, 9, 4, 2, 64, 64, None, False, scale=2.0 ** -12, eps=0.0)
    check(g, "f16", dtype, 9, 4, 2, 64, 64, None, False, eps=3.0)
    out, cache = check(g, "f16", dtype, 9, 4, 2, 64, 64, None, False, x=0.0)
    assert (out == 0).all() and (cache.k == 0).all()


def test_heads_beside_one_that_is_not_finite():
    """A NaN or an infinity stays within its head."""
    g = rng("nan")
    q, k = normal(g, (6, 4, 64)), normal(g, (6, 2, 64))
    gain = 1 + 0.1 * normal(g, (64,))
    slots = torch.arange(6, device=DEV)

    def call():
        cache = bq.PagedKVCache.zeros(1, 6, 2, 64)
        return bq.kv_append(cache, k, k, slots, q=q, q_norm=gain, k_norm=gain), cache.k[0].transpose(0, 1).clone()

    a, ka = call()
    q[2, 1, 5], q[3, 0, 63], k[4, 1, 0] = float("nan"), float("inf"), float("nan")
    b, kb = call()
    hurt, khurt = torch.zeros(6, 4, dtype=torch.bool, device=DEV), torch.zeros(6, 2, dtype=torch.bool, device=DEV)
    hurt[2, 1] = hurt[3, 0] = khurt[4, 1] = True
    assert torch.equal(a[~hurt], b[~hurt]) and torch.equal(ka[~khurt], kb[~khurt])
    assert b[2, 1].isnan().all() and b[3, 0, 63].isnan() and kb[4, 1].isnan().all()


def test_a_token_has_the_bits_of_a_call_of_its_own():
    g = rng("bits")
    T = 300
    q, k, v = normal(g, (T, 6, 96)), normal(g, (T, 2, 96)), normal(g, (T, 2, 96))
    gain = 1 + 0.1 * normal(g, (96,))
    rope = bq.Rope.from_theta(96)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 77
    whole, single = bq.PagedKVCache.zeros(20, 16, 2, 96, "q8_0"), bq.PagedKVCache.zeros(20, 16, 2, 96, "q8_0")
    slots = torch.arange(T, device=DEV)
    out = bq.kv_append(whole, k, v, slots, q=q, rope=rope, positions=pos, q_norm=gain, k_norm=gain)
    for t in (0, 1, 2, 3, 150, 299):
        one = bq.kv_append(single, k[t:t + 1], v[t:t + 1], slots[t:t + 1], q=q[t:t + 1], rope=rope, positions=pos[t:t + 1],
                           q_norm=gain, k_norm=gain)
        assert torch.equal(one[0], out[t])
        for a, b in ((whole.k, single.k), (whole.k_scale, single.k_scale), (whole.v, single.v)):
            assert torch.equal(a[t // 16, :, t % 16], b[t // 16, :, t % 16])


def test_a_decoder_with_norms_of_queries_and_keys():
    """The first layer's queries and keys of a PagedDecode step: the norms are in
    its path (the keys kept are the normed ones, turned), rows of a verify step
    keep the single steps' bits, and a captured step is the eager one."""
    g = rng("dec")
    gains = [dict(q_norm=1 + 0.2 * normal(g, (DEC_D,)), k_norm=1 + 0.2 * normal(g, (DEC_D,))) for _ in range(2)]

    def made(rows=1):
        dec = decoder("q8_0", "f16", rows=rows)
        for L, extra in zip(dec.layers, gains):
            L.update(extra)
        return dec

    h = wl.normal_torch((12, 256), 1.0, seed=3, stream=12, device=DEV)
    one, three = made(), made(rows=3)
    a, b = decode(one, bq.BlockTables(1, 8, 12, 16, 8), h), decode(three, bq.BlockTables(1, 8, 12, 16, 8), h)
    assert torch.equal(a, b)
    assert not torch.equal(a, decode(decoder("q8_0", "f16"), bq.BlockTables(1, 8, 12, 16, 8), h))
    # keys of layer 0: the products are there in fp32 (the last token's stay in _qkv)
    L = one.layers[0]
    x = bq.sandwich_norm(h, h, pre_gain=L["attn_gamma"], alpha=1.0, beta=0.0)[1]
    k = torch.stack([bq.gemv_qkv_bias("q8_0", L["qkv"], x[t], L["qkv_bias"]) for t in range(12)])
    k = k[:, 8 * DEC_D:10 * DEC_D].view(12, 2, DEC_D)
    pos = torch.arange(12, dtype=torch.int32)[None]
    want, off = turned(*normed(k.cpu(), L["k_norm"].cpu(), 1e-6), one.rope.freq.cpu(), [DEC_D // 2], pos, False)
    got = one.caches[0].k[0].transpose(0, 1)[:12].cpu().double()  # page 0 is the first taken
    assert ((got - want).abs() <= off + 2.0 ** -11 * (want.abs() + off) + 2.0 ** -25).all()
    # captured
    dec, tables = made(), bq.BlockTables(1, 8, 12, 16, 8)
    decode(dec, tables, h[:1])
    buf = h[1:2].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tables.resize(tables.lens + 1)
        dec.step(buf, tables.slots[:1], tables.positions[:1], tables.table, tables.lens)
    for t in range(1, 12):
        buf.copy_(h[t:t + 1])
        graph.replay()
        assert torch.equal(dec.logits, a[t:t + 1])


def test_refusals():
    cache = bq.PagedKVCache.zeros(2, 16, 2, 64)
    k, gain = torch.zeros(3, 2, 64, device=DEV), torch.ones(64, device=DEV)
    slots = torch.arange(3, device=DEV)
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k, slots, q_norm=gain)  # without q
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k, slots, k_norm=gain[:32])
    with pytest.raises(TypeError):
        bq.kv_append(cache, k, k, slots, k_norm=gain.half())
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k, slots, k_norm=gain.cpu())
    with pytest.raises(ValueError):
        bq.kv_append(cache, k, k, slots, k_norm=torch.ones(128, device=DEV)[::2])
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(bq.BQError):
            bq.kv_append(cache, k, k, slots, k_norm=gain, eps=eps)
    bq.kv_append(cache, k[:0], k[:0], slots[:0], k_norm=gain)
