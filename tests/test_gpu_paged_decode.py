"""Whole decoder layers over a paged cache (PagedDecode): a step against a plain
64-bit decoder, the rows of a verify step against the one-row steps bit for bit,
and a step captured in a CUDA graph."""
import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import workloads as wl
from block_quantized_weight_dequant_gb300.decode import PagedDecode

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
HIDDEN, HEADS, KV, D, INTER, VOCAB, LAYERS = 256, 8, 2, 64, 512, 300, 2


def model(qt, seed=3):
    def W(M, K, *tag):
        return bq.quantize_pack(wl.normal_torch((M, K), 0.05, seed=seed, stream=wl.stream_id(*tag), device=DEV), qt)

    def gain(*tag):
        return wl.normal_torch(HIDDEN, 0.1, seed=seed, stream=wl.stream_id(*tag), device=DEV, mean=1.0)

    layers = []
    for l in range(LAYERS):
        layers.append(dict(qkv=W((HEADS + 2 * KV) * D, HIDDEN, l, "qkv"), o=W(HIDDEN, HEADS * D, l, "o"),
                           gate=W(INTER, HIDDEN, l, "gate"), up=W(INTER, HIDDEN, l, "up"),
                           down=W(HIDDEN, INTER, l, "down"), attn_gamma=gain(l, "a"), gamma=gain(l, "g"),
                           qkv_bias=wl.normal_torch((HEADS + 2 * KV) * D, 0.1, seed=seed, stream=l, device=DEV)))
    layers[1].update(attn_post=gain("p1"), ffn_post=gain("p2"), attn_gate=gain("g1"), ffn_gate=gain("g2"))
    return layers, W(VOCAB, HIDDEN, "lm"), gain("final")


def dense(P, qt, K):
    """Packed Q8_0 or Q4_0 weights in float64."""
    raw = P.cpu().numpy()
    M = raw.shape[0]
    blocks = raw.reshape(M, K // 32, -1)
    d = blocks[..., :2].copy().view(np.float16).astype(np.float64)
    if qt == "q8_0":
        q = blocks[..., 2:].view(np.int8).astype(np.float64)
    else:
        b = blocks[..., 2:]
        q = np.concatenate([b & 15, b >> 4], -1).astype(np.float64) - 8
    return torch.from_numpy((d * q).reshape(M, K))


def decoder(qt, kind, rows=1, alpha=1.0, beta=1.0):
    layers, lm, final = model(qt)
    caches = [bq.PagedKVCache.zeros(12, 16, KV, D, kind) for _ in layers]
    rope = bq.Rope.from_theta(D, device=DEV)
    return PagedDecode(qt, layers, lm, final, caches, HEADS, rope, alpha=alpha, beta=beta, rows=rows)


def run(dec, tables, h):
    """h [tokens, hidden] of one request in steps of dec.rows tokens."""
    out = []
    for i in range(0, h.shape[0], dec.rows):
        assert int(tables.resize(tables.lens + dec.rows)) == 0
        n = dec.rows
        out.append(dec.step(h[i:i + n], tables.slots[:n], tables.positions[:n], tables.table, tables.lens).clone())
    return torch.cat(out)


def norm(x, g):
    return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * g


@pytest.mark.parametrize("qt", ["q8_0", "q4_0"])
def test_a_decode_against_a_plain_decoder(qt):
    dec = decoder(qt, "bf16", alpha=0.9, beta=1.1)
    tables = bq.BlockTables(1, 8, 12, 16, 8)
    tokens = 20
    h0 = wl.normal_torch((tokens, HIDDEN), 1.0, seed=3, stream=9, device=DEV)
    got = run(dec, tables, h0).cpu().double()
    # the plain decoder over all tokens at once, in 64 bits but for the cache's rounding
    h = h0.cpu().double()
    pos = torch.arange(tokens, dtype=torch.int32)[None]
    freq = dec.rope.freq.cpu()
    for L in dec.layers:
        P = {n: t.cpu().double() for n, t in L.items() if t.dtype == torch.float32}
        x = norm(h, P["attn_gamma"])
        qkv = x @ dense(L["qkv"], qt, HIDDEN).t() + P["qkv_bias"]
        q, k, v = (t.view(tokens, -1, D) for t in qkv.split([HEADS * D, KV * D, KV * D], 1))
        q, k = plain.turn(q, freq, [D // 2], pos, False)[0], plain.turn(k, freq, [D // 2], pos, False)[0]
        k, v = k.to(torch.bfloat16).double(), v.to(torch.bfloat16).double()
        s = torch.einsum("thd,shd->hts", q, k.repeat_interleave(HEADS // KV, 1)) * D ** -0.5
        s = s.masked_fill(torch.triu(torch.ones(tokens, tokens, dtype=torch.bool), 1), -torch.inf)
        a = torch.einsum("hts,shd->thd", torch.softmax(s, -1), v.repeat_interleave(HEADS // KV, 1)).reshape(tokens, -1)
        for W, K, inp, post, gate, g in (("o", HEADS * D, a, "attn_post", "attn_gate", "gamma"),
                                         ("down", INTER, None, "ffn_post", "ffn_gate", None)):
            if inp is None:
                x = norm(h, P["gamma"])
                z = x @ dense(L["gate"], qt, HIDDEN).t()
                inp = z / (1 + torch.exp(-z)) * (x @ dense(L["up"], qt, HIDDEN).t())
            b = inp @ dense(L[W], qt, K).t()
            if post in P:
                b = norm(b, P[post])
            h = 0.9 * h + 1.1 * P.get(gate, 1.0) * b
    want = norm(h, dec.final_gamma.cpu().double()) @ dense(dec.lm_head, qt, HIDDEN).t()
    # A key or value next to a rounding border of bf16 may be stored one step away
    # (2^-8 of it) where fp32 and 64 bits fall on different sides; fp32 errors are
    # near 2^-20 per stage, so such values are one in 2^10 or fewer.  Weighted into
    # sums of at least 64 products they move a logit by less than 2^-8 * 2^-4 of
    # the logits' rms even if one in 256 of them were.
    rms = float(want.square().mean().sqrt())
    assert float((got - want).abs().max()) <= 2.0 ** -12 * 16 * rms


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("rows", [2, 3, 6])
def test_verify_steps_have_the_bits_of_single_steps(kind, rows):
    h = wl.normal_torch((24, HIDDEN), 1.0, seed=3, stream=10, device=DEV)
    one, many = decoder("q8_0", kind), decoder("q8_0", kind, rows=rows)
    # the same table geometry for both: the bits depend on it
    a = run(one, bq.BlockTables(1, 8, 12, 16, 8), h)
    b = run(many, bq.BlockTables(1, 8, 12, 16, 8), h)
    assert torch.equal(a, b)
    for x, y in zip(one.caches, many.caches):
        assert torch.equal(x.k, y.k) and torch.equal(x.v, y.v)


def test_rows_of_several_requests_and_a_captured_step():
    """Three requests' tokens in one step, eager and captured."""
    rows, steps = 3, 5
    h = wl.normal_torch((steps, rows, HIDDEN), 1.0, seed=3, stream=11, device=DEV)
    results = []
    for captured in (False, True):
        dec = decoder("q8_0", "f16", rows=rows)
        t = bq.BlockTables(rows, 4, 12, 16, rows)
        goal = torch.zeros(rows, dtype=torch.int32, device=DEV)
        t.resize(goal)
        buf = torch.zeros((rows, HIDDEN), device=DEV)

        def step():
            t.resize(goal)
            dec.step(buf, t.slots, t.positions, t.table, t.lens)

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        out = []
        for i in range(steps):
            goal.fill_(i + 1)
            buf.copy_(h[i])
            graph.replay() if captured else step()
            out.append(dec.logits.clone())
        results.append(torch.stack(out))
    assert torch.equal(results[0], results[1])
    # each request alone gives the same tokens' logits within the GEMV bound's scale: here bit for bit,
    # since every call treats its rows apart and the chunks are single
    for r in range(rows):
        dec = decoder("q8_0", "f16")
        alone = run(dec, bq.BlockTables(1, 4, 12, 16, 1), h[:, r])
        assert torch.equal(alone, results[0][:, r])


def test_paged_decode_refusals():
    layers, lm, final = model("q8_0")
    caches = [bq.PagedKVCache.zeros(4, 16, KV, D) for _ in layers]
    with pytest.raises(ValueError):
        PagedDecode("q8_0", layers, lm, final, caches[:1], HEADS, None)
    with pytest.raises(ValueError):
        PagedDecode("q8_0", layers, lm, final, caches, HEADS, None, rows=7)
    with pytest.raises(ValueError):
        PagedDecode("q8_0", layers, lm, final, caches, HEADS + 1, None)
    dec = PagedDecode("q8_0", layers, lm, final, caches, HEADS, None, rows=3)
    i32 = dict(dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        dec.step(torch.zeros((3, HIDDEN), device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), None,
                 torch.zeros((2, 4), **i32), torch.zeros(2, **i32))


def test_a_step_of_fewer_embeddings_than_rows_is_refused():
    """One embedding is not spread over all rows; of one row it may come flat."""
    dec, tables = decoder("q8_0", "f16", rows=3), bq.BlockTables(3, 4, 12, 16, 3)
    tables.resize(tables.lens + 1)
    more = (tables.slots, tables.positions, tables.table, tables.lens)
    for shape in ((1, HIDDEN), (HIDDEN,), (3, 1), (4, HIDDEN)):
        with pytest.raises(ValueError, match="h must be"):
            dec.step(torch.ones(shape, device=DEV), *more)
    one, table = decoder("q8_0", "f16"), bq.BlockTables(1, 4, 12, 16, 1)
    table.resize(table.lens + 1)
    h = wl.normal_torch(HIDDEN, 1.0, seed=3, stream=12, device=DEV)
    more = (table.slots, table.positions, table.table, table.lens)
    a = one.step(h, *more).clone()
    assert torch.equal(a, one.step(h.view(1, HIDDEN), *more))
