"""The norms around a block (sandwich_norm) against a plain 64-bit form: widths
from one to the largest, odd ones, every type, gates, options, strides, in place;
a row's bits do not depend on the rows beside it or on alignment."""
import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq

import paged_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def normal(g, shape, dtype=F32):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(dtype).to(DEV)


def check(y, h, pre, post, gate, alpha=0.9, beta=1.3, eps=1e-6, **outs):
    y0, h0 = y.cpu().clone(), h.cpu().clone()
    cpu = [None if t is None else t.cpu() for t in (post, gate, pre)]
    ho, xo = bq.sandwich_norm(y, h, pre_gain=pre, post_gain=post, gate=gate, alpha=alpha, beta=beta, eps=eps, **outs)
    wh, wx, bh, bx = plain.sandwich(y0, h0, cpu[0], cpu[1], cpu[2], alpha, beta, eps)
    for got, want, bound in ((ho, wh, bh), (xo, wx, bx)):
        if want is None:
            assert got is None
            continue
        err = (got.cpu().double() - want).abs()
        # the type's rounding: half a unit, or half of fp16's smallest subnormal
        assert (err <= bound + plain.EPS[got.dtype] / 2 * (want.abs() + bound) + 2.0 ** -25).all(), float(err.max())
    return ho, xo


TYPES = [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]


@pytest.mark.parametrize("x,r", TYPES)
@pytest.mark.parametrize("width", [1, 7, 8, 250, 1000, 1024, 2047, 2048, 3584, 5120, 8192, 12345, 16384])
def test_widths_and_types(x, r, width):
    g = np.random.default_rng([width, TYPES.index((x, r))])
    for rows in (1, 3):
        y, h = normal(g, (rows, width), x), normal(g, (rows, width), r)
        pre, post = 1 + 0.1 * normal(g, (width,)), 1 + 0.1 * normal(g, (width,))
        check(y, h, pre, post, normal(g, (width,), x))
        check(y, h, pre, None, normal(g, (rows, width), x))
    check(y, h, None, post, None)
    check(y, h, None, None, None)
    check(y, h, pre, post, None, alpha=1.0, beta=0.0)


@pytest.mark.parametrize("x,r", [(BF16, F32), (F32, F32)])
@pytest.mark.parametrize("width", [896, 1024, 2047, 5120, 16384])
def test_many_rows_have_the_single_rows_bits(x, r, width):
    """More rows than fit the GPU at once (rows fetched ahead), the same rows one
    by one, and the same rows at odd addresses."""
    g = np.random.default_rng([width, 5])
    rows = 2500 if width < 3000 else 700
    y, h = normal(g, (rows, width), x), normal(g, (rows, width), r)
    pre, post, gate = 1 + 0.1 * normal(g, (width,)), 1 + 0.1 * normal(g, (width,)), normal(g, (rows, width), x)
    ho, xo = check(y, h, pre, post, gate)
    again = bq.sandwich_norm(y, h, pre, post, gate, 0.9, 1.3)
    assert torch.equal(again[0], ho) and torch.equal(again[1], xo)
    for i in (0, 1, rows // 2, rows - 1):
        one = bq.sandwich_norm(y[i:i + 1], h[i:i + 1], pre, post, gate[i:i + 1], 0.9, 1.3)
        assert torch.equal(one[0][0], ho[i]) and torch.equal(one[1][0], xo[i])
    odd_y = torch.empty(rows * (width + 1) + 1, dtype=x, device=DEV)[1:].view(rows, width + 1)[:, :width]
    odd_y.copy_(y)
    odd = bq.sandwich_norm(odd_y, h, pre, post, gate, 0.9, 1.3)
    assert torch.equal(odd[0], ho) and torch.equal(odd[1], xo)


def test_in_place_strided_and_graph():
    g = np.random.default_rng(6)
    rows, width = 5, 1024
    y, h = normal(g, (rows, width)), normal(g, (rows, width))
    pre, post = 1 + 0.1 * normal(g, (width,)), 1 + 0.1 * normal(g, (width,))
    want = bq.sandwich_norm(y, h, pre, post)
    y1, h1 = y.clone(), h.clone()
    check(y1, h1, pre, post, None, alpha=1.0, beta=1.0, h_out=h1, x_out=y1)
    assert torch.equal(h1, want[0]) and torch.equal(y1, want[1])
    room = torch.full((rows, width + 64), 3.0, device=DEV)
    check(y, h, pre, post, None, x_out=room[:, 32:32 + width])
    room[:, 32:32 + width] = 3.0
    assert (room == 3.0).all()
    graph, hs, xs = torch.cuda.CUDAGraph(), torch.empty_like(h), torch.empty_like(y)
    with torch.cuda.graph(graph):
        bq.sandwich_norm(y, h, pre, post, h_out=hs, x_out=xs)
    y.copy_(normal(g, (rows, width)))
    graph.replay()
    again = bq.sandwich_norm(y, h, pre, post)
    assert torch.equal(again[0], hs) and torch.equal(again[1], xs)


@pytest.mark.parametrize("rows,width", [(3, 64), (3, 2047), (2500, 1024), (700, 8192), (700, 5120), (400, 12345)])
def test_outputs_over_inputs(rows, width):
    """y, h and h_out one tensor; the outputs over each other's inputs; over a gate."""
    g = np.random.default_rng([width, 9])
    y, h, gate = (normal(g, (rows, width)) for _ in range(3))
    pre, post = 1 + 0.1 * normal(g, (width,)), 1 + 0.1 * normal(g, (width,))
    want = bq.sandwich_norm(h, h, pre, alpha=1.0, beta=0.0)
    one = h.clone()
    got = bq.sandwich_norm(one, one, pre, alpha=1.0, beta=0.0, h_out=one)
    assert torch.equal(one, want[0]) and torch.equal(got[1], want[1])
    want = bq.sandwich_norm(y, h, pre, post, gate)
    for h_out, x_out in ((0, 1), (1, 0), (2, 1), (0, 2)):
        t = [y.clone(), h.clone(), gate.clone()]
        bq.sandwich_norm(t[0], t[1], pre, post, t[2], h_out=t[h_out], x_out=t[x_out])
        assert torch.equal(t[h_out], want[0]) and torch.equal(t[x_out], want[1])


def test_zero_rows_and_zero_values():
    width = 64
    z = torch.zeros((3, width), device=DEV)
    one = torch.ones(width, device=DEV)
    ho, xo = bq.sandwich_norm(z, z, one, one)
    assert (ho == 0).all() and (xo == 0).all()
    ho, xo = bq.sandwich_norm(z[:0], z[:0], one, one)
    assert ho.shape == (0, width) and xo.shape == (0, width)
    bad = z.clone()
    bad[1, 5] = float("nan")
    ho, xo = bq.sandwich_norm(bad, z + 1, one, one)
    assert torch.isnan(xo[1]).all() and torch.isfinite(xo[0]).all() and torch.isfinite(xo[2]).all()


def test_refusals():
    y = torch.zeros((2, 64), device=DEV)
    g = torch.ones(64, device=DEV)
    with pytest.raises(ValueError):
        bq.sandwich_norm(y[0], y[0], g)
    with pytest.raises(ValueError):
        bq.sandwich_norm(y, y[:1], g)
    with pytest.raises(TypeError):
        bq.sandwich_norm(y, y.half(), g)
    with pytest.raises(TypeError):
        bq.sandwich_norm(y, y, g.half())
    with pytest.raises(ValueError):
        bq.sandwich_norm(y, y, g[:32])
    with pytest.raises(TypeError):
        bq.sandwich_norm(y, y, g, gate=g.half())
    with pytest.raises(ValueError):
        bq.sandwich_norm(y, y, x_out=y)
    with pytest.raises(ValueError, match="overlaps"):
        bq.sandwich_norm(y, y, g, x_out=y[:1].expand(2, 64))
    with pytest.raises(bq.BQError):
        bq.sandwich_norm(y, y, g, eps=-1.0)
    with pytest.raises(bq.BQError):
        wide = torch.zeros((1, 16385), device=DEV)
        bq.sandwich_norm(wide, wide)
