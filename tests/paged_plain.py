"""Plain 64-bit forms of the calls around the paged key-value cache, for the
tests, and the bounds their outputs are held to.  numpy / torch on the host."""
import math

import numpy as np
import torch

EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


def values(cache):
    """k and v of a PagedKVCache as float64 [pages, kv_heads, page_size, head_dim] on the host."""
    out = []
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = codes.cpu().double()
        if scale is not None:
            x = (x.unflatten(-1, (-1, 32)) * scale.cpu().double()[..., None]).flatten(-2)
        out.append(x)
    return out


def attention(k, v, q, table, lens, rows, scale):
    """(out, bound factor A, S) in float64: q [requests * rows, heads, D]; A = sum
    of weight |v| per element, S the largest scale * sum |q k| of the row."""
    page, D = k.shape[2], k.shape[3]
    q = q.double()
    group = q.shape[1] // k.shape[1]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    top = torch.zeros(q.shape[:2] + (1,), dtype=torch.float64)
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // page)].long()
        for h in range(k.shape[1]):
            kk, vv = k[ids, h].reshape(-1, D)[:n], v[ids, h].reshape(-1, D)[:n]
            for r in range(rows):
                m = n - rows + r + 1
                if m <= 0:
                    continue
                hs = slice(h * group, (h + 1) * group)
                qq = q[b * rows + r, hs]
                p = torch.softmax(scale * qq @ kk[:m].t(), -1)
                out[b * rows + r, hs] = p @ vv[:m]
                mag[b * rows + r, hs] = p @ vv[:m].abs()
                top[b * rows + r, hs] = (abs(scale) * qq.abs() @ kk[:m].abs().t()).amax(-1, keepdim=True)
    return out, mag, top


def attention_bound(out, mag, top, dtype, one_part):
    """|error| of paged_attention.  A score is a sum of exact products; at most
    24 additions of the tensor core or fp32 in sequence, each off by 2^-23 of
    the sum of magnitudes: below 2^-18 top (nats), with the parts' 2^-22 and the
    scale's rounding below 2^-17 top.  Weights: that, plus 2^-20 for the power of
    two and its argument.  Numerator and denominator: twice that.  Sums over
    tiles, warps and chunks: under 300 fp32 roundings, 2^-15.  A weight carried as
    one fp16 part (Q8_0 cache, bf16 queries): 2^-12.  The output's rounding:
    half a unit, at least half the smallest fp16 subnormal."""
    rel = 2 * (2.0 ** -17 * top + 2.0 ** -20) + 2.0 ** -15 + (2.0 ** -12 if one_part else 0.0)
    return rel * mag + EPS[dtype] / 2 * (out.abs() + rel * mag) + 2.0 ** -25


def turn(x, freq, sections, positions, interleaved):
    """Rotated heads in float64: x [tokens, heads, D], positions [axes, tokens]."""
    x = x.double()
    half = freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))
    angle = positions.double()[axis].t() * freq.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y = x.clone()
    if interleaved:
        e, o = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        e, o = slice(0, half), slice(half, 2 * half)
    y[..., e] = x[..., e] * c - x[..., o] * s
    y[..., o] = x[..., o] * c + x[..., e] * s
    # |error|: the angle (a turn right to 2^-23 turns and the 48-bit split's 2^-48 of
    # position * freq, in radians), 2^-22 for sine and cosine, two roundings
    off = 2 * math.pi * 2.0 ** -22 + 2.0 ** -48 * angle.abs() + 2.0 ** -21
    bound = torch.zeros_like(x)
    pair = (x[..., e].abs() + x[..., o].abs()) * off[:, None]
    bound[..., e], bound[..., o] = pair, pair
    return y, bound


def q8(x):
    """Q8_0 codes and scales of [..., D] fp32 (numpy), as bq_quantize_pack."""
    x = np.asarray(x, dtype=np.float32)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    d = (np.abs(b).max(-1) / np.float32(127)).astype(np.float16)
    f = d.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        r = b / f
        r = np.where(f == 0, 0, np.clip(np.sign(r) * np.floor(np.abs(r) + np.float32(0.5)), -127, 127))
    return r.astype(np.int8).reshape(x.shape), d


def block_tables(lens, new, table, free, count, page, room):
    """kv_block_tables told request by request: (table, free, slots, positions,
    starts, lens_out, count_out, refused)."""
    table, free = table.copy(), free.copy()
    most = table.shape[1] * page
    pages = [(-(-int(a) // page), -(-int(z) // page)) for a, z in zip(lens, new)]
    bad = [not (0 <= a <= most and 0 <= z <= most) for a, z in zip(lens, new)]
    stack = free[:count].tolist()
    for b, (p, q) in enumerate(pages):
        if not bad[b] and q < p:
            stack += table[b, q:p].tolist()
    avail = len(stack)
    slots, positions = np.full(room, -1, np.int64), np.zeros(room, np.int32)
    starts, out, asked, refused = [0], [], 0, 0
    for b, (a, z) in enumerate(zip(lens, new)):
        p, q = pages[b]
        rows = 0 if bad[b] else max(0, z - a)
        asked += 0 if bad[b] else max(0, q - p)
        ok = not bad[b] and (q <= p or asked <= avail) and (rows == 0 or starts[-1] + rows <= room)
        if ok:
            for j in range(p, q):
                table[b, j] = stack.pop()
            for t in range(rows):
                pos = a + t
                slots[starts[-1] + t] = int(table[b, pos // page]) * page + pos % page
                positions[starts[-1] + t] = pos
        refused += not ok
        out.append(z if ok else a)
        starts.append(starts[-1] + rows)
    # what was popped from below the old top leaves the stack's words as they were
    final = free.copy()
    if len(stack) > count:
        final[count:len(stack)] = stack[count:]
    return (table, final, slots, positions, np.array(starts, np.int32), np.array(out, np.int32), len(stack), refused)


def sandwich(y, h, post, gate, pre, alpha, beta, eps):
    """(h', x', bound of h', bound of x') in float64, without the outputs' rounding.

    fp32 sums of n squares: each thread's chain, a butterfly and the warps, under
    64 + 5 + 16 roundings of terms of one sign: 85 * 2^-24 of the sum, halved by
    the root; the root's approximation 2^-22 and the products' roundings: below
    2^-17 relative in all for each norm.  h' adds two terms: the bound is relative
    to their magnitudes."""
    y, h = y.double(), h.double()
    b = y
    if post is not None:
        b = y / (y.square().mean(1, keepdim=True) + eps).sqrt() * post.double()
    if gate is not None:
        b = b * gate.double()
    ho = alpha * h + beta * b
    bh = 2.0 ** -17 * ((alpha * h).abs() + (beta * b).abs())
    if pre is None:
        return ho, None, bh, None
    norm = (ho.square().mean(1, keepdim=True) + eps).sqrt()
    x = ho / norm * pre.double()
    # an error of h' moves x' directly and through the norm (by the rms of the errors)
    bx = (bh + (bh.square().mean(1, keepdim=True)).sqrt() * ho.abs() / norm) / norm * pre.double().abs() + 2.0 ** -17 * x.abs()
    return ho, x, bh, bx
