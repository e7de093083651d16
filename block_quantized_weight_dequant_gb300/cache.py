"""What stands between the weight products of a decode step: a paged key-value
cache (block tables, append with rotary positions, attention of the new
tokens) and the norms around a block.

Like the rest of the package these functions only marshal arguments: tensors
are checked, outputs allocated with PyTorch when the caller passes none, and
the C ABI (include/bqgemv.h) is called on the current stream of the tensors'
device.  Activations are fp32, fp16 or bf16.  (RunIT README, data-flow diagram
and kernel table: attention, rope and the KV cache; EdgeRunner blog post: the
GPU-resident paged cache.)
"""
import ctypes
import math

import torch

from . import _lib
from ._lib import BQ_VERIFY_MAX_ROWS, lib

__all__ = ["PagedKVCache", "Rope", "BlockTables", "kv_block_tables", "kv_append", "paged_attention",
           "paged_attention_workspace", "sandwich_norm"]

_DTYPES = {torch.float32: _lib.BQ_F32, torch.float16: _lib.BQ_F16, torch.bfloat16: _lib.BQ_BF16}
_KINDS = {"f16": torch.float16, "bf16": torch.bfloat16, "q8_0": torch.int8}


def _need(t, name, dtype=None, like=None):
    """A CUDA tensor of the given dtype on the device of `like`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this package has no CPU path)")
    if like is not None and t.device != like:
        raise ValueError(f"{name} is on {t.device}, expected {like}")


def _activation(t, name, shape, dtype, device):
    """An activation [..., n] of a known shape whose last dimension is contiguous."""
    _need(t, name, dtype, device)
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be fp32, fp16 or bf16, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError(f"the last dimension of {name} must be contiguous")


def _dense(t, name, dtype, device, numel=None):
    _need(t, name, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def _call(fn, what, device, *args):
    """fn(*args, stream) on `device`'s current stream."""
    if torch.cuda.current_device() == device.index:
        status = fn(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch.cuda.current_stream().cuda_stream)
    if status != _lib.BQ_OK:
        raise _lib.BQError(status, what)


class PagedKVCache:
    """One layer's paged key-value cache: ``k`` and ``v`` [pages, kv_heads,
    page_size, head_dim], fp16 or bf16, or int8 codes with ``k_scale`` and
    ``v_scale`` fp16 [pages, kv_heads, page_size, head_dim / 32] (Q8_0: value =
    scale * code).  Any strides will do as long as head_dim is contiguous, k and
    v share them, and the scales are laid out as the codes are: pages of
    [page_size, kv_heads, head_dim] are a ``transpose(1, 2)`` away, and k and v
    may be slices of one tensor.  The object keeps the tensors, not copies."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _need(k, "k")
        if k.dtype not in _KINDS.values():
            raise TypeError(f"k must be fp16, bf16 or int8 (Q8_0 codes), got {k.dtype}")
        if k.dim() != 4:
            raise ValueError("k must be [pages, kv_heads, page_size, head_dim]")
        _need(v, "v", k.dtype, k.device)
        quantized = k.dtype == torch.int8
        if v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("k and v must have the same shape and strides")
        if k.numel() == 0:
            raise ValueError("the cache must hold at least one page, head, slot and value")
        if k.stride(3) != 1:
            raise ValueError("head_dim must be contiguous")
        pages, kv_heads, page_size, head_dim = k.shape
        # a stride over one entry says nothing: leave it out of the checks
        strides = [s if n > 1 else 0 for s, n in zip(k.stride()[:3], k.shape[:3])]
        if quantized:
            if head_dim % 32:
                raise ValueError("a Q8_0 cache needs head_dim % 32 == 0")
            want = (pages, kv_heads, page_size, head_dim // 32)
            for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
                _need(s, name, torch.float16, k.device)
                if tuple(s.shape) != want:
                    raise ValueError(f"{name} must be {list(want)}, got {list(s.shape)}")
                ok = s.stride(3) == 1 or s.shape[3] == 1
                for n, a, b in zip(s.shape[:3], s.stride()[:3], strides):
                    ok = ok and (n == 1 or 32 * a == b)
                if not ok:
                    raise ValueError(f"{name} must be laid out as the codes (one scale per 32 of them)")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to int8 codes (a Q8_0 cache)")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kind = {d: n for n, d in _KINDS.items()}[k.dtype]
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, kv_heads, page_size, head_dim
        self.device = k.device
        kind = {"f16": _lib.BQ_F16, "bf16": _lib.BQ_BF16, "q8_0": _lib.BQ_Q8_0}[self.kind]
        ptr = (lambda t: t.data_ptr()) if quantized else (lambda t: None)
        self._c = _lib.BqKvCache(kind, kv_heads, head_dim, page_size, pages, *strides, k.data_ptr(),
                                 v.data_ptr(), ptr(k_scale), ptr(v_scale))
        self._ref = ctypes.byref(self._c)
        self._workspace = {}  # workspace bytes by call geometry

    @classmethod
    def zeros(cls, pages, page_size, kv_heads, head_dim, kind="f16", device="cuda"):
        """A zeroed cache of `kind` "f16", "bf16" or "q8_0"."""
        if kind not in _KINDS:
            raise ValueError(f"kind must be one of {sorted(_KINDS)}, got {kind!r}")
        shape = (int(pages), int(kv_heads), int(page_size), int(head_dim))
        k, v = (torch.zeros(shape, dtype=_KINDS[kind], device=device) for _ in range(2))
        if kind != "q8_0":
            return cls(k, v)
        scales = shape[:3] + (shape[3] // 32,)
        return cls(k, v, *(torch.zeros(scales, dtype=torch.float16, device=device) for _ in range(2)))


class Rope:
    """Rotary positions: pair p of a head turns by position * freq[p] radians.
    ``freq``: fp64 CUDA [rot / 2] (rot values of a head are rotated, a multiple
    of 8; the rest pass).  ``sections``: pairs of each position axis, one to
    three of them, in order (time, height, width); one axis by default.
    ``interleaved``: pairs are (2p, 2p + 1) instead of (p, p + rot / 2)."""

    def __init__(self, freq, sections=None, interleaved=False):
        _need(freq, "freq", torch.float64)
        _dense(freq, "freq", torch.float64, freq.device)
        if freq.dim() != 1 or freq.numel() == 0 or freq.numel() % 4:
            raise ValueError("freq must be [rot / 2] with rot a multiple of 8")
        sections = [freq.numel()] if sections is None else [int(s) for s in sections]
        if not 1 <= len(sections) <= 3 or min(sections) < 0 or sum(sections) != freq.numel():
            raise ValueError("sections must be one to three counts that sum to rot / 2")
        self.freq, self.sections, self.interleaved = freq, sections, bool(interleaved)
        self.rot, self.axes = 2 * freq.numel(), len(sections)
        self._sections = (ctypes.c_int32 * 3)(*(sections + [0] * (3 - len(sections))))

    @classmethod
    def from_theta(cls, rot, theta=10000.0, sections=None, interleaved=False, device="cuda"):
        """freq[p] = theta ** (-2 p / rot)."""
        p = torch.arange(int(rot) // 2, dtype=torch.float64)
        return cls((float(theta) ** (-2.0 * p / int(rot))).to(device), sections, interleaved)


def kv_block_tables(lens, new_lens, table, free_pages, free_count, page_size, slots, positions, starts,
                    lens_out=None, free_count_out=None, refused=None):
    """Block tables, slot map and free pages of a step from the requests'
    lengths before (`lens`) and after (`new_lens`), int32 [requests]: requests
    that shrink give their pages back to the stack `free_pages` [pool], of
    which the first `free_count` [1] are free, requests that grow take theirs
    from its top into their row of `table` [requests, width]; every new token
    gets its position and its slot (page * page_size + place), rows of request b
    at starts[b] .. starts[b + 1] - 1.  Requests that the pool or `slots` cannot
    hold are refused whole: they keep their length, their slots are -1 (see
    bq_kv_block_tables in include/bqgemv.h for the order).  slots int64 and
    positions int32 [room] are filled to their ends (-1, 0).  lens_out and
    free_count_out default to lens and free_count themselves (updated in place).
    Returns `refused` [1], the number of refused requests."""
    _need(lens, "lens")
    dev = lens.device
    i32 = torch.int32
    _dense(lens, "lens", i32, dev)
    n = lens.numel()
    _dense(new_lens, "new_lens", i32, dev, n)
    _need(table, "table", i32, dev)
    if table.dim() != 2 or table.shape[0] != n or (n and table.shape[1] < 1):
        raise ValueError(f"table must be [{n}, width]")
    if table.numel() and table.stride(1) != 1 and table.shape[1] > 1:
        raise ValueError("rows of table must be contiguous")
    _dense(free_pages, "free_pages", i32, dev)
    _dense(free_count, "free_count", i32, dev, 1)
    _dense(slots, "slots", torch.int64, dev)
    _dense(positions, "positions", i32, dev, slots.numel())
    _dense(starts, "starts", i32, dev, n + 1)
    lens_out = lens if lens_out is None else lens_out
    free_count_out = free_count if free_count_out is None else free_count_out
    refused = torch.empty(1, dtype=i32, device=dev) if refused is None else refused
    _dense(lens_out, "lens_out", i32, dev, n)
    _dense(free_count_out, "free_count_out", i32, dev, 1)
    _dense(refused, "refused", i32, dev, 1)
    width = max(1, table.shape[1])
    stride = table.stride(0) if n > 1 else width
    args = _lib.BqKvTables(n, int(page_size), width, free_pages.numel(), stride, slots.numel(),
                           lens.data_ptr(), new_lens.data_ptr(), table.data_ptr(), free_pages.data_ptr(),
                           free_count.data_ptr(), slots.data_ptr(), positions.data_ptr(), starts.data_ptr(),
                           lens_out.data_ptr(), free_count_out.data_ptr(), refused.data_ptr())
    _call(lib.bq_kv_block_tables, "kv_block_tables", dev, ctypes.byref(args))
    return refused


class BlockTables:
    """The requests' side of a paged cache, on the GPU: lengths, block table and
    the stack of free pages, shared by all layers' caches.  ``resize`` moves
    every request to its new length and fills ``slots``, ``positions`` and
    ``starts`` for the tokens that came; it enqueues one kernel, allocates
    nothing and can be captured in a CUDA graph (new lengths are read from the
    tensor that it is given)."""

    def __init__(self, requests, max_pages, pages, page_size, max_tokens, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = int(page_size)
        self.lens = torch.zeros(requests, **i32)
        self.table = torch.full((requests, max_pages), -1, **i32)
        self.free_pages = torch.arange(pages - 1, -1, -1, **i32)  # page 0 on top
        self.free_count = torch.full((1,), pages, **i32)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
        self.positions = torch.zeros(max_tokens, **i32)
        self.starts = torch.zeros(requests + 1, **i32)
        self.refused = torch.zeros(1, **i32)

    def resize(self, new_lens):
        """Lengths become new_lens (int32 [requests]) where pages and rows
        suffice; returns ``refused``."""
        return kv_block_tables(self.lens, new_lens, self.table, self.free_pages, self.free_count,
                               self.page_size, self.slots, self.positions, self.starts, refused=self.refused)


def _strides(t):
    """Token and head strides of [tokens, heads, head_dim]; 0 over one entry."""
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def kv_append(cache, k, v, slots, q=None, q_out=None, rope=None, positions=None):
    """Store keys and values k, v [tokens, kv_heads, head_dim] at `slots` (int64
    [tokens], < 0: not stored; the others must differ) of `cache`.  With `rope`,
    keys are rotated by `positions` (int32 [axes, tokens], or [tokens] for one
    axis), and so are queries q [tokens, heads, head_dim] into q_out (a new
    tensor, or q itself).  Inputs may be slices of one projection's rows.
    Returns q_out, or None without q."""
    if not isinstance(cache, PagedKVCache):
        raise TypeError("cache must be a PagedKVCache")
    dev, kv, D = cache.device, cache.kv_heads, cache.head_dim
    _need(k, "k", None, dev)
    T = k.shape[0] if k.dim() == 3 else -1
    _activation(k, "k", (T, kv, D), None, dev)
    _activation(v, "v", (T, kv, D), k.dtype, dev)
    _dense(slots, "slots", torch.int64, dev, T)
    heads, qp, op, qs, os = 0, None, None, (0, 0), (0, 0)
    if q is not None:
        _need(q, "q", k.dtype, dev)
        heads = q.shape[1] if q.dim() == 3 else -1
        _activation(q, "q", (T, heads, D), k.dtype, dev)
        if q_out is None:
            q_out = torch.empty((T, heads, D), dtype=q.dtype, device=dev)
        _activation(q_out, "q_out", (T, heads, D), q.dtype, dev)
        qp, op, qs, os = q.data_ptr(), q_out.data_ptr(), _strides(q), _strides(q_out)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot, axes, inter, sections, freq, pos, ps = 0, 0, 0, _NO_SECTIONS, None, None, 0
    if rope is not None:
        if not isinstance(rope, Rope):
            raise TypeError("rope must be a Rope")
        _need(positions, "positions", torch.int32, dev)
        if rope.freq.device != dev:
            raise ValueError(f"rope is on {rope.freq.device}, expected {dev}")
        want = (rope.axes, T)
        if tuple(positions.shape) != want and not (rope.axes == 1 and tuple(positions.shape) == (T,)):
            raise ValueError(f"positions must be {list(want)}, got {list(positions.shape)}")
        if T > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous over the tokens")
        ps = positions.stride(0) if rope.axes > 1 else 0
        rot, axes, inter, sections = rope.rot, rope.axes, rope.interleaved, rope._sections
        freq, pos = rope.freq.data_ptr(), positions.data_ptr()
    elif positions is not None:
        raise ValueError("positions without rope")
    args = _lib.BqKvAppendArgs(_DTYPES[k.dtype], heads, rot, axes, inter, sections, T, k.data_ptr(),
                               v.data_ptr(), qp, op, *_strides(k), *_strides(v), *qs, *os,
                               slots.data_ptr(), pos, ps, freq)
    _call(lib.bq_kv_append, "kv_append", dev, cache._ref, ctypes.byref(args))
    return q_out


_NO_SECTIONS = (ctypes.c_int32 * 3)()


def paged_attention(cache, q, table, lens, rows=1, scale=None, out=None, workspace=None):
    """Attention of each request's last `rows` tokens (1 to 6) over its cached
    positions: q [requests * rows, heads, head_dim] (row r of request b at b *
    rows + r) sees the first lens[b] - rows + r + 1 positions, so `lens` (int32
    [requests]) counts the new tokens, which have been appended.  `table` int32
    [requests, width] holds the requests' pages.  heads is a multiple of the
    cache's kv_heads.  A row that sees nothing gives zeros.  scale defaults to
    1 / sqrt(head_dim).  Row r's bits are those of the one-row call at its
    length.  workspace: uint8, ``paged_attention_workspace(...)`` bytes, one per
    call that may overlap others; allocated when None."""
    if not isinstance(cache, PagedKVCache):
        raise TypeError("cache must be a PagedKVCache")
    dev, D = cache.device, cache.head_dim
    if not 1 <= rows <= BQ_VERIFY_MAX_ROWS:
        raise ValueError(f"rows must be 1 to {BQ_VERIFY_MAX_ROWS}, got {rows}")
    _dense(lens, "lens", torch.int32, dev)
    n = lens.numel()
    _need(q, "q", None, dev)
    heads = q.shape[1] if q.dim() == 3 else -1
    _activation(q, "q", (n * rows, heads, D), None, dev)
    _need(table, "table", torch.int32, dev)
    if table.dim() != 2 or table.shape[0] != n or (n and table.shape[1] < 1):
        raise ValueError(f"table must be [{n}, width]")
    if table.numel() and table.stride(1) != 1 and table.shape[1] > 1:
        raise ValueError("rows of table must be contiguous")
    if out is None:
        out = torch.empty((n * rows, heads, D), dtype=q.dtype, device=dev)
    else:
        _activation(out, "out", (n * rows, heads, D), q.dtype, dev)
    width = max(1, table.shape[1])
    args = _lib.BqAttentionArgs(_DTYPES[q.dtype], n, rows, heads, width,
                                1.0 / math.sqrt(D) if scale is None else scale,
                                table.stride(0) if n > 1 else width, *_strides(q), *_strides(out),
                                q.data_ptr(), out.data_ptr(), table.data_ptr(), lens.data_ptr())
    ref = ctypes.byref(args)
    key = (n, rows, heads, width)
    nbytes = cache._workspace.get(key)
    if nbytes is None:
        nbytes = lib.bq_paged_attention_workspace_bytes(cache._ref, ref)
        if nbytes >= 0:
            cache._workspace[key] = nbytes
    if workspace is None:
        if nbytes > 0:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        _dense(workspace, "workspace", torch.uint8, dev)
        nbytes = workspace.numel()
    _call(lib.bq_paged_attention, "paged_attention", dev, cache._ref, ref,
          None if workspace is None else workspace.data_ptr(), nbytes)
    return out


def paged_attention_workspace(cache, requests, rows, heads, width):
    """Bytes of workspace of a paged_attention call of this geometry."""
    args = _lib.BqAttentionArgs(_lib.BQ_F32, requests, rows, heads, width, 1.0, width)
    nbytes = lib.bq_paged_attention_workspace_bytes(cache._ref, ctypes.byref(args))
    if nbytes < 0:
        raise ValueError(f"no paged_attention of requests={requests} rows={rows} heads={heads} width={width}")
    return nbytes


def sandwich_norm(y, h, pre_gain=None, post_gain=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6,
                  h_out=None, x_out=None):
    """The norms after one block and before the next, with the block's gate
    and the residual scales, per row of [rows, width]:

        b  = RMSNorm(y) * post_gain        (b = y without post_gain)
        h' = alpha * h + beta * gate * b   (no gate: 1)
        x' = RMSNorm(h') * pre_gain        (not computed without pre_gain)

    y: the block's output; h: the residual stream, of y's dtype or fp32; gains
    fp32 [width]; gate of y's dtype, [width] or [rows, width].  Returns (h',
    x'), x' of y's dtype (None without pre_gain).  h_out may be h, x_out may be
    y."""
    _need(y, "y")
    dev = y.device
    if y.dim() != 2:
        raise ValueError("y must be [rows, width]")
    shape = tuple(y.shape)
    _activation(y, "y", shape, None, dev)
    _need(h, "h", None, dev)
    _activation(h, "h", shape, None, dev)
    if h.dtype != y.dtype and h.dtype != torch.float32:
        raise TypeError(f"h must be {y.dtype} or fp32, got {h.dtype}")
    width = shape[1]
    gp, gs = None, 0
    if gate is not None:
        _need(gate, "gate", y.dtype, dev)
        _activation(gate, "gate", (width,) if gate.dim() == 1 else shape, y.dtype, dev)
        gp, gs = gate.data_ptr(), (gate.stride(0) if gate.dim() == 2 and shape[0] > 1 else 0)
    for name, g in (("pre_gain", pre_gain), ("post_gain", post_gain)):
        if g is not None:
            _dense(g, name, torch.float32, dev, width)
    if h_out is None:
        h_out = torch.empty(shape, dtype=h.dtype, device=dev)
    else:
        _activation(h_out, "h_out", shape, h.dtype, dev)
    if pre_gain is None:
        if x_out is not None:
            raise ValueError("x_out without pre_gain")
    elif x_out is None:
        x_out = torch.empty(shape, dtype=y.dtype, device=dev)
    else:
        _activation(x_out, "x_out", shape, y.dtype, dev)

    def row(t):
        return t.stride(0) if shape[0] > 1 else 0

    args = _lib.BqSandwichArgs(_DTYPES[y.dtype], _DTYPES[h.dtype], shape[0], width, y.data_ptr(), h.data_ptr(),
                               gp, None if post_gain is None else post_gain.data_ptr(),
                               None if pre_gain is None else pre_gain.data_ptr(), h_out.data_ptr(),
                               None if x_out is None else x_out.data_ptr(), row(y), row(h), gs, row(h_out),
                               0 if x_out is None else row(x_out), alpha, beta, eps)
    _call(lib.bq_sandwich_norm, "sandwich_norm", dev, ctypes.byref(args))
    return h_out, x_out
