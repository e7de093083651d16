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


# (one attribute lookup each: a call's checks cost as much as its launch)
_Tensor = torch.Tensor
_byref = ctypes.byref
# the current stream's handle and the current device, without a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _i32(n):
    """n for a 32-bit field of the C ABI: -1, which is refused, for a number that
    ctypes would cut short."""
    n = int(n)
    return n if -(1 << 31) <= n < 1 << 31 else -1


def _need(t, name, dtype=None, like=None):
    """A CUDA tensor of the given dtype on the device of `like`."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this package has no CPU path)")
    if like is not None and t.device != like:
        raise ValueError(f"{name} is on {t.device}, expected {like}")


def _activation(t, name, shape, dtype, device):
    """An activation of a known shape whose last dimension is contiguous."""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device.index and t.shape == shape
            and t.is_contiguous()):
        return
    _need(t, name, dtype, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError(f"the last dimension of {name} must be contiguous")


def _result(t, name, shape, dtype, device):
    """An activation that is written: no element of it twice."""
    _activation(t, name, shape, dtype, device)
    if not t.is_contiguous() and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{name} overlaps itself")


def _empty(shape, dtype, like):
    """A new contiguous tensor on the device of `like` (cheapest in its image)."""
    if like.shape == shape and like.dtype is dtype and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, dtype=dtype, device=like.device)


def _first(t, name, device=None):
    """An activation that says dtype, and device if that is None."""
    if not (isinstance(t, _Tensor) and t.dtype in _DTYPES and t.is_cuda and (device is None or t.device == device)):
        _need(t, name, None, device)
        raise TypeError(f"{name} must be fp32, fp16 or bf16, got {t.dtype}")


def _dense(t, name, dtype, device, numel=None):
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device.index and t.is_contiguous()
            and (numel is None or t.numel() == numel)):
        return
    _need(t, name, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def _table(t, n, device):
    """The block table: rows of contiguous page numbers; returns width and row stride."""
    if (isinstance(t, _Tensor) and t.dtype is torch.int32 and t.get_device() == device.index and t.dim() == 2
            and t.is_contiguous()):
        rows, width = t.shape
        if rows == n and width:
            return width, width
    _need(t, "table", torch.int32, device)
    if t.dim() != 2 or t.shape[0] != n or (n and t.shape[1] < 1):
        raise ValueError(f"table must be [{n}, width]")
    if t.stride(1) != 1 and t.shape[1] > 1 and n:
        raise ValueError("rows of table must be contiguous")
    width = t.shape[1] or 1
    return width, (t.stride(0) if n > 1 else width)


def _call(fn, what, device, *args):
    """fn(*args, stream) on `device`'s current stream."""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status:
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
        if any(n > 1 and s == 0 for n, s in zip(k.shape, k.stride())):
            raise ValueError("the cache overlaps itself")
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
        self._scale = 1.0 / math.sqrt(head_dim)
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
    of 16; the rest pass).  ``sections``: pairs of each position axis, one to
    three of them, in order (time, height, width); one axis by default.
    ``interleaved``: pairs are (2p, 2p + 1) instead of (p, p + rot / 2)."""

    def __init__(self, freq, sections=None, interleaved=False):
        _need(freq, "freq", torch.float64)
        _dense(freq, "freq", torch.float64, freq.device)
        if freq.dim() != 1 or freq.numel() == 0 or freq.numel() % 8:
            raise ValueError("freq must be [rot / 2] with rot a multiple of 16")
        sections = [freq.numel()] if sections is None else [int(s) for s in sections]
        if not 1 <= len(sections) <= 3 or min(sections) < 0 or sum(sections) != freq.numel():
            raise ValueError("sections must be one to three counts that sum to rot / 2")
        self.freq, self.sections, self.interleaved = freq, sections, bool(interleaved)
        self.rot, self.axes = 2 * freq.numel(), len(sections)
        self.device, self._ptr = freq.device, freq.data_ptr()
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
    width, stride = _table(table, n, dev)
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
    args = _lib.BqKvTables(n, _i32(page_size), width, _i32(free_pages.numel()), stride, slots.numel(),
                           lens.data_ptr(), new_lens.data_ptr(), table.data_ptr(), free_pages.data_ptr(),
                           free_count.data_ptr(), slots.data_ptr(), positions.data_ptr(), starts.data_ptr(),
                           lens_out.data_ptr(), free_count_out.data_ptr(), refused.data_ptr())
    _call(lib.bq_kv_block_tables, "kv_block_tables", dev, _byref(args))
    return refused


class BlockTables:
    """The requests' side of a paged cache, on the GPU: lengths, block table and
    the stack of free pages, shared by all layers' caches.  ``resize`` moves
    every request to its new length and fills ``slots``, ``positions`` and
    ``starts`` for the tokens that came; it enqueues one kernel (two where
    max_tokens is above 4096), allocates nothing and can be captured in a CUDA
    graph (new lengths are read from the tensor that it is given).  max_pages is
    the table's width, which decides how paged_attention cuts its work: one much
    wider than the requests are long costs time."""

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


def _strides(t, tokens, heads):
    """Token and head strides of [tokens, heads, head_dim]; 0 over one entry."""
    a, b, _ = t.stride()
    return (a if tokens > 1 else 0), (b if heads > 1 else 0)


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
    _first(k, "k", dev)
    dtype = k.dtype
    T = k.shape[0] if k.dim() == 3 else -1
    _activation(k, "k", (T, kv, D), dtype, dev)
    _activation(v, "v", (T, kv, D), dtype, dev)
    _dense(slots, "slots", torch.int64, dev, T)
    heads, qp, op, qs, os = 0, None, None, (0, 0), (0, 0)
    if q is not None:
        _need(q, "q", dtype, dev)
        heads = q.shape[1] if q.dim() == 3 else -1
        _activation(q, "q", (T, heads, D), dtype, dev)
        if q_out is None:
            q_out = _empty((T, heads, D), dtype, q)
        else:
            _result(q_out, "q_out", (T, heads, D), dtype, dev)
        qp, op, qs, os = q.data_ptr(), q_out.data_ptr(), _strides(q, T, heads), _strides(q_out, T, heads)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot, axes, inter, sections, freq, pos, ps = 0, 0, 0, _NO_SECTIONS, None, None, 0
    if rope is not None:
        if not isinstance(rope, Rope):
            raise TypeError("rope must be a Rope")
        _need(positions, "positions", torch.int32, dev)
        if rope.device != dev:
            raise ValueError(f"rope is on {rope.device}, expected {dev}")
        axes = rope.axes
        if tuple(positions.shape) != (axes, T) and not (axes == 1 and tuple(positions.shape) == (T,)):
            raise ValueError(f"positions must be {[axes, T]}, got {list(positions.shape)}")
        if T > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous over the tokens")
        ps = positions.stride(0) if axes > 1 else 0
        rot, inter, sections = rope.rot, rope.interleaved, rope._sections
        freq, pos = rope._ptr, positions.data_ptr()
    elif positions is not None:
        raise ValueError("positions without rope")
    args = _lib.BqKvAppendArgs(_DTYPES[dtype], heads, rot, axes, inter, sections, T, k.data_ptr(),
                               v.data_ptr(), qp, op, *_strides(k, T, kv), *_strides(v, T, kv), *qs, *os,
                               slots.data_ptr(), pos, ps, freq)
    _call(lib.bq_kv_append, "kv_append", dev, cache._ref, _byref(args))
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
    length.  The work is cut by the table's width, not by the lengths: a table
    much wider than its requests leaves a part of the GPU idle (one request of
    8000 positions: 9 us in a table of that width, 26 in one of 131072).  out may be q.  workspace: uint8, ``paged_attention_workspace(...)`` bytes, one per
    call that may overlap others, also calls of two host threads on one stream;
    None: one of the call's own from PyTorch's allocator."""
    if not isinstance(cache, PagedKVCache):
        raise TypeError("cache must be a PagedKVCache")
    dev, D = cache.device, cache.head_dim
    if not 1 <= rows <= BQ_VERIFY_MAX_ROWS:
        raise ValueError(f"rows must be 1 to {BQ_VERIFY_MAX_ROWS}, got {rows}")
    _dense(lens, "lens", torch.int32, dev)
    n = lens.numel()
    _first(q, "q", dev)
    dtype = q.dtype
    T, heads = n * rows, (q.shape[1] if q.dim() == 3 else -1)
    shape = (T, heads, D)
    if q.shape != shape or not q.is_contiguous():
        _activation(q, "q", shape, dtype, dev)
    width, stride = _table(table, n, dev)
    if out is None:
        out = _empty(shape, dtype, q)
        os = (heads * D, D)
    else:
        _result(out, "out", shape, dtype, dev)
        os = _strides(out, T, heads)
    args = _lib.BqAttentionArgs(_DTYPES[dtype], n, rows, heads, width, cache._scale if scale is None else scale, stride,
                                *_strides(q, T, heads), *os, q.data_ptr(), out.data_ptr(),
                                table.data_ptr(), lens.data_ptr())
    ref = _byref(args)
    if workspace is None:
        key = (n, rows, heads, width)
        nbytes = cache._workspace.get(key)
        if nbytes is None:
            nbytes = lib.bq_paged_attention_workspace_bytes(cache._ref, ref)
            if nbytes >= 0:
                if len(cache._workspace) >= 1024:
                    cache._workspace.clear()
                cache._workspace[key] = nbytes
        # One of the call's own, not one that stays with the stream: two threads may
        # launch on it at once (the call is two kernels), a graph keeps what it captured,
        # and a handle does not say which stream it was.  The allocator hands it on in
        # the stream's order.
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
    args = _lib.BqAttentionArgs(_lib.BQ_F32, _i32(requests), _i32(rows), _i32(heads), _i32(width), 1.0, int(width))
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
    x'), x' of y's dtype (None without pre_gain).  y and h may be one tensor, and
    h_out and x_out, apart from one another, may each be y, h or a gate per row of
    their dtype."""
    _first(y, "y")
    dev, dtype, shape = y.device, y.dtype, y.shape
    if len(shape) != 2:
        raise ValueError("y must be [rows, width]")
    if not y.is_contiguous():
        _activation(y, "y", shape, dtype, dev)
    h_dtype = h.dtype if isinstance(h, _Tensor) else None
    if h_dtype is not dtype and h_dtype is not torch.float32:
        _need(h, "h")
        raise TypeError(f"h must be {dtype} or fp32, got {h_dtype}")
    _activation(h, "h", shape, h_dtype, dev)
    T, width = shape
    gp = post = pre = xp = None
    gs = xs = 0
    if gate is not None:
        one = gate.dim() == 1 if isinstance(gate, _Tensor) else False
        _activation(gate, "gate", (width,) if one else shape, dtype, dev)
        gp, gs = gate.data_ptr(), (0 if one or T < 2 else gate.stride(0))
    if post_gain is not None:
        _dense(post_gain, "post_gain", torch.float32, dev, width)
        post = post_gain.data_ptr()
    if h_out is None:
        h_out = _empty(shape, h_dtype, h)
    else:
        _result(h_out, "h_out", shape, h_dtype, dev)
    if pre_gain is not None:
        _dense(pre_gain, "pre_gain", torch.float32, dev, width)
        pre = pre_gain.data_ptr()
        if x_out is None:
            x_out = _empty(shape, dtype, y)
        else:
            _result(x_out, "x_out", shape, dtype, dev)
        xp, xs = x_out.data_ptr(), x_out.stride(0)
    elif x_out is not None:
        raise ValueError("x_out without pre_gain")
    ys, hs, hos = y.stride(0), h.stride(0), h_out.stride(0)
    if T < 2:
        ys = hs = hos = xs = 0
    args = _lib.BqSandwichArgs(_DTYPES[dtype], _DTYPES[h_dtype], T, width, y.data_ptr(), h.data_ptr(), gp, post, pre,
                               h_out.data_ptr(), xp, ys, hs, gs, hos, xs, alpha, beta, eps)
    _call(lib.bq_sandwich_norm, "sandwich_norm", dev, _byref(args))
    return h_out, x_out
