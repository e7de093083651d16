"""The GEMV weight stream of one batch-1 decode step.

A decoder layer's weight stream, in model order (RunIT README, data-flow
diagram: RMSNorm -> Q/K/V projections -> attention -> FFN gate/up -> SiLU ->
down -> ... -> lm_head):

    stage 4l+0: q, k, v        x = the layer input h
    stage 4l+1: o              x = q's output (stand-in for the attention
                               output, which has q's width)
    stage 4l+2: gate+up+SiLU   x = o's output, RMSNorm-ed with the layer gain
    stage 4l+3: down           x = the gate+up output; its output is the next
                               layer's input h
    last stage: LM head        x = the last layer's output

Attention itself, residual adds and the other norms are outside this stream
(they are not weight streaming).  Every op reads the previous stage's output,
so the stages are truly dependent, as in decode.  ``run_plan()`` runs the
stream through a plan (bq_stream_plan_*): one streaming-kernel launch per
stage, each waiting for the stage before (programmatic dependent launch; the
cooperative executor in one launch is the alternative); ``run_per_op()``
launches one kernel per op in stage order; the two give identical bits.

With ``chained=False`` every op instead reads an input vector of its own (the
same shapes and weights, no data flowing between ops): the pure per-token
weight stream, which a plan runs as ONE launch of the streaming kernel.

With ``fused_qkv=True`` each layer's q, k and v run as ONE op over their
rows concatenated at load time (``layer["qkv"]``, see ``concat_packed``)
with an optional fp32 bias (``layer["qkv_bias"]``): the fused QKV+bias
projection of the RunIT README (6 dispatches -> 1 per layer on the Qwen
path).  The op's output holds q, k and v back to back; o reads its q part.

``PagedDecode`` runs whole decoder layers, with what DecodeStream leaves out:
the norms, rotary positions, the paged key-value cache, attention over it and
the residual stream.
"""
import torch

from . import StreamOp, StreamPlan, gemv, gemv_gate_up_silu, gemv_qkv_bias, gemv_verify
from .cache import kv_append, paged_attention, paged_prefix_attention, sandwich_norm


class DecodeStream:
    def __init__(self, qtype, layers, lm_head, eps=1e-6, chained=True, fused_qkv=False):
        """layers: list of dicts with packed q, k, v, o, gate, up, down
        (uint8 [M, row bytes]) and gamma (fp32 [hidden]); with fused_qkv,
        packed qkv (the q, k, v rows concatenated) and optional qkv_bias
        (fp32) instead of q, k, v; lm_head: packed."""
        from . import _packed_shape, _qt
        self.qtype = _qt(qtype)
        self.eps = eps
        dev = lm_head.device
        self.layers = layers
        self.lm_head = lm_head
        f32 = dict(dtype=torch.float32, device=dev)

        def rows(P):
            return _packed_shape(P, self.qtype)

        hidden = rows(layers[0]["qkv" if fused_qkv else "q"])[1]
        self.fused_qkv = fused_qkv
        self.chained = chained
        # every vector the stream reads from outside lives in one buffer, so a
        # caller fills them with a single copy: x0 (chained), or x0 and one
        # input per op (unchained)
        n_in = hidden
        if not chained:
            for L in layers:
                n_in += rows(L["o"])[1] + hidden + rows(L["down"])[1] + hidden
        self.inputs = torch.zeros(n_in, **f32)
        self.x0 = self.inputs[:hidden]
        # likewise every op's output is a slice of one buffer, so a caller
        # reads them all back with a single copy; each slice starts on 16
        # bytes, as an output that a later stage reads as its x must
        def pad4(n):
            return (n + 3) // 4 * 4

        n_out = pad4(rows(lm_head)[0])
        for L in layers:
            n_out += sum(pad4(rows(L[n])[0]) for n in (("qkv",) if fused_qkv else ("q", "k", "v")))
            n_out += pad4(rows(L["o"])[0]) + pad4(rows(L["gate"])[0]) + pad4(rows(L["down"])[0])
        self.outputs = torch.zeros(n_out, **f32)
        ocursor = [0]

        def out(n):
            t = self.outputs[ocursor[0]:ocursor[0] + n]
            ocursor[0] += pad4(n)
            return t

        self.ops = []
        self.buffers = []
        cursor = [hidden]

        def src(produced, K):
            # chained: the producing op's output; otherwise an input of its own
            if chained:
                return produced
            t = self.inputs[cursor[0]:cursor[0] + K]
            cursor[0] += K
            return t

        h = self.x0
        st = 0
        for L in layers:
            q_dim = rows(L["o"])[1]  # o reads the attention output, q's width
            bufs = {}
            if fused_qkv:
                bufs["qkv"] = out(rows(L["qkv"])[0])
                bufs["q"] = bufs["qkv"][:q_dim]
                self.ops.append(StreamOp(st, L["qkv"], h, bufs["qkv"], bias=L.get("qkv_bias")))
            else:
                for n in ("q", "k", "v"):
                    bufs[n] = out(rows(L[n])[0])
                    self.ops.append(StreamOp(st, L[n], h, bufs[n]))
            bufs["o"] = out(rows(L["o"])[0])
            bufs["ffn"] = out(rows(L["gate"])[0])
            bufs["down"] = out(rows(L["down"])[0])
            self.buffers.append(bufs)
            self.ops.append(StreamOp(st + 1, L["o"], src(bufs["q"], q_dim), bufs["o"]))
            self.ops.append(StreamOp(st + 2, L["gate"], src(bufs["o"], hidden), bufs["ffn"],
                                     W_up=L["up"], gamma=L["gamma"], eps=eps))
            self.ops.append(StreamOp(st + 3, L["down"], src(bufs["ffn"], rows(L["down"])[1]),
                                     bufs["down"]))
            h = src(bufs["down"], hidden)
            st += 4
        self.logits = out(rows(lm_head)[0])
        assert ocursor[0] == n_out
        self.ops.append(StreamOp(st, lm_head, h, self.logits))
        self._plan = None

    @property
    def n_stages(self):
        return self.ops[-1].stage + 1

    def weight_bytes(self):
        n = 0
        for op in self.ops:
            n += op.W.numel() + (op.W_up.numel() if op.W_up is not None else 0)
        return n

    def activation_bytes(self):
        """Algorithmic activation traffic: every op reads x (and gamma or
        bias) and writes y once."""
        n = 0
        for op in self.ops:
            n += 4 * (op.x.numel() + op.y.numel())
            if op.gamma is not None:
                n += 4 * op.gamma.numel()
            if op.bias is not None:
                n += 4 * op.bias.numel()
        return n

    def plan(self):
        if self._plan is None:
            self._plan = StreamPlan(self.qtype, self.ops)
        return self._plan

    def run_plan(self):
        self.plan().launch()

    def run_per_op(self):
        for op in self.ops:
            if op.W_up is None and op.bias is not None:
                gemv_qkv_bias(self.qtype, op.W, op.x, op.bias, op.y)
            elif op.W_up is None:
                gemv(self.qtype, op.W, op.x, op.y)
            else:
                gemv_gate_up_silu(self.qtype, op.W, op.W_up, op.x, op.gamma, op.eps, op.y)


class PagedDecode:
    """A decode step of whole decoder layers over a paged key-value cache, for
    up to BQ_VERIFY_MAX_ROWS tokens at once: one token of each of several
    requests, or the rows of a verify step.

        x  = RMSNorm(h) * attn_gamma
        q, k, v = Wqkv x (+ bias), q and k turned by their positions
                                   [normed per head by q_norm, k_norm first if given]
        a  = attention of q over the cache, k and v appended
        h  = alpha h + beta attn_gate (o a)     [(o a) normed by attn_post if given]
        x  = RMSNorm(h) * gamma
        h  = alpha h + beta ffn_gate (down (silu(gate x) * up x))   [normed by ffn_post]
    then logits = lm_head (RMSNorm(h) * final_gamma).

    Every product is the package's GEMV (or its verify form, whose rows have the
    single row's bits; the gate and up pair, which has no verify form, runs once per
    row and reads its weights as often), and the calls between them compute each row
    on its own, so a row of a verify step has the bits of the one-row step (but with
    ``shared`` pages, whose attention cuts its sums by the whole step).
    ``step`` enqueues kernels only and can be captured in a CUDA graph."""

    def __init__(self, qtype, layers, lm_head, final_gamma, caches, heads, rope, eps=1e-6, alpha=1.0, beta=1.0,
                 rows=1):
        """layers: dicts with packed qkv (the q, k, v rows concatenated, see
        concat_packed), o, gate, up, down, fp32 [hidden] attn_gamma and gamma, and
        optionally qkv_bias (fp32), attn_post, ffn_post (fp32 [hidden] gains of a
        norm after the block), attn_gate, ffn_gate (fp32 [hidden]), q_norm, k_norm
        (fp32 [head_dim] gains of the norms of queries and keys); caches: one
        PagedKVCache per layer; heads: query heads; rope: a Rope or None; rows:
        tokens of a step."""
        from . import _packed_shape, _qt
        from ._lib import BQ_VERIFY_MAX_ROWS
        if not 1 <= rows <= BQ_VERIFY_MAX_ROWS:
            raise ValueError(f"rows must be 1 to {BQ_VERIFY_MAX_ROWS}, got {rows}")
        if not layers or len(caches) != len(layers):
            raise ValueError("one cache per layer")
        self.qtype, self.layers, self.lm_head, self.caches = _qt(qtype), layers, lm_head, caches
        self.final_gamma, self.rope, self.eps, self.alpha, self.beta = final_gamma, rope, eps, alpha, beta
        self.rows, self.heads = rows, heads
        kv, D = caches[0].kv_heads, caches[0].head_dim
        M, hidden = _packed_shape(layers[0]["qkv"], self.qtype)
        if M != (heads + 2 * kv) * D:
            raise ValueError(f"qkv has {M} rows, heads and cache need {(heads + 2 * kv) * D}")
        inter = _packed_shape(layers[0]["gate"], self.qtype)[0]
        vocab = _packed_shape(lm_head, self.qtype)[0]
        f32 = dict(dtype=torch.float32, device=lm_head.device)
        self.h = torch.zeros((rows, hidden), **f32)
        self._x = torch.zeros((rows, hidden), **f32)
        self._qkv = torch.zeros((rows, M), **f32)
        self._q, self._k, self._v = (t.view(rows, -1, D) for t in self._qkv.split([heads * D, kv * D, kv * D], dim=1))
        self._turned = torch.zeros((rows, heads, D), **f32)
        self._a = torch.zeros((rows, heads, D), **f32)
        self._y = torch.zeros((rows, hidden), **f32)
        self._ffn = torch.zeros((rows, inter), **f32)
        self.logits = torch.zeros((rows, vocab), **f32)

    def _product(self, W, x, y):
        if self.rows == 1:
            gemv(self.qtype, W, x[0], y[0])
        else:
            gemv_verify(self.qtype, W, x, y)

    def _between(self, gain, post=None, gate=None):
        """Residual add of the block's output and the norm before the next block."""
        sandwich_norm(self._y, self.h, pre_gain=gain, post_gain=post, gate=gate, alpha=self.alpha, beta=self.beta,
                      eps=self.eps, h_out=self.h, x_out=self._x)

    def step(self, h, slots, positions, table, lens, shared=None):
        """One step: h fp32 [rows, hidden] the tokens' embeddings; slots int64
        [rows] and positions int32 ([rows], or [axes, rows]) of the new tokens, as
        kv_block_tables gives them; table, lens: the requests' tables and lengths,
        the new tokens counted (rows / requests tokens each).  shared: the positions
        that the requests share, or groups of them, as for paged_prefix_attention
        (their pages are then read once for all of them, and the logits are those of a
        step without it but for the last bits).  Returns logits [rows, vocab], a buffer
        of this object."""
        requests = lens.numel()
        if requests < 1 or self.rows % requests:
            raise ValueError(f"{self.rows} rows do not share out among {requests} requests")
        each = self.rows // requests
        rope = self.rope
        if h.shape != self.h.shape and not (self.rows == 1 and h.shape == self.h.shape[1:]):
            raise ValueError(f"h must be {list(self.h.shape)}, got {list(h.shape)}")
        self.h.copy_(h)
        # x = RMSNorm(h) * attn_gamma
        sandwich_norm(self.h, self.h, pre_gain=self.layers[0]["attn_gamma"], alpha=1.0, beta=0.0, eps=self.eps,
                      h_out=self.h, x_out=self._x)
        for l, L in enumerate(self.layers):
            bias = L.get("qkv_bias")
            if self.rows == 1:
                gemv_qkv_bias(self.qtype, L["qkv"], self._x[0], bias, self._qkv[0])
            else:
                gemv_verify(self.qtype, L["qkv"], self._x, self._qkv)
                if bias is not None:
                    self._qkv.add_(bias)  # the fused call's one fp32 add
            kv_append(self.caches[l], self._k, self._v, slots, q=self._q, q_out=self._turned, rope=rope,
                      positions=None if rope is None else positions, q_norm=L.get("q_norm"), k_norm=L.get("k_norm"),
                      eps=self.eps)
            if shared is None:
                paged_attention(self.caches[l], self._turned, table, lens, rows=each, out=self._a)
            else:
                paged_prefix_attention(self.caches[l], self._turned, table, lens, shared, rows=each, out=self._a)
            self._product(L["o"], self._a.view(self.rows, -1), self._y)
            self._between(L["gamma"], L.get("attn_post"), L.get("attn_gate"))
            for r in range(self.rows):
                gemv_gate_up_silu(self.qtype, L["gate"], L["up"], self._x[r], None, self.eps, self._ffn[r])
            self._product(L["down"], self._ffn, self._y)
            last = l + 1 == len(self.layers)
            self._between(self.final_gamma if last else self.layers[l + 1]["attn_gamma"], L.get("ffn_post"),
                          L.get("ffn_gate"))
        self._product(self.lm_head, self._x, self.logits)
        return self.logits
