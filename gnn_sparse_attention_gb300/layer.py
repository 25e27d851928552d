"""PyTorch layers over the fused graph-attention kernels.

"On Efficient Scaling of GNNs via IO-Aware Layers Implementations", zh/ko
technical summaries, "Methodology" (the layers are meant as drop-in
replacements) and results (GATv2: peak memory cut because no edge-wise
tensor is materialised).

``graph_attention`` is an autograd function whose forward is ``gattn_fwd``
and whose backward is ``gattn_bwd``: it saves only the node tensors (Q, K, V,
out) and the per-node lse, never an O(M*H) edge tensor.  The two modules put
the usual projections around it (plain dense GEMMs, run by torch/cuBLAS):

* ``GraphTransformerConv``: Q, K, V = x W_q, x W_k, x W_v (H heads of D),
  dot-product attention over the in-neighbours, heads concatenated, output
  projection W_o.
* ``GATv2Conv``: x_l = x W_l, x_r = x W_r; score a . LeakyReLU(x_l[i] +
  x_r[j]), the message of source j is x_r[j] (one tensor passed as both K
  and V; its gradient is dK + dV), heads concatenated.

Both run the attention in the dtype of their parameters (bf16 by default)
with fp32 arithmetic inside the kernels.

Next to the attention over given edges stand the other parts of a transformer
layer: ``block_attention`` (attention over blocks of nodes that a cheap score
selects, ``gattn_block_select`` / ``gattn_block_fwd`` / ``gattn_block_bwd``),
``gated_residual_norm`` (the norms around a block with its gate and residual,
``gattn_norm_fwd`` / ``gattn_norm_bwd``), and ``GraphTransformerBlock``, which
puts them together: local attention over the edges plus global attention over
the selected blocks, then an MLP, each behind a norm and added through a gate.
"""
from __future__ import annotations

import math

import torch
from torch import nn

from . import binding as gb


class _GraphAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, kind, scale, slope, Q, K, V, a):
        score = gb.Score(kind, scale=scale, a=a, neg_slope=slope)
        out, lse = gb.gattn_fwd(plan, Q, K, V, score)
        ctx.plan, ctx.score = plan, score
        ctx.save_for_backward(Q, K, V, out, lse, a if a is not None else torch.empty(0))
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _dlse):
        Q, K, V, out, lse, a = ctx.saved_tensors
        dout = dout.to(Q.dtype).contiguous()
        dQ, dK, dV, da = gb.gattn_bwd(ctx.plan, Q, K, V, out, dout, lse, ctx.score)
        return None, None, None, None, dQ, dK, dV, da


def graph_attention(plan: gb.Plan, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                    kind: str = "dot", scale: float = 0.0, a: torch.Tensor | None = None,
                    neg_slope: float = 0.2):
    """Fused softmax attention over each destination's in-neighbours.

    Q, K, V: contiguous CUDA [N, H, D] (fp32 or bf16); for ``kind="gatv2"``
    ``a`` is a contiguous fp32 CUDA [H, D] parameter.  Returns (out [N, H, D],
    lse fp32 [N, H]); differentiable in Q, K, V and a.
    """
    if kind == "gatv2" and (a is None or a.dtype != torch.float32 or not a.is_contiguous()):
        raise ValueError("GATv2 needs a contiguous fp32 tensor a of shape [H, D]")
    return _GraphAttention.apply(plan, kind, float(scale), float(neg_slope), Q.contiguous(),
                                 K.contiguous(), V.contiguous(), a if kind == "gatv2" else None)


class GraphTransformerConv(nn.Module):
    """Multi-head graph-transformer attention layer (dot score)."""

    def __init__(self, in_dim: int, heads: int, head_dim: int, out_dim: int | None = None,
                 dtype=torch.bfloat16, device=None):
        super().__init__()
        self.heads, self.head_dim = heads, head_dim
        hd = heads * head_dim
        kw = {"dtype": dtype, "device": device}
        self.q = nn.Linear(in_dim, hd, bias=False, **kw)
        self.k = nn.Linear(in_dim, hd, bias=False, **kw)
        self.v = nn.Linear(in_dim, hd, bias=False, **kw)
        self.o = nn.Linear(hd, out_dim or hd, bias=False, **kw)

    def forward(self, x: torch.Tensor, plan: gb.Plan) -> torch.Tensor:
        N = x.shape[0]
        shape = (N, self.heads, self.head_dim)
        Q, K, V = (p(x).view(shape) for p in (self.q, self.k, self.v))
        out, _ = graph_attention(plan, Q, K, V, "dot", 1.0 / math.sqrt(self.head_dim))
        return self.o(out.reshape(N, self.heads * self.head_dim))


class GATv2Conv(nn.Module):
    """Multi-head GATv2 attention layer (messages x_r[j], heads concatenated)."""

    def __init__(self, in_dim: int, heads: int, head_dim: int, negative_slope: float = 0.2,
                 dtype=torch.bfloat16, device=None):
        super().__init__()
        self.heads, self.head_dim, self.slope = heads, head_dim, negative_slope
        hd = heads * head_dim
        kw = {"dtype": dtype, "device": device}
        self.lin_l = nn.Linear(in_dim, hd, bias=False, **kw)
        self.lin_r = nn.Linear(in_dim, hd, bias=False, **kw)
        self.att = nn.Parameter(torch.randn(heads, head_dim, device=device) / math.sqrt(head_dim))

    def forward(self, x: torch.Tensor, plan: gb.Plan) -> torch.Tensor:
        N = x.shape[0]
        shape = (N, self.heads, self.head_dim)
        xl = self.lin_l(x).view(shape)
        xr = self.lin_r(x).view(shape)
        out, _ = graph_attention(plan, xl, xr, xr, "gatv2", a=self.att, neg_slope=self.slope)
        return out.reshape(N, self.heads * self.head_dim)


def _packed(t: torch.Tensor | None) -> torch.Tensor | None:
    """t as the kernels read it, contiguous from a 16-byte border on: a copy where it is not, as
    with a column slice, or with rows of an odd size that start in the middle of a tensor."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _Once(torch.autograd.Function):
    """The first n tensors, as functions of the others that cannot be differentiated."""

    @staticmethod
    def forward(ctx, n, *ts):
        return tuple(t.view_as(t) for t in ts[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("block_attention and gated_residual_norm are differentiable once only")


def _once(grads, *roots):
    """Gradients of a kernel under create_graph: a second derivative is refused, not left out."""
    if not torch.is_grad_enabled():
        return grads
    some = [g for g in grads if g is not None]
    done = iter(_Once.apply(len(some), *some, *(t for t in roots if t is not None)))
    return tuple(None if g is None else next(done) for g in grads)


class _BlockAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, idx, seq_q, seq_k, len_k, block, q_block, scale, causal):
        # rows of no sequence are not written by the kernels: zeros
        out = torch.zeros_like(Q)
        lse = torch.zeros(Q.shape[:2], dtype=torch.float32, device=Q.device)
        ctx.args = {"block": block, "q_block": q_block, "scale": scale, "causal": causal}
        gb.gattn_block_fwd(Q, K, V, idx, seq_q, seq_k, len_k=len_k, out=out, lse=lse, **ctx.args)
        ctx.has_len = len_k is not None
        ctx.save_for_backward(Q, K, V, idx, seq_q, seq_k, out, lse,
                              *((len_k,) if ctx.has_len else ()))
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _dlse):
        Q, K, V, idx, seq_q, seq_k, out, lse, *more = ctx.saved_tensors
        dQ, dK, dV = (torch.zeros_like(t) for t in (Q, K, V))
        gb.gattn_block_bwd(Q, K, V, idx, seq_q, seq_k, out, _packed(dout.to(Q.dtype)), lse,
                           len_k=more[0] if ctx.has_len else None, dQ=dQ, dK=dK, dV=dV, **ctx.args)
        return _once((dQ, dK, dV), Q, K, V, dout) + (None,) * 8


def block_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seq: torch.Tensor,
                    topk: int = 16, block: int = 64, q_block: int = 64, causal: bool = False,
                    scale: float = 0.0, seq_k: torch.Tensor | None = None,
                    len_k: torch.Tensor | None = None, idx: torch.Tensor | None = None,
                    max_len_k: int = 0):
    """Softmax attention of each query over the ``topk`` blocks of its own sequence that score
    highest for its unit of ``q_block`` queries.

    Q: [Nq, H, D]; K, V: [Nk, Hkv, D]; seq: int32 [S + 1], the sequences' (graphs') first
    rows; seq_k and len_k (both optional) give the keys their own offsets and lengths.  ``idx``
    (int32 [units, Hkv, blocks], see gattn_block_select) replaces the choice; ``max_len_k``, the
    most keys of one sequence (0: all rows), keeps its score tables small (without it a batch may
    have about 27,900 blocks together).  Returns
    (out [Nq, H, D], lse fp32 [Nq, H], idx).  out is differentiable in Q, K and V, once, and not
    in the choice; lse carries no gradient.  Rows of no sequence get zeros.  Kernels that give up
    a bounded wait leave their results undefined and raise nothing here: gattn_block_check_errors,
    which synchronises, tells.
    """
    Q, K, V = _packed(Q), _packed(K), _packed(V)
    keys = seq if seq_k is None else seq_k
    if idx is None:
        with torch.no_grad():
            sums = gb.gattn_block_sums(K, keys, block, lens=len_k)
            idx = gb.gattn_block_select(Q, sums, seq, keys, topk, block, q_block, K.shape[0],
                                        len_k=len_k, causal=causal, max_len_k=max_len_k)
    out, lse = _BlockAttention.apply(Q, K, V, idx, seq, keys, len_k, block, q_block,
                                     float(scale), causal)
    return out, lse, idx


class _GatedResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, res, x, gate, w_post, b_post, w_pre, b_pre, alpha, kind, eps):
        h, y, stats = gb.gattn_norm_fwd(res, x, gate, w_post, b_post, w_pre, b_pre, alpha, kind,
                                        eps)
        some = (res, stats, x, gate, w_post, b_post, w_pre, b_pre)
        ctx.present = [t is not None for t in some]
        ctx.alpha, ctx.kind = alpha, kind
        ctx.save_for_backward(*(t for t in some if t is not None))
        ctx.set_materialize_grads(False)
        return (h.view_as(h) if x is None else h), y

    @staticmethod
    def backward(ctx, dh, dy):
        saved = iter(ctx.saved_tensors)
        res, stats, x, gate, w_post, b_post, w_pre, b_pre = (
            next(saved) if there else None for there in ctx.present)
        dh, dy = (None if t is None else _packed(t.to(res.dtype)) for t in (dh, dy))
        if dy is None and w_pre is not None:
            dy = torch.zeros_like(res)
        if dh is None and dy is None:
            return (None,) * 10
        g = gb.gattn_norm_bwd(res, stats, dh, dy, x, gate, w_post, b_post, w_pre, b_pre,
                              ctx.alpha, ctx.kind)
        return _once((g["dres"], g["dx"], g["dgate"], g["dw_post"], g["db_post"], g["dw_pre"],
                      g["db_pre"]), res, x, gate, w_post, b_post, w_pre, b_pre, dh, dy) + (None,) * 3


def gated_residual_norm(res: torch.Tensor, x: torch.Tensor | None = None,
                        gate: torch.Tensor | None = None, w_post=None, b_post=None, w_pre=None,
                        b_pre=None, alpha: float = 1.0, kind: str = "rms", eps: float = 1e-6):
    """(h, y): h = res + alpha * gate * norm(x; w_post, b_post), y = norm(h; w_pre, b_pre).

    res, x: [N, F] rows (fp32 or bf16); gate: [N, F] like them, or fp32 [F]; weights and biases
    fp32 [F].  Parts left out are skipped (see gattn_norm_fwd); y is None without w_pre.
    Differentiable in every tensor, once.  Tensors that are not contiguous, or not aligned to 16
    bytes, are copied, and vectors of another type (of a module that was cast whole) converted.
    """
    res, x, gate, w_post, b_post, w_pre, b_pre = (
        _packed(t.float() if t is not None and t.dim() == 1 else t)
        for t in (res, x, gate, w_post, b_post, w_pre, b_pre))
    return _GatedResidualNorm.apply(res, x, gate, w_post, b_post, w_pre, b_pre, float(alpha), kind,
                                    float(eps))


class GraphTransformerBlock(nn.Module):
    """A transformer layer over the nodes of a batch of graphs.

    h = h + gate_a * norm(W_o (local + global)), where local is the attention over the plan's
    edges (left out without a plan) and global that over the selected blocks of the node's own
    graph, both on the same heads of norm(h); then h = h + gate_m * norm(MLP(norm(h))).  The
    gates are learned per channel.  ``seq`` holds the graphs' first node rows, ``max_nodes``
    (0: unknown) the size of the largest graph; see block_attention for both, and for errors.
    """

    def __init__(self, dim: int, heads: int, head_dim: int, mlp_dim: int | None = None,
                 topk: int = 16, block: int = 64, q_block: int = 64, causal: bool = False,
                 kind: str = "rms", gate_init: float = 1.0, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.heads, self.head_dim, self.kind = heads, head_dim, kind
        self.choice = {"topk": topk, "block": block, "q_block": q_block, "causal": causal}
        kw = {"dtype": dtype, "device": device}
        hd = heads * head_dim
        self.qkv = nn.Linear(dim, 3 * hd, bias=False, **kw)
        self.o = nn.Linear(hd, dim, bias=False, **kw)
        self.up = nn.Linear(dim, mlp_dim or 4 * dim, bias=False, **kw)
        self.down = nn.Linear(mlp_dim or 4 * dim, dim, bias=False, **kw)

        def vector(value):
            return nn.Parameter(torch.full((dim,), float(value), device=device))

        for name in ("in", "attn", "mid", "mlp"):
            setattr(self, f"w_{name}", vector(1.0))
            setattr(self, f"b_{name}", vector(0.0) if kind == "layer" else None)
        self.gate_attn, self.gate_mlp = vector(gate_init), vector(gate_init)

    def forward(self, h: torch.Tensor, seq: torch.Tensor, plan: gb.Plan | None = None,
                idx: torch.Tensor | None = None, max_nodes: int = 0) -> torch.Tensor:
        N = h.shape[0]
        h, y = gated_residual_norm(h, w_pre=self.w_in, b_pre=self.b_in, kind=self.kind)
        Q, K, V = (t.reshape(N, self.heads, self.head_dim) for t in self.qkv(y).chunk(3, -1))
        Q, K, V = Q.contiguous(), K.contiguous(), V.contiguous()
        a, _, _ = block_attention(Q, K, V, seq, idx=idx, max_len_k=max_nodes, **self.choice)
        if plan is not None:
            a = a + graph_attention(plan, Q, K, V, "dot", 1.0 / math.sqrt(self.head_dim))[0]
        a = self.o(a.reshape(N, self.heads * self.head_dim))
        h, y = gated_residual_norm(h, a, self.gate_attn, self.w_attn, self.b_attn, self.w_mid,
                                   self.b_mid, kind=self.kind)
        m = self.down(nn.functional.gelu(self.up(y)))
        h, _ = gated_residual_norm(h, m, self.gate_mlp, self.w_mlp, self.b_mlp, kind=self.kind)
        return h
