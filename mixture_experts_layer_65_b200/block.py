"""The norms before and after a block, fused with its gate, the residual scale and the
residual add (moe_block_norm* in include/moe.h), forward and backward; and `MoEBlock`, a layer
between them.

Per row, s(v) = 1 / sqrt(mean(v^2) + eps):
  r = beta x + gate p,  p = y s(y) post_weight   (p = y without post_weight)
  u = r s(r) pre_weight                          (the next block's input)
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._call import DTYPES, check_tensor, on_stream, rows_of
from ._lib import check, lib
from .clip import clip_grad_norm
from .layer import MoELayer, MoEOutput, _ptr

GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2


class BlockNorm(NamedTuple):
    r: torch.Tensor                  # [T, d] the residual stream after the block
    u: torch.Tensor | None           # [T, d] the next block's input (pre_weight given)
    post_rstd: torch.Tensor | None   # [T] fp32 (post_weight given)
    pre_rstd: torch.Tensor | None    # [T] fp32 (pre_weight given)


class BlockNormGrads(NamedTuple):
    dx: torch.Tensor                     # [T, d]
    dy: torch.Tensor | None              # [T, d] (y given)
    d_gate: torch.Tensor | None          # fp32, the gate's shape
    d_post_weight: torch.Tensor | None   # [d] fp32
    d_pre_weight: torch.Tensor | None    # [d] fp32


def _params(dev, rows, d, gate, post_weight, pre_weight) -> int:
    """Check the parameters; the gate's kind."""
    kind = GATE_NONE
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise ValueError("gate must be a tensor")
        kind = GATE_TOKEN if gate.dim() == 2 else GATE_CHANNEL
        check_tensor("gate (one value per channel [d], or per token [T, 1])", gate, dev,
                     (rows, 1) if kind == GATE_TOKEN else (d,), torch.float32)
    if post_weight is not None:
        check_tensor("post_weight", post_weight, dev, (d,), torch.float32)
    if pre_weight is not None:
        check_tensor("pre_weight", pre_weight, dev, (d,), torch.float32)
    return kind


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, *, gate: torch.Tensor | None = None,
               post_weight: torch.Tensor | None = None, pre_weight: torch.Tensor | None = None,
               beta: float = 1.0, eps: float = 1e-6, out: BlockNorm | None = None,
               stream: torch.cuda.Stream | None = None) -> BlockNorm:
    """The step between two blocks.  x [T, d] the residual stream, y [T, d] the block's output
    (None: only the norm before the first block, r is x itself); gate fp32 [d] per channel or
    [T, 1] per token; weights fp32 [d].  `out` may reuse x or y as r or u."""
    dev, rows, d, dt = rows_of("x", x)
    if y is not None:
        check_tensor("y", y, dev, (rows, d), dt)
    kind = _params(dev, rows, d, gate, post_weight, pre_weight)
    if out is not None:
        if (out.u is not None) != (pre_weight is not None) or \
                (out.pre_rstd is not None) != (pre_weight is not None) or \
                (out.post_rstd is not None) != (post_weight is not None):
            raise ValueError("out.u and out.pre_rstd go with pre_weight, out.post_rstd with post_weight")
        if y is not None:
            check_tensor("out.r", out.r, dev, (rows, d), dt)
        if pre_weight is not None:
            check_tensor("out.u", out.u, dev, (rows, d), dt)
            check_tensor("out.pre_rstd", out.pre_rstd, dev, (rows,), torch.float32)
        if post_weight is not None:
            check_tensor("out.post_rstd", out.post_rstd, dev, (rows,), torch.float32)
    with on_stream(dev, stream, (x, y, gate, post_weight, pre_weight, *(out or ()))) as s:
        if out is None:
            out = BlockNorm(
                r=torch.empty_like(x) if y is not None else x,
                u=torch.empty_like(x) if pre_weight is not None else None,
                post_rstd=torch.empty(rows, dtype=torch.float32, device=dev) if post_weight is not None else None,
                pre_rstd=torch.empty(rows, dtype=torch.float32, device=dev) if pre_weight is not None else None)
        elif y is None:
            out = out._replace(r=x)
        check(lib().moe_block_norm(_ptr(x), _ptr(y), _ptr(gate), kind, _ptr(post_weight), _ptr(pre_weight),
                                   rows, d, DTYPES[dt], beta, eps,
                                   _ptr(out.r) if y is not None else None, _ptr(out.u),
                                   _ptr(out.post_rstd), _ptr(out.pre_rstd), s))
    return out


def block_norm_backward(fwd: BlockNorm, y: torch.Tensor | None, *, dr: torch.Tensor | None = None,
                        du: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                        post_weight: torch.Tensor | None = None, pre_weight: torch.Tensor | None = None,
                        beta: float = 1.0, stream: torch.cuda.Stream | None = None) -> BlockNormGrads:
    """Gradients of block_norm from dr and du, the gradients of its r and u: `fwd` is its
    result (u is not read), y and the parameters are its arguments.  dr may be None (zero)
    when pre_weight is given."""
    dev, rows, d, dt = rows_of("fwd.r", fwd.r)
    kind = _params(dev, rows, d, gate, post_weight, pre_weight)
    for name, t in (("y", y), ("dr", dr), ("du", du)):
        if t is not None:
            check_tensor(name, t, dev, (rows, d), dt)
    if (du is not None) != (pre_weight is not None):
        raise ValueError("du goes with pre_weight")
    if dr is None and pre_weight is None:
        raise ValueError("dr is required without pre_weight")
    if post_weight is not None:
        check_tensor("fwd.post_rstd", fwd.post_rstd, dev, (rows,), torch.float32)
    if pre_weight is not None:
        check_tensor("fwd.pre_rstd", fwd.pre_rstd, dev, (rows,), torch.float32)
    with on_stream(dev, stream, (fwd.r, y, dr, du, gate, post_weight, pre_weight, fwd.post_rstd,
                                 fwd.pre_rstd)) as s:
        g = BlockNormGrads(
            dx=torch.empty_like(fwd.r), dy=torch.empty_like(fwd.r) if y is not None else None,
            d_gate=torch.empty_like(gate) if gate is not None else None,
            d_post_weight=torch.empty_like(post_weight) if post_weight is not None else None,
            d_pre_weight=torch.empty_like(pre_weight) if pre_weight is not None else None)
        L = lib()
        size = L.moe_block_norm_workspace(rows, d)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        check(L.moe_block_norm_backward(
            _ptr(y), fwd.r.data_ptr(), _ptr(dr), _ptr(du), _ptr(gate), kind, _ptr(post_weight), _ptr(pre_weight),
            fwd.post_rstd.data_ptr() if post_weight is not None else None,
            fwd.pre_rstd.data_ptr() if pre_weight is not None else None, rows, d, DTYPES[dt], beta,
            g.dx.data_ptr(), _ptr(g.dy), _ptr(g.d_gate), _ptr(g.d_post_weight), _ptr(g.d_pre_weight),
            ws.data_ptr(), size, s))
    return g


class MoEBlockOutput(NamedTuple):
    r: torch.Tensor              # [T, d] the residual stream after the block
    norm_in: BlockNorm           # the norm before the layer: its u is the layer's input
    layer: MoEOutput             # the layer without its residual
    norm_out: BlockNorm          # r, and the next block's input when next_weight was given


class MoEBlockGrads(NamedTuple):
    dx: torch.Tensor                     # [T, d]; with norm_in given to forward: without its part
    du: torch.Tensor | None              # that part: the gradient of norm_in.u (norm_in given)
    d_gate: torch.Tensor | None
    d_post_weight: torch.Tensor | None
    d_pre_weight: torch.Tensor | None    # (None when norm_in was given)
    d_next_weight: torch.Tensor | None
    d_centroids: torch.Tensor
    d_bias: torch.Tensor
    d_w_gate: torch.Tensor | None
    d_w_up: torch.Tensor | None
    d_w_down: torch.Tensor | None
    grad_norm: torch.Tensor | None       # [1] fp32, before clipping (max_norm given)
    inputs: tuple = ()                   # names of the fields above that are no parameter's gradient

    def parameters(self) -> list:
        """The parameters' gradients that there are, which `max_norm` clips.  A gradient that is
        no parameter's (`inputs`: d_gate when the gate was given to the call, a value per token
        among them; d_bias of a layer without a logit_bias) keeps its place in the list as a
        tensor of no elements: it neither counts in the norm nor is scaled."""
        return [t[:0] if name in self.inputs else t
                for name, t in zip(self._fields[2:11], self[2:11]) if t is not None]


class MoEBlock:
    """r = beta x + gate * norm(FFN(norm(x))): a MoELayer (its experts without its own residual)
    between the norms.  pre_weight [d], optional post_weight [d] and gate ([d], or [T, 1] given to
    each call) are fp32.  The block's own gate is a parameter; one given to a call is an input.

    In a stack, `next_weight` of one block's forward is the next block's pre_weight: the step
    between two blocks is then one kernel, and its norm goes to the next forward as `norm_in`
    (out.norm_out); the gradients go back the same way, dx and du of the later block as dr and du
    of the earlier one's backward."""

    def __init__(self, layer: MoELayer, pre_weight: torch.Tensor, post_weight: torch.Tensor | None = None,
                 gate: torch.Tensor | None = None, beta: float = 1.0, eps: float = 1e-6):
        self.layer, self.pre_weight, self.post_weight = layer, pre_weight, post_weight
        self.gate, self.beta, self.eps = gate, beta, eps

    def forward(self, x: torch.Tensor, *, gate: torch.Tensor | None = None, norm_in: BlockNorm | None = None,
                next_weight: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> MoEBlockOutput:
        """`gate` replaces the block's own for this call; norm_in: the norm of x, computed by the
        block before (its r is x itself)."""
        if norm_in is None:
            norm_in = block_norm(x, pre_weight=self.pre_weight, eps=self.eps, stream=stream)
        elif norm_in.u is None:
            raise ValueError("norm_in has no u: give the earlier block this block's pre_weight as next_weight")
        elif norm_in.r.data_ptr() != x.data_ptr() or norm_in.r.shape != x.shape:
            raise ValueError("norm_in is the norm of another tensor: its r must be x")
        with on_stream(x.device, stream, (norm_in.u,)):
            out = self.layer.forward_branch(norm_in.u)
        norm_out = block_norm(x, out.h, gate=self.gate if gate is None else gate, post_weight=self.post_weight,
                              pre_weight=next_weight, beta=self.beta, eps=self.eps, stream=stream)
        return MoEBlockOutput(norm_out.r, norm_in, out, norm_out)

    __call__ = forward

    def backward(self, out: MoEBlockOutput, dr: torch.Tensor | None, du: torch.Tensor | None = None, *,
                 d_aux: float = 0.0, gate: torch.Tensor | None = None, norm_in_given: bool = False,
                 next_weight: torch.Tensor | None = None, weights: bool = True,
                 max_norm: float | None = None, stream: torch.cuda.Stream | None = None) -> MoEBlockGrads:
        """Gradients of sum(dr r) + sum(du u_next) + d_aux aux after `forward` (the layer's last
        one; the same gate, next_weight and whether norm_in was given).  max_norm: the parameters'
        gradients (`MoEBlockGrads.parameters`) are clipped to it together, and their norm before
        is returned; dx, du and the gradient of a gate given to the call stay as they are."""
        after = block_norm_backward(out.norm_out, out.layer.h, dr=dr, du=du,
                                    gate=self.gate if gate is None else gate, post_weight=self.post_weight,
                                    pre_weight=next_weight, beta=self.beta, stream=stream)
        with on_stream(out.r.device, stream, (out.norm_in.u, *out.layer)):
            d_in, *rest = self.layer.backward_branch(out.norm_in.u, out.layer, after.dy, d_aux, weights)
        dx, d_pre = after.dx, None
        if not norm_in_given:
            before = block_norm_backward(out.norm_in, None, dr=after.dx, du=d_in, pre_weight=self.pre_weight,
                                         stream=stream)
            dx, d_pre, d_in = before.dx, before.d_pre_weight, None
        # (one value per token is an input whoever holds it)
        own_gate = (gate is None or gate is self.gate) and (self.gate is None or self.gate.dim() == 1)
        inputs = (() if own_gate else ("d_gate",)) + (() if self.layer.has_bias else ("d_bias",))
        g = MoEBlockGrads(dx, d_in, after.d_gate, after.d_post_weight, d_pre, after.d_pre_weight, *rest, None, inputs)
        if max_norm is not None:
            g = g._replace(grad_norm=clip_grad_norm(g.parameters(), max_norm, stream=stream))
        return g
