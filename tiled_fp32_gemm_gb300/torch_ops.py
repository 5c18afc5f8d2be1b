"""Torch operator registrations for the library's products, the feed-forward
operators, the residual joins and the vocabulary's loss.

Importing this module registers ``torch.ops.mt.sgemm(a, b)``,
``torch.ops.mt.gemm_bias(a, b, bias)``, ``torch.ops.mt.linear``,
``torch.ops.mt.rms_norm``, ``torch.ops.mt.layer_norm``, ``torch.ops.mt.dropout``
and ``torch.ops.mt.linear_cross_entropy`` as torch custom operators: the same
C-ABI calls as the functions of those names (``gemm(..., bias=...)``), visible
to torch's dispatcher, graph capture and tracing (each has a shape-only fake
implementation, so tracing needs no GPU).  Tracing takes them forwards: a backward
pass is captured in a graph but not traced (``torch.compile`` of one raises).  All
but the first two are differentiable, once: their gradients are the ``*_backward`` functions (for
dropout, dropout itself), which have none themselves, so a second derivative
raises.  A seed that is advanced in place between an operator and its gradient
raises too: torch notices it.  No gradient of zeros is made for an output that
nothing reads.  Marshalling only: the work runs in the library's kernels.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import (dropout, gemm, layer_norm, layer_norm_backward, linear, linear_backward,
               linear_cross_entropy, linear_cross_entropy_backward, rms_norm, rms_norm_backward,
               sgemm)


@torch.library.custom_op("mt::sgemm", mutates_args=())
def sgemm_op(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """a @ b (float32, CUDA, row-major) through mt_sgemm_ex."""
    return sgemm(a.contiguous(), b.contiguous())


@sgemm_op.register_fake
def _sgemm_fake(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    torch._check(a.dim() == 2 and b.dim() == 2 and a.shape[1] == b.shape[0],
                 lambda: "mt::sgemm needs (M, K) @ (K, N)")
    return a.new_empty((a.shape[0], b.shape[1]))


@torch.library.custom_op("mt::gemm_bias", mutates_args=())
def gemm_bias_op(a: torch.Tensor, b: torch.Tensor, bias: torch.Tensor) -> torch.Tensor:
    """a @ b + bias (bias: N values added to every row) through
    mt_sgemm_general_bias."""
    return gemm(a.contiguous(), b.contiguous(), bias=bias.contiguous())


@gemm_bias_op.register_fake
def _gemm_bias_fake(a: torch.Tensor, b: torch.Tensor, bias: torch.Tensor) -> torch.Tensor:
    torch._check(a.dim() == 2 and b.dim() == 2 and a.shape[1] == b.shape[0],
                 lambda: "mt::gemm_bias needs (M, K) @ (K, N)")
    torch._check(bias.dim() == 1 and bias.shape[0] == b.shape[1],
                 lambda: "mt::gemm_bias needs a bias of N values")
    return a.new_empty((a.shape[0], b.shape[1]))


@torch.library.custom_op("mt::linear", mutates_args=())
def linear_op(a: torch.Tensor, b: torch.Tensor, bias: Optional[torch.Tensor],
              residual: Optional[torch.Tensor], activation: str,
              trans_b: bool) -> Tuple[torch.Tensor, torch.Tensor]:
    """(act(a @ op(b) + bias) + residual, pre-activation) through mt_linear;
    the pre-activation is empty for activation "none" (its gradient needs
    none)."""
    if activation == "none":
        y = linear(a, b, bias=bias, residual=residual, trans_b=trans_b)
        return y, y.new_empty((0,))
    return linear(a, b, bias=bias, residual=residual, activation=activation, trans_b=trans_b,
                  preact=True)


@linear_op.register_fake
def _linear_fake(a, b, bias, residual, activation, trans_b):
    n, k = (b.shape[0], b.shape[1]) if trans_b else (b.shape[1], b.shape[0])
    torch._check(a.dim() == 2 and b.dim() == 2 and a.shape[1] == k,
                 lambda: "mt::linear needs (M, K) and a weight of K x N (N x K with trans_b)")
    y = a.new_empty((a.shape[0], n))
    return y, a.new_empty((0,)) if activation == "none" else torch.empty_like(y)


def _linear_setup(ctx, inputs, output):
    a, b, bias, residual, activation, trans_b = inputs
    ctx.save_for_backward(a, b, output[1])
    ctx.options = activation, trans_b
    ctx.set_materialize_grads(False)
    ctx.mark_non_differentiable(output[1])


@once_differentiable
def _linear_grad(ctx, dy, _):
    if dy is None:
        return (None,) * 6
    a, b, z = ctx.saved_tensors
    activation, trans_b = ctx.options
    need_a, need_b, need_bias, need_residual = ctx.needs_input_grad[:4]
    da, db, dbias = linear_backward(dy.contiguous(), a, b,
                                    z=None if activation == "none" else z,
                                    activation=activation, trans_b=trans_b, need_a=need_a,
                                    need_b=need_b, need_bias=need_bias)
    return da, db, dbias, dy if need_residual else None, None, None


linear_op.register_autograd(_linear_grad, setup_context=_linear_setup)


@torch.library.custom_op("mt::rms_norm", mutates_args=())
def rms_norm_op(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor],
                eps: float) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, h, rstd) of the root-mean-square norm of h = x + residual through
    mt_rms_norm; without a residual h is empty (it is x)."""
    y, h, rstd = rms_norm(x, weight, residual=residual, eps=eps)
    return y, x.new_empty((0,)) if residual is None else h, rstd


@rms_norm_op.register_fake
def _rms_norm_fake(x, weight, residual, eps):
    torch._check(x.dim() == 2 and weight.dim() == 1 and weight.shape[0] == x.shape[1],
                 lambda: "mt::rms_norm needs rows x d and a weight of d values")
    h = x.new_empty((0,)) if residual is None else x.new_empty(tuple(x.shape))
    return x.new_empty(tuple(x.shape)), h, x.new_empty((x.shape[0],), dtype=torch.float32)


def _rms_norm_setup(ctx, inputs, output):
    x, weight, residual, _ = inputs
    _, h, rstd = output
    ctx.save_for_backward(x if residual is None else h, weight, rstd)
    ctx.has_residual = residual is not None
    ctx.set_materialize_grads(False)
    ctx.mark_non_differentiable(rstd)


def _both(dy, dh, h):
    """The gradients of a norm's y and h as its gradient takes them: h's is None
    where nothing reads it, y's is needed."""
    dy = torch.zeros_like(h, memory_format=torch.contiguous_format) if dy is None \
        else dy.contiguous()
    return dy, None if dh is None else dh.contiguous()


@once_differentiable
def _rms_norm_grad(ctx, dy, dh, _):
    h, weight, rstd = ctx.saved_tensors
    dy, dh = _both(dy, dh if ctx.has_residual else None, h)
    dx, dweight = rms_norm_backward(dy, h, weight, rstd, dh=dh,
                                    need_weight=ctx.needs_input_grad[1])
    if dweight is not None:
        dweight = dweight.to(weight.dtype)
    return dx, dweight, dx if ctx.has_residual else None, None


rms_norm_op.register_autograd(_rms_norm_grad, setup_context=_rms_norm_setup)


@torch.library.custom_op("mt::layer_norm", mutates_args=())
def layer_norm_op(x: torch.Tensor, weight: Optional[torch.Tensor],
                  bias: Optional[torch.Tensor], residual: Optional[torch.Tensor], eps: float,
                  dropout: float, seed: Optional[torch.Tensor], sequence: int
                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, h, mean, rstd) of the layer norm of h = drop(x) + residual through
    mt_layer_norm (no weight: ones, no bias: zeros); where nothing is dropped or
    added h is empty (it is x)."""
    y, h, mean, rstd = layer_norm(x, weight, bias, residual=residual, eps=eps, dropout=dropout,
                                  seed=seed, sequence=sequence)
    return y, x.new_empty((0,)) if h is x else h, mean, rstd


@layer_norm_op.register_fake
def _layer_norm_fake(x, weight, bias, residual, eps, dropout, seed, sequence):
    torch._check(x.dim() == 2 and all(v is None or v.dim() == 1 and v.shape[0] == x.shape[1]
                                      for v in (weight, bias)),
                 lambda: "mt::layer_norm needs rows x d, a weight and a bias of d values or none")
    joined = residual is not None or dropout > 0.0
    stats = [x.new_empty((x.shape[0],), dtype=torch.float32) for _ in range(2)]
    return (x.new_empty(tuple(x.shape)),
            x.new_empty(tuple(x.shape)) if joined else x.new_empty((0,)), *stats)


def _layer_norm_setup(ctx, inputs, output):
    x, weight, bias, residual, _, p, seed, sequence = inputs
    _, h, mean, rstd = output
    ctx.joined = residual is not None or p > 0.0
    ctx.save_for_backward(h if ctx.joined else x, weight, mean, rstd, seed if p > 0.0 else None)
    ctx.options = p, sequence
    ctx.vector_dtype = next((v.dtype for v in (weight, bias) if v is not None), None)
    ctx.has_residual = residual is not None
    ctx.set_materialize_grads(False)
    ctx.mark_non_differentiable(mean, rstd)


@once_differentiable
def _layer_norm_grad(ctx, dy, dh, *_):
    h, weight, mean, rstd, seed = ctx.saved_tensors
    p, sequence = ctx.options
    dy, dh = _both(dy, dh if ctx.joined else None, h)
    dx, dres, dweight, dbias = layer_norm_backward(
        dy, h, weight, mean, rstd, dh=dh, dropout=p, seed=seed, sequence=sequence,
        need_weight=ctx.needs_input_grad[1], need_bias=ctx.needs_input_grad[2])
    if dweight is not None:
        dweight = dweight.to(ctx.vector_dtype)
    if dbias is not None:
        dbias = dbias.to(ctx.vector_dtype)
    return dx, dweight, dbias, dres if ctx.has_residual else None, None, None, None, None


layer_norm_op.register_autograd(_layer_norm_grad, setup_context=_layer_norm_setup)


@torch.library.custom_op("mt::dropout", mutates_args=())
def dropout_op(x: torch.Tensor, p: float, seed: torch.Tensor, sequence: int,
               residual: Optional[torch.Tensor]) -> torch.Tensor:
    """drop(x) + residual through mt_dropout."""
    return dropout(x, p, seed, sequence=sequence, residual=residual)


@dropout_op.register_fake
def _dropout_fake(x, p, seed, sequence, residual):
    torch._check(x.dim() == 2, lambda: "mt::dropout needs rows x d")
    return x.new_empty(tuple(x.shape))


def _dropout_setup(ctx, inputs, output):
    _, p, seed, sequence, residual = inputs
    ctx.save_for_backward(seed)
    ctx.options = p, sequence
    ctx.has_residual = residual is not None
    ctx.set_materialize_grads(False)


@once_differentiable
def _dropout_grad(ctx, dy):
    if dy is None:
        return (None,) * 5
    seed, = ctx.saved_tensors
    p, sequence = ctx.options
    dx = dropout(dy.contiguous(), p, seed, sequence=sequence) if ctx.needs_input_grad[0] else None
    return dx, None, None, None, dy if ctx.has_residual else None


dropout_op.register_autograd(_dropout_grad, setup_context=_dropout_setup)


@torch.library.custom_op("mt::linear_cross_entropy", mutates_args=())
def linear_cross_entropy_op(a: torch.Tensor, b: torch.Tensor, target: torch.Tensor,
                            trans_b: bool, ignore_index: int, label_smoothing: float,
                            z_loss: float) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse) per token through mt_linear_cross_entropy; lse is not
    differentiable."""
    return linear_cross_entropy(a, b, target, trans_b=trans_b, ignore_index=ignore_index,
                                label_smoothing=label_smoothing, z_loss=z_loss)


@linear_cross_entropy_op.register_fake
def _linear_cross_entropy_fake(a, b, target, trans_b, ignore_index, label_smoothing, z_loss):
    k = b.shape[1] if trans_b else b.shape[0]
    torch._check(a.dim() == 2 and b.dim() == 2 and a.shape[1] == k
                 and target.shape == (a.shape[0],),
                 lambda: "mt::linear_cross_entropy needs (T, K), a weight of K x V (V x K with "
                         "trans_b) and T targets")
    return tuple(a.new_empty((a.shape[0],), dtype=torch.float32) for _ in range(2))


def _linear_cross_entropy_setup(ctx, inputs, output):
    a, b, target, trans_b, ignore_index, label_smoothing, z_loss = inputs
    ctx.save_for_backward(a, b, target, output[1])
    ctx.options = dict(trans_b=trans_b, ignore_index=ignore_index,
                       label_smoothing=label_smoothing, z_loss=z_loss)
    ctx.set_materialize_grads(False)
    ctx.mark_non_differentiable(output[1])


@once_differentiable
def _linear_cross_entropy_grad(ctx, dloss, _):
    if dloss is None:
        return (None,) * 7
    a, b, target, lse = ctx.saved_tensors
    da, db = linear_cross_entropy_backward(dloss.contiguous(), a, b, target, lse,
                                           need_a=ctx.needs_input_grad[0],
                                           need_b=ctx.needs_input_grad[1], **ctx.options)
    return da, db, None, None, None, None, None


linear_cross_entropy_op.register_autograd(_linear_cross_entropy_grad,
                                          setup_context=_linear_cross_entropy_setup)
