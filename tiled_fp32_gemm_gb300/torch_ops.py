"""Torch operator registrations for the library's products and the
feed-forward operators.

Importing this module registers ``torch.ops.mt.sgemm(a, b)``,
``torch.ops.mt.gemm_bias(a, b, bias)``, ``torch.ops.mt.linear`` and
``torch.ops.mt.rms_norm`` as torch custom operators: the same C-ABI calls as
``sgemm``, ``gemm(..., bias=...)``, ``linear`` and ``rms_norm``, visible to
torch's dispatcher, graph capture and tracing (each has a shape-only fake
implementation, so tracing needs no GPU).  ``linear`` and ``rms_norm`` are
differentiable, once: their gradients are ``linear_backward`` and
``rms_norm_backward``, which have none themselves, so a second derivative
raises.  Marshalling only: the work runs in the library's
kernels.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import gemm, linear, linear_backward, rms_norm, rms_norm_backward, sgemm


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
    ctx.mark_non_differentiable(output[1])


@once_differentiable
def _linear_grad(ctx, dy, _):
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
    ctx.mark_non_differentiable(rstd)


@once_differentiable
def _rms_norm_grad(ctx, dy, dh, _):
    h, weight, rstd = ctx.saved_tensors
    dx, dweight = rms_norm_backward(
        dy.contiguous(), h, weight, rstd, need_weight=ctx.needs_input_grad[1],
        dh=dh.contiguous() if ctx.has_residual and dh is not None else None)
    if dweight is not None:
        dweight = dweight.to(weight.dtype)
    return dx, dweight, dx if ctx.has_residual else None, None


rms_norm_op.register_autograd(_rms_norm_grad, setup_context=_rms_norm_setup)
