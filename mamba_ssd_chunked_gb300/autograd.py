"""The training operators as differentiable torch functions.

    from mamba_ssd_chunked_gb300.autograd import gated_scan, block_norm, linear_cross_entropy

Each runs its forward and its gradients in the library's kernels (ssd_gated_scan and
_bwd, ssd_block_norm and _bwd, ssd_linear_cross_entropy and _bwd), with their
arguments, layouts and errors. What a gradient needs is kept by torch's graph.
Gradients that reach an operator non-contiguous are copied once. The gradients
have no derivative of their own: differentiating them again raises.
"""
from __future__ import annotations

import functools

import torch

from . import (ssd_block_norm, ssd_block_norm_bwd, ssd_gated_scan, ssd_gated_scan_bwd, ssd_linear_cross_entropy,
               ssd_linear_cross_entropy_bwd)

__all__ = ["gated_scan", "block_norm", "linear_cross_entropy"]


def _dense(t, dtype):
    return None if t is None else t.to(dtype).contiguous()


class _Final(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad, name, *depends_on):
        ctx.name = name
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name}: its gradients cannot be differentiated again")


def _first_order(name):
    """Decorates a backward whose results depend on the operator's inputs in ways that torch does not see. Under
    create_graph they would count as constants; here whoever differentiates them gets an error."""
    def wrap(backward):
        @functools.wraps(backward)
        def run(ctx, *grads):
            with torch.no_grad():
                out = backward(ctx, *grads)
            if not torch.is_grad_enabled():
                return out
            on = [t for t in (*ctx.saved_tensors, *grads) if t is not None and t.requires_grad]
            return tuple(None if g is None else _Final.apply(g, name, *on) for g in out)
        return run
    return wrap


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, dt_bias, A, D, init_state, seq_idx):
        y, final, chunks = ssd_gated_scan(x, dt, dt_bias, A, D, init_state=init_state, seq_idx=seq_idx,
                                          return_chunk_states=True)
        ctx.save_for_backward(x, dt, dt_bias, A, D, seq_idx, chunks)
        ctx.with_init = init_state is not None
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @_first_order("gated_scan")
    def backward(ctx, dy, dfinal):
        x, dt, dt_bias, A, D, seq_idx, chunks = ctx.saved_tensors
        dy = torch.zeros_like(x, memory_format=torch.contiguous_format) if dy is None else _dense(dy, x.dtype)
        dx, ddt, dbias, dA, dD, dinit = ssd_gated_scan_bwd(dy, x, dt, dt_bias, A, chunks, D=D, seq_idx=seq_idx,
                                                          dfinal_state=_dense(dfinal, torch.float32))
        return dx, ddt, dbias, dA, dD, dinit if ctx.with_init else None, None


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, z, post_weight, scale, pre_weight, eps, residual_dtype):
        r, out, rstd = ssd_block_norm(y, residual=residual, z=z, post_weight=post_weight, scale=scale,
                                      pre_weight=pre_weight, eps=eps, residual_dtype=residual_dtype, return_rstd=True)
        ctx.save_for_backward(y, residual, z, post_weight, scale, pre_weight, rstd)
        ctx.residual_dtype = r.dtype
        ctx.set_materialize_grads(False)
        return r, out

    @staticmethod
    @_first_order("block_norm")
    def backward(ctx, dr, dout):
        y, residual, z, post_weight, scale, pre_weight, rstd = ctx.saved_tensors
        if pre_weight is not None and dout is None:
            dout = torch.zeros(y.shape, dtype=y.dtype, device=y.device)
        if dr is None and dout is None:
            return (None,) * 8
        dy, dres, dz, dpost, dscale, dpre = ssd_block_norm_bwd(
            _dense(dout, y.dtype), _dense(dr, ctx.residual_dtype), y, rstd, residual=residual, z=z,
            post_weight=post_weight, scale=scale, pre_weight=pre_weight, residual_dtype=ctx.residual_dtype)
        return dy, dres, dz, dpost, dscale, dpre, None, None


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, target, ignore_index):
        loss, lse = ssd_linear_cross_entropy(hidden, weight, target, ignore_index=ignore_index)
        ctx.save_for_backward(hidden, weight, target, lse)
        ctx.ignore_index = ignore_index
        ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    @_first_order("linear_cross_entropy")
    def backward(ctx, dloss, _):
        hidden, weight, target, lse = ctx.saved_tensors
        dh, dw = ssd_linear_cross_entropy_bwd(_dense(dloss, torch.float32), hidden, weight, target, lse,
                                              ignore_index=ctx.ignore_index)
        return dh, dw, None, None


def gated_scan(x, dt, dt_bias, A, D=None, init_state=None, seq_idx=None):
    """ssd_gated_scan; differentiable in everything but seq_idx. Returns y, final_state."""
    return _GatedScan.apply(x, dt, dt_bias, A, D, init_state, seq_idx)


def block_norm(y, residual=None, z=None, post_weight=None, scale=None, pre_weight=None, eps: float = 1e-5,
               residual_dtype=None):
    """ssd_block_norm; differentiable in all its tensors. Returns residual_out, out (None without pre_weight)."""
    return _BlockNorm.apply(y, residual, z, post_weight, scale, pre_weight, eps, residual_dtype)


def linear_cross_entropy(hidden, weight, target, ignore_index: int = -100):
    """ssd_linear_cross_entropy; differentiable in hidden and weight. Returns loss, lse (no gradient through lse)."""
    return _LinearCrossEntropy.apply(hidden, weight, target, ignore_index)
