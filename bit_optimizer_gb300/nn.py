"""The training operators for autograd: each function keeps for its backward
pass what the operator's 8-bit form keeps, and nothing else.

* ``layer_norm``: the normalised input in E4M3 (save="fp8"), or the input.
* ``gelu``: the input in E4M3.
* ``linear``: the product is torch's; its input, which the weight's gradient
  needs, is kept in E4M3.
* ``linear_cross_entropy``: the input, the weight and one float per token; no
  logits (the backward pass makes the probabilities again, two pieces of the
  vocabulary at a time).
* ``linear_distillation``: the same, and the teacher's ids and logits.
* ``embedding``: the ids.
* ``policy_loss``: its inputs, and one float per sequence.

A GPT block's feed-forward half and its loss are then, with x the residual
stream in FP16 or BF16:

    h = nn.layer_norm(x, ln_w, ln_b)
    x = x + nn.linear(nn.gelu(nn.linear(h, fc_w, fc_b)), proj_w, proj_b)
    loss = nn.linear_cross_entropy(nn.layer_norm(x, lnf_w, lnf_b), wte, target)

and x starts as nn.embedding(tokens, wte).  The policy loss takes the log
probabilities that the cross entropy gives:

    logp = -nn.linear_cross_entropy(x, wte, answer, reduction="none")
    loss, stats = nn.policy_loss(logp, old_logp, advantage, mask, ref_logp, kl_coef=0.04)

Under torch.autocast the linear layers cast their input and parameters to
its dtype, as torch's do, so FP32 weights get FP32 gradients; ``layer_norm`` and
``gelu`` take what they are given, and their result has its type.  Under no_grad
the checkpoints are written all the same, and freed.

A step with its backward pass can be captured into a CUDA graph once it has run on
the stream, as long as no eager graph of the same leaves lives: torch's engine would
order the capturing stream against the one that graph used, and the capture fails.
"""
from __future__ import annotations

import torch
from torch.autograd import Function
from torch.autograd.function import once_differentiable

from . import ops

__all__ = ["layer_norm", "gelu", "linear", "linear_cross_entropy",
           "linear_distillation", "embedding", "policy_loss"]


class _LayerNorm(Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, save):
        ctx.save, ctx.has_bias = save, bias is not None
        if save == "fp8":
            y, codes, scales, rstd = ops.layer_norm(x, weight, bias, eps, "fp8")
            ctx.save_for_backward(weight, rstd, codes, scales)
        else:
            y, mean, rstd = ops.layer_norm(x, weight, bias, eps, save)
            ctx.save_for_backward(weight, rstd, x, mean)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, rstd, a, b = ctx.saved_tensors
        saved = dict(codes=a, scales=b) if ctx.save == "fp8" else dict(x=a, mean=b)
        dx, dw, db = ops.layer_norm_backward(dy.contiguous(), weight, rstd,
                                             need_bias=ctx.has_bias, **saved)
        return dx, dw, db, None, None


class _Gelu(Function):
    @staticmethod
    def forward(ctx, x, approximate):
        y, codes, scales = ops.gelu(x, approximate)
        ctx.save_for_backward(codes, scales)
        ctx.approximate = approximate
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return ops.gelu_backward(dy.contiguous(), *ctx.saved_tensors, ctx.approximate), None


class _Linear(Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(weight, *ops.act_save(x))
        ctx.has_bias = bias is not None
        return torch.nn.functional.linear(x, weight, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, codes, scales = ctx.saved_tensors
        dy = dy.reshape(-1, weight.shape[0])
        dx = dw = db = None
        if ctx.needs_input_grad[0]:
            dx = (dy @ weight).view(codes.shape)
        if ctx.needs_input_grad[1]:
            x = ops.act_load(codes, scales, weight.dtype)
            dw = dy.T @ x.view(-1, weight.shape[1])
        if ctx.has_bias and ctx.needs_input_grad[2]:
            db = dy.sum(0)
        return dx, dw, db


class _LinearCrossEntropy(Function):
    @staticmethod
    def forward(ctx, x, weight, target, ignore_index):
        loss, lse = ops.linear_cross_entropy(x, weight, target, ignore_index)
        ctx.save_for_backward(x, weight, target, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x, weight, target, lse = ctx.saved_tensors
        dx, dw = ops.linear_cross_entropy_backward(dloss.contiguous(), x, weight, target, lse,
                                                   ctx.ignore_index)
        return dx, dw, None, None


class _LinearDistillation(Function):
    @staticmethod
    def forward(ctx, x, weight, ids, logits, temperature):
        loss, lse = ops.linear_distillation(x, weight, ids, logits, temperature)
        ctx.save_for_backward(x, weight, ids, logits, lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        dx, dw = ops.linear_distillation_backward(dloss.contiguous(), *ctx.saved_tensors,
                                                  ctx.temperature)
        return dx, dw, None, None, None


class _Embedding(Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, padding_idx):
        ctx.save_for_backward(ids)
        ctx.args = weight.shape[0], scale, padding_idx
        return ops.embedding(ids, weight, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return None, ops.embedding_backward(dy.contiguous(), *ctx.saved_tensors, *ctx.args), None, None


class _PolicyLoss(Function):
    @staticmethod
    def forward(ctx, logp, old_logp, advantage, mask, ref_logp, low, high, kl_coef, reduction):
        stats, weight = ops.policy_loss(logp, old_logp, advantage, mask, ref_logp, low, high,
                                        kl_coef, reduction)
        ctx.save_for_backward(logp, old_logp, advantage, weight, mask, ref_logp)
        ctx.args = low, high, kl_coef
        ctx.mark_non_differentiable(stats)
        return stats[0].clone(), stats

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        return (ops.policy_loss_backward(dloss, *ctx.saved_tensors, *ctx.args), *[None] * 8)


def layer_norm(x, weight, bias=None, eps: float = 1e-5, save: str = "fp8"):
    """Layer norm over the last dimension (``ops.layer_norm``)."""
    return _LayerNorm.apply(x.contiguous(), weight, bias, eps, save)


def gelu(x, approximate: str = "tanh"):
    """GELU (``ops.gelu``)."""
    return _Gelu.apply(x.contiguous(), approximate)


def _autocast(*tensors):
    """The tensors in autocast's dtype where it is on (float64 stays, as there)."""
    if not torch.is_autocast_enabled("cuda"):
        return tensors
    dtype = torch.get_autocast_dtype("cuda")
    return tuple(t if t is None or not t.is_floating_point() or t.dtype == torch.float64
                 else t.to(dtype) for t in tensors)


def linear(x, weight, bias=None):
    """x weight^T + bias."""
    x, weight, bias = _autocast(x, weight, bias)
    return _Linear.apply(x.contiguous(), weight, bias)


def linear_cross_entropy(x, weight, target, ignore_index: int = -100,
                         reduction: str = "mean"):
    """Cross entropy of x weight^T against target (``ops.linear_cross_entropy``).
    x: (..., dim), target: (...).  reduction: "none" (one loss per token, 0
    where ignored), "sum", or "mean" over the tokens that are not ignored (0
    when all are)."""
    if reduction not in ("none", "sum", "mean"):
        raise ValueError(f"reduction must be 'none', 'sum' or 'mean', not {reduction!r}")
    x, weight = _autocast(x, weight)
    loss = _LinearCrossEntropy.apply(x.contiguous().view(-1, x.shape[-1]), weight,
                                     target.contiguous().view(-1), ignore_index)
    if reduction == "none":
        return loss.view(target.shape)
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (target != ignore_index).sum().clamp(min=1)


def linear_distillation(x, weight, ids, logits, temperature: float = 1.0,
                        reduction: str = "mean"):
    """Divergence of x weight^T from a teacher's top logits (``ops.linear_distillation``).
    x: (..., dim), ids and logits: (..., k) with x's leading dimensions; no gradient
    for the logits.  reduction: "none" (one loss per token), "sum", or "mean" over the
    tokens that have an id (0 when none has).  Soft targets' usual factor temperature ** 2 is the caller's."""
    if reduction not in ("none", "sum", "mean"):
        raise ValueError(f"reduction must be 'none', 'sum' or 'mean', not {reduction!r}")
    if (x.dim() < 1 or ids.dim() != x.dim() or ids.shape[:-1] != x.shape[:-1]
            or logits.shape != ids.shape or ids.shape[-1] < 1):
        raise ValueError("ids and logits must have one shape, of x's leading dimensions and at "
                         f"least one entry, not {tuple(ids.shape)} and {tuple(logits.shape)} "
                         f"for x of {tuple(x.shape)}")
    x, weight = _autocast(x, weight)
    k = ids.shape[-1]
    loss = _LinearDistillation.apply(x.contiguous().view(-1, x.shape[-1]), weight,
                                     ids.contiguous().view(-1, k), logits.contiguous().view(-1, k),
                                     temperature)
    if reduction == "none":
        return loss.view(ids.shape[:-1])
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (ids >= 0).any(-1).sum().clamp(min=1)


def embedding(ids, weight, scale: float = 1.0, padding_idx=None):
    """scale * weight[ids] (``ops.embedding``); the word padding_idx gets no gradient."""
    if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
        raise ValueError(f"padding_idx must be in [0, {weight.shape[0]}), not {padding_idx}")
    return _Embedding.apply(ids.contiguous(), weight, scale, padding_idx)


def policy_loss(logp, old_logp, advantage, mask=None, ref_logp=None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, reduction: str = "token"):
    """(loss, stats) of ``ops.policy_loss``: the mean loss, for whose gradient logp is
    the only input, and what it consists of, without a gradient."""
    mask, ref_logp = (t if t is None else t.contiguous() for t in (mask, ref_logp))
    return _PolicyLoss.apply(logp.contiguous(), old_logp.contiguous(), advantage.contiguous(),
                             mask, ref_logp, clip_low, clip_high, kl_coef, reduction)
