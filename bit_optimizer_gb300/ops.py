"""The training operators around the optimizer: 8-bit activation checkpoints,
GELU, layer norm, the cross entropy of a linear layer over a large vocabulary and
its distillation from a teacher, the embedding and the clipped policy loss, forward
and backward, as functions of CUDA tensors.

Like the rest of the package this is argument checking and marshalling: every
step runs in the library's kernels (include/fp8opt.h describes the arithmetic).
The checks, the outputs' allocation and the call are made natively
(csrc/binding.cpp): a training step calls these functions often, and on small
tensors the same steps in Python take longer than the kernels.

Tensors must be contiguous and on one device: another kind of object, device or
dtype raises TypeError, a wrong shape, layout or option ValueError, and what the
library itself refuses Fp8OptError.  Outputs are allocated on ``stream`` (the
current stream unless given), where the work runs too, and the caller orders
other streams' use of the inputs and outputs against it, as for any CUDA work.
No function waits for the GPU, but when the scratch of the backward passes and
the cross entropy has to grow: the stream keeps its scratch (a quarter more than
the largest call's, where there is room), outside torch's memory, until
``release_stream`` or ``release``.

These functions are not seen by autograd: their results require no gradient,
whatever the arguments do.  ``bit_optimizer_gb300.nn`` wraps them for it.
"""
from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import _lib
from ._lib import BF16, F16, F32

__all__ = ["act_save", "act_load", "gelu", "gelu_backward", "layer_norm",
           "layer_norm_backward", "linear_cross_entropy",
           "linear_cross_entropy_backward", "embedding", "embedding_backward",
           "policy_loss", "policy_loss_backward", "linear_distillation",
           "linear_distillation_backward", "ACT_GROUP"]

ACT_GROUP = _lib.ACT_GROUP
_REDUCTIONS = {"token": _lib.MEAN_TOKEN, "sequence": _lib.MEAN_SEQUENCE}
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
BINDING_PATH = os.path.join(_lib.HERE, "_build", "fp8opt_binding.so")
# The C entry points the binding calls, in its order.
_ENTRIES = ("fp8_act_save", "fp8_act_load", "fp8_gelu", "fp8_gelu_backward",
            "fp8_layer_norm", "fp8_layer_norm_backward", "fp8_linear_xent",
            "fp8_linear_xent_backward", "fp8_embedding", "fp8_embedding_backward",
            "fp8_policy_loss", "fp8_policy_loss_backward", "fp8_linear_distill",
            "fp8_linear_distill_backward", "fp8opt_last_error")


def _load_binding():
    if not os.path.exists(BINDING_PATH):
        raise ImportError(
            f"the PyTorch binding is not built ({BINDING_PATH} is missing); run "
            "`python bit_optimizer_gb300/build.py` or __graft_entry__.build()")
    loader = importlib.machinery.ExtensionFileLoader("fp8opt_binding", BINDING_PATH)
    module = importlib.util.module_from_spec(
        importlib.util.spec_from_loader("fp8opt_binding", loader))
    loader.exec_module(module)
    lib = _lib.load()
    module.bind(*(C.cast(getattr(lib, name), C.c_void_p).value for name in _ENTRIES),
                _lib.check)
    return module


class _Unloaded:
    """Stands for the binding until a function below is first called: the
    optimizer needs the C library alone, and is there without it."""
    _lock = threading.Lock()

    def __getattr__(self, name):
        global _b
        with self._lock:
            if _b is self:
                _b = _load_binding()
        return getattr(_b, name)


_b = _Unloaded()


# ------------------------------------------------- activation checkpoints

def act_save(x: torch.Tensor, stream=None):
    """The 8-bit checkpoint of x: (codes, scales), E4M3 codes in x's shape
    (uint8) and one float32 scale per ACT_GROUP consecutive elements."""
    return _b.act_save(x, stream)


def act_load(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.float16,
             stream=None) -> torch.Tensor:
    """The activation of an ``act_save`` checkpoint, in ``dtype``."""
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    return _b.act_load(codes, scales, _DT[dtype], stream)[0]


def gelu(x: torch.Tensor, approximate: str = "none", stream=None):
    """(y, codes, scales): y = gelu(x) and the 8-bit checkpoint of x, in one
    pass.  approximate: "none" (x Phi(x)) or "tanh", as torch's."""
    return _b.gelu(x, approximate, stream)


def gelu_backward(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                  approximate: str = "none", stream=None) -> torch.Tensor:
    """dx = dy * gelu'(x), with x read from its 8-bit checkpoint."""
    return _b.gelu_backward(dy, codes, scales, approximate, stream)[0]


# -------------------------------------------------------------- layer norm

def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias=None, eps: float = 1e-5,
               save: str = "x", stream=None):
    """Layer norm over the last dimension.

    save="x": returns (y, mean, rstd); the backward pass takes x again.
    save="fp8": returns (y, codes, scales, rstd): the normalised x in E4M3
    (uint8, x's shape) with one float32 scale per row, instead of x.
    mean, rstd and scales have x's shape without its last dimension.
    """
    if save not in ("x", "fp8"):
        raise ValueError(f"save must be 'x' or 'fp8', not {save!r}")
    return _b.layer_norm(x, weight, bias, eps, save == "fp8", stream)


def layer_norm_backward(dy: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                        x=None, mean=None, codes=None, scales=None,
                        need_bias: bool = True, stream=None):
    """(dx, dweight, dbias) of ``layer_norm``, from x and mean (save="x") or
    from codes and scales (save="fp8"); dbias is None without need_bias."""
    return _b.layer_norm_backward(dy, weight, rstd, x, mean, codes, scales, bool(need_bias),
                                  stream)


# ----------------------------------------------- vocabulary cross entropy

def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                         ignore_index: int = -100, stream=None):
    """(loss, lse), both float32, one per token: lse = log sum exp of the
    token's logits x w^T, loss = lse - logit of its target (0 for a target of
    ignore_index, NaN for another one outside the vocabulary).  x: (tokens,
    dim), w: (vocabulary, dim), bfloat16 or float16; target: int64.  The
    logits are never in memory."""
    return _b.linear_cross_entropy(x, w, target, ignore_index, stream)


def linear_cross_entropy_backward(dloss: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                                  target: torch.Tensor, lse: torch.Tensor,
                                  ignore_index: int = -100, stream=None):
    """(dx, dw), in x's type, for the gradient dloss (float32, one per token)
    of ``linear_cross_entropy``'s loss; lse is that call's.  In scratch: the
    probabilities of two pieces of the vocabulary, in 16 bits (128 to 256 MiB each;
    for few tokens that is all of them)."""
    return _b.linear_cross_entropy_backward(dloss, x, w, target, lse, ignore_index, stream)


def linear_distillation(x: torch.Tensor, w: torch.Tensor, ids: torch.Tensor,
                        logits: torch.Tensor, temperature: float = 1.0, stream=None):
    """(loss, lse), both float32, one per token: the divergence sum q (log q - log p)
    of p = softmax(x w^T / temperature) from q = softmax(logits / temperature), a
    teacher's top logits (tokens, up to 256) of the words ids (int64, the same shape;
    negative: not given), and lse = log sum exp(x w^T / temperature).  A token without
    entries has loss 0; an id outside the vocabulary gives NaN.  x: (tokens, dim), w:
    (vocabulary, dim), bfloat16 or float16; logits: these or float32.  The student's
    logits are never in memory."""
    return _b.linear_distillation(x, w, ids, logits, temperature, stream)


def linear_distillation_backward(dloss: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                                 ids: torch.Tensor, logits: torch.Tensor, lse: torch.Tensor,
                                 temperature: float = 1.0, stream=None):
    """(dx, dw), in x's type, for the gradient dloss (float32, one per token) of
    ``linear_distillation``'s loss; lse is that call's, and being float32 leaves the
    student's probabilities off by 2^-23 |lse| of themselves (low temperatures: lse is
    about the largest logit over it).  Scratch as ``linear_cross_entropy_backward``'s."""
    return _b.linear_distillation_backward(dloss, x, w, ids, logits, lse, temperature, stream)


# --------------------------------------------------------------- embedding

def embedding(ids: torch.Tensor, w: torch.Tensor, scale: float = 1.0,
              stream=None) -> torch.Tensor:
    """scale * w[ids], ids' shape and a last dimension of w's rows.  ids: int64, w:
    (vocabulary, dim).  An id outside the vocabulary gives a row of NaN."""
    return _b.embedding(ids, w, scale, stream)[0]


def embedding_backward(dy: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                       padding_idx=None, stream=None) -> torch.Tensor:
    """dw (vocab, dim) of ``embedding`` in dy's type: scale times the sum of the
    rows of dy that belong to each word, in their order; 0 for the word padding_idx
    and words without tokens.  Ids outside the vocabulary take no part."""
    return _b.embedding_backward(dy, ids, vocab, scale, padding_idx, stream)[0]


# ------------------------------------------------------------- policy loss

def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                mask=None, ref_logp=None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, reduction: str = "token", stream=None):
    """(stats, weight) of the clipped policy loss with a KL term on the tokens' log
    probabilities (float32, (batch, length)): with r = exp(logp - old_logp) and e =
    ref_logp - logp a token's loss is

        -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(e) - 1 - e).

    advantage A: (batch,) or (batch, length).  mask (bool): False where a token takes
    no part, whatever its values are.  stats (float32): the mean loss, the means of
    its first term and of exp(e) - 1 - e, and the part of the tokens that are
    clipped.  The mean is over all tokens (reduction="token"), or of each sequence's
    own mean, over the sequences that have tokens ("sequence"); weight (batch,) is
    what a token of each sequence weighs in it, which the backward pass takes."""
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be 'token' or 'sequence', not {reduction!r}")
    return _b.policy_loss(logp, old_logp, advantage, mask, ref_logp, clip_low, clip_high,
                          kl_coef, _REDUCTIONS[reduction], stream)


def policy_loss_backward(dloss: torch.Tensor, logp: torch.Tensor, old_logp: torch.Tensor,
                         advantage: torch.Tensor, weight: torch.Tensor, mask=None,
                         ref_logp=None, clip_low: float = 0.2, clip_high: float = 0.2,
                         kl_coef: float = 0.0, stream=None) -> torch.Tensor:
    """dlogp (float32) for the gradient dloss (one float32, on the device) of the mean
    loss of ``policy_loss``; weight is that call's."""
    return _b.policy_loss_backward(dloss, weight, logp, old_logp, advantage, mask, ref_logp,
                                   clip_low, clip_high, kl_coef, stream)[0]
