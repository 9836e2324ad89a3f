"""The training operators around the optimizer: 8-bit activation checkpoints,
GELU, layer norm and the cross entropy of a linear layer over a large
vocabulary, forward and backward, as functions of CUDA tensors.

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
           "linear_cross_entropy_backward", "ACT_GROUP"]

ACT_GROUP = _lib.ACT_GROUP
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
BINDING_PATH = os.path.join(_lib.HERE, "_build", "fp8opt_binding.so")
# The C entry points the binding calls, in its order.
_ENTRIES = ("fp8_act_save", "fp8_act_load", "fp8_gelu", "fp8_gelu_backward",
            "fp8_layer_norm", "fp8_layer_norm_backward", "fp8_linear_xent",
            "fp8_linear_xent_backward", "fp8opt_last_error")


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
