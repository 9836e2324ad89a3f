"""The training operators around the optimizer: 8-bit activation checkpoints,
GELU, layer norm and the cross entropy of a linear layer over a large
vocabulary, forward and backward, as functions of CUDA tensors.

Like the rest of the package this is argument checking and marshalling: every
step runs in the library's kernels (include/fp8opt.h describes the arithmetic).
Tensors must be contiguous and on one device; outputs are allocated on
``stream`` (the current stream unless given), where the work runs too, and the
caller orders other streams' use of the inputs and outputs against it, as for
any CUDA work.  No function waits for the GPU.

``bit_optimizer_gb300.nn`` wraps these functions for autograd.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import BF16, F16, F32, check, load

__all__ = ["act_save", "act_load", "gelu", "gelu_backward", "layer_norm",
           "layer_norm_backward", "linear_cross_entropy",
           "linear_cross_entropy_backward", "ACT_GROUP"]

_L = load()
ACT_GROUP = _lib.ACT_GROUP
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_FORMS = {"none": _lib.GELU_ERF, "tanh": _lib.GELU_TANH}


def _dtype(t: torch.Tensor, name: str) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}") from None


def _check(t, name: str, dev: int, dtype=None, shape=None) -> int:
    """The address of a contiguous CUDA tensor on device ``dev`` (any device
    when dev < 0) with the given dtype and shape, where given."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dev >= 0 and t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _run(call, dev: int, stream, *args):
    """call(stream handle, *args) with the tensors' device, and the stream
    given for them, current (the usual case, the current stream of the current
    device, needs no context)."""
    if stream is None and dev == _current_device():
        return call(_raw_stream(dev), *args)
    if stream is not None and stream.device_index != dev:
        raise ValueError("stream is on another device than the tensors")
    with torch.cuda.device(dev) if stream is None else torch.cuda.stream(stream):
        return call(_raw_stream(dev), *args)


def _form(approximate: str) -> int:
    try:
        return _FORMS[approximate]
    except (KeyError, TypeError):
        raise ValueError(f"approximate must be 'none' or 'tanh', not {approximate!r}") from None


def _groups(numel: int) -> int:
    return -(-numel // ACT_GROUP)


# ------------------------------------------------- activation checkpoints

def _new_checkpoint(x):
    return (torch.empty_like(x, dtype=torch.uint8),
            torch.empty(_groups(x.numel()), dtype=torch.float32, device=x.device))


def _checkpoint(codes, scales, dev: int, shape=None):
    pc = _check(codes, "codes", dev, torch.uint8, shape)
    return pc, _check(scales, "scales", codes.get_device(), torch.float32,
                      (_groups(codes.numel()),))


def act_save(x: torch.Tensor, stream=None):
    """The 8-bit checkpoint of x: (codes, scales), E4M3 codes in x's shape
    (uint8) and one float32 scale per ACT_GROUP consecutive elements."""
    px, dt = _check(x, "x", -1), _dtype(x, "x")

    def call(s):
        codes, scales = _new_checkpoint(x)
        check(_L.fp8_act_save(px, x.numel(), dt, codes.data_ptr(), scales.data_ptr(), s))
        return codes, scales
    return _run(call, x.get_device(), stream)


def act_load(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.float16,
             stream=None) -> torch.Tensor:
    """The activation of an ``act_save`` checkpoint, in ``dtype``."""
    pc, ps = _checkpoint(codes, scales, -1)
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")

    def call(s):
        x = torch.empty_like(codes, dtype=dtype)
        check(_L.fp8_act_load(pc, ps, codes.numel(), _DT[dtype], x.data_ptr(), s))
        return x
    return _run(call, codes.get_device(), stream)


def gelu(x: torch.Tensor, approximate: str = "none", stream=None):
    """(y, codes, scales): y = gelu(x) and the 8-bit checkpoint of x, in one
    pass.  approximate: "none" (x Phi(x)) or "tanh", as torch's."""
    px, dt, form = _check(x, "x", -1), _dtype(x, "x"), _form(approximate)

    def call(s):
        y = torch.empty_like(x)
        codes, scales = _new_checkpoint(x)
        check(_L.fp8_gelu(px, x.numel(), dt, form, y.data_ptr(), codes.data_ptr(),
                          scales.data_ptr(), s))
        return y, codes, scales
    return _run(call, x.get_device(), stream)


def gelu_backward(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                  approximate: str = "none", stream=None) -> torch.Tensor:
    """dx = dy * gelu'(x), with x read from its 8-bit checkpoint."""
    pd, dt, dev, form = _check(dy, "dy", -1), _dtype(dy, "dy"), dy.get_device(), _form(approximate)
    pc, ps = _checkpoint(codes, scales, dev, dy.shape)

    def call(s):
        dx = torch.empty_like(dy)
        check(_L.fp8_gelu_backward(pd, pc, ps, dy.numel(), dt, form, dx.data_ptr(), s))
        return dx
    return _run(call, dev, stream)


# -------------------------------------------------------------- layer norm

def _rows_cols(t: torch.Tensor, name: str):
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} needs a last dimension of at least 1")
    cols = t.shape[-1]
    return t.numel() // cols, cols


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
    px, dt, dev = _check(x, "x", -1), _dtype(x, "x"), x.get_device()
    rows, cols = _rows_cols(x, "x")
    pw, wdt = _check(weight, "weight", dev, None, (cols,)), _dtype(weight, "weight")
    pb = None if bias is None else _check(bias, "bias", dev, weight.dtype, (cols,))

    def call(s):
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        if save == "x":
            mean = torch.empty_like(rstd)
            check(_L.fp8_layer_norm(px, pw, pb, rows, cols, dt, wdt, eps, y.data_ptr(),
                                    mean.data_ptr(), rstd.data_ptr(), None, None, s))
            return y, mean, rstd
        codes = torch.empty_like(x, dtype=torch.uint8)
        scales = torch.empty_like(rstd)
        check(_L.fp8_layer_norm(px, pw, pb, rows, cols, dt, wdt, eps, y.data_ptr(), None,
                                rstd.data_ptr(), codes.data_ptr(), scales.data_ptr(), s))
        return y, codes, scales, rstd
    return _run(call, dev, stream)


def layer_norm_backward(dy: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                        x=None, mean=None, codes=None, scales=None,
                        need_bias: bool = True, stream=None):
    """(dx, dweight, dbias) of ``layer_norm``, from x and mean (save="x") or
    from codes and scales (save="fp8"); dbias is None without need_bias."""
    pd, dt, dev = _check(dy, "dy", -1), _dtype(dy, "dy"), dy.get_device()
    rows, cols = _rows_cols(dy, "dy")
    lead = dy.shape[:-1]
    pw, wdt = _check(weight, "weight", dev, None, (cols,)), _dtype(weight, "weight")
    pr = _check(rstd, "rstd", dev, torch.float32, lead)
    px = pm = pc = ps = None
    if codes is not None and scales is not None and x is None and mean is None:
        pc = _check(codes, "codes", dev, torch.uint8, dy.shape)
        ps = _check(scales, "scales", dev, torch.float32, lead)
    elif x is not None and mean is not None and codes is None and scales is None:
        px = _check(x, "x", dev, dy.dtype, dy.shape)
        pm = _check(mean, "mean", dev, torch.float32, lead)
    else:
        raise ValueError("give x and mean, or codes and scales")

    def call(s):
        dx = torch.empty_like(dy)
        dw = torch.empty_like(weight)
        db = torch.empty_like(weight) if need_bias else None
        check(_L.fp8_layer_norm_backward(
            pd, px, pm, pc, ps, pr, pw, rows, cols, dt, wdt, dx.data_ptr(), dw.data_ptr(),
            db.data_ptr() if need_bias else None, s))
        return dx, dw, db
    return _run(call, dev, stream)


# ----------------------------------------------- vocabulary cross entropy

def _linear(x, w, target):
    """Addresses and sizes of a linear layer's input, weight and targets."""
    px, dt, dev = _check(x, "x", -1), _dtype(x, "x"), x.get_device()
    if dt == F32:
        raise TypeError("x must be bfloat16 or float16")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError("x must have shape (tokens, dim)")
    pw = _check(w, "w", dev, x.dtype)
    if w.dim() != 2 or w.shape[0] < 1 or w.shape[1] != x.shape[1]:
        raise ValueError(f"w must have shape (vocabulary, {x.shape[1]}), not {tuple(w.shape)}")
    pt = _check(target, "target", dev, torch.int64, x.shape[:1])
    return px, pw, pt, x.shape[0], x.shape[1], w.shape[0], dt, dev


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                         ignore_index: int = -100, stream=None):
    """(loss, lse), both float32, one per token: lse = log sum exp of the
    token's logits x w^T, loss = lse - logit of its target (0 for a target of
    ignore_index, NaN for another one outside the vocabulary).  x: (tokens,
    dim), w: (vocabulary, dim), bfloat16 or float16; target: int64.  The
    logits are never in memory as a whole."""
    px, pw, pt, rows, dim, vocab, dt, dev = _linear(x, w, target)

    def call(s):
        loss = torch.empty(rows, dtype=torch.float32, device=x.device)
        lse = torch.empty_like(loss)
        check(_L.fp8_linear_xent(px, pw, pt, rows, dim, vocab, dt, ignore_index,
                                 loss.data_ptr(), lse.data_ptr(), s))
        return loss, lse
    return _run(call, dev, stream)


def linear_cross_entropy_backward(dloss: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                                  target: torch.Tensor, lse: torch.Tensor,
                                  ignore_index: int = -100, stream=None):
    """(dx, dw), in x's type, for the gradient dloss (float32, one per token)
    of ``linear_cross_entropy``'s loss; lse is that call's."""
    px, pw, pt, rows, dim, vocab, dt, dev = _linear(x, w, target)
    pd = _check(dloss, "dloss", dev, torch.float32, (rows,))
    pl = _check(lse, "lse", dev, torch.float32, (rows,))

    def call(s):
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        check(_L.fp8_linear_xent_backward(pd, px, pw, pt, pl, rows, dim, vocab, dt,
                                          ignore_index, dx.data_ptr(), dw.data_ptr(), s))
        return dx, dw
    return _run(call, dev, stream)
