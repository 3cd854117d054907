"""Torch-tensor front end of the root-mean-square norm (include/ag_layer.h), with the
residual's addition, its gradient, and outputs as the 8- or 4-bit rows of a product.  No
arithmetic here: tensors are checked and passed to libaggemm.so by the native module
``_front`` (csrc/front.cpp).

A layer's way in::

    r = rms_norm(branch, weight, residual=stream)         # r.h is the new residual stream
    dx, dweight = rms_norm_backward(dy, r.h, weight, r.rstd, dh=dstream)

    xq, xs, stream = rms_norm_quantized(branch, weight, "e4m3", residual=stream)
    y = fp8.Fp8Linear(H, N).forward(xq, xs, wq, ws)       # "mxfp4": fp4.Fp4Linear

As in moe.py the functions know nothing of autograd, the tensors of a call and its stream are
on one device, and ``stream`` is a torch stream, None for the current one.  x, the residual
and the gradients may be column blocks of wider matrices.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B_
from . import _front
from .moe import _on

CODES = {"e4m3": B_.E4M3, "mxfp4": B_.E2M1}


class Norm(NamedTuple):
    """What :func:`rms_norm` makes of (rows, H)."""
    y: torch.Tensor     # (rows, H), x's type
    h: torch.Tensor     # (rows, H): x + residual, x's type; x itself without a residual
    rstd: torch.Tensor  # (rows,) float32


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, stream=None) -> Norm:
    """``h = x + residual`` rounded to x's type, ``rstd = 1 / sqrt(mean(h^2) + eps)`` and
    ``y = h * rstd * weight``, in 32 bits, y rounded once.  x is (rows, H) float16, bfloat16
    or float32, weight (H,) of x's type or float32."""
    if stream is not None:
        return _on(stream, rms_norm, x, weight, eps, residual)
    return tuple.__new__(Norm, _front.rms_norm(x, weight, eps, residual))


def rms_norm_quantized(x: torch.Tensor, weight: torch.Tensor, codes: str, eps: float = 1e-6,
                       residual: Optional[torch.Tensor] = None, stream=None):
    """(codes, scales, h): :func:`rms_norm` with y as the rows of a product, what
    ``fp8.quantize_rows`` ("e4m3", H a multiple of 16) or ``fp4.quantize_rows`` ("mxfp4", of
    32) would make of the unrounded y.  x, the residual and the weight are 16-byte aligned, rows
    a multiple of 16 bytes apart; others are refused (:func:`rms_norm` takes any)."""
    if stream is not None:
        return _on(stream, rms_norm_quantized, x, weight, codes, eps, residual)
    if codes not in CODES:
        raise ValueError("codes must be 'e4m3' or 'mxfp4'")
    return _front.rms_norm_quantized(x, weight, eps, residual, CODES[codes])


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      dh: Optional[torch.Tensor] = None, stream=None):
    """(dx, dweight) of :func:`rms_norm` from dy, the gradient of y, and dh, that of h from
    elsewhere: dx, in dy's type, is the gradient of x and of the residual alike; dweight (H,)
    is float32, summed over the rows in a fixed order."""
    if stream is not None:
        return _on(stream, rms_norm_backward, dy, h, weight, rstd, dh)
    return _front.rms_norm_backward(dy, h, weight, rstd, dh)
