"""Torch-tensor front end of the gated activation (include/ag_layer.h): ``y = g * s * u`` with
``s = 1 / (1 + exp(-g))``, its gradient, and its output as the 8- or 4-bit rows of the next
product.  No arithmetic here: tensors are checked and passed to libaggemm.so by the native
module ``_front`` (csrc/front.cpp).

x is (rows, 2 N): the gate g in its first N columns, u in the others, as one product with
weights (K, 2 N) makes them.  As in moe.py the functions know nothing of autograd, the tensors
of a call and its stream are on one device, and ``stream`` is a torch stream, None for the
current one.  x and dy may be column blocks of wider matrices.
"""
from __future__ import annotations

import torch

from . import _front
from .moe import _on
from .norm import CODES


def swiglu(x: torch.Tensor, stream=None) -> torch.Tensor:
    """y (rows, N) in x's type (float16, bfloat16 or float32): in 32 bits, rounded once."""
    if stream is not None:
        return _on(stream, swiglu, x)
    return _front.swiglu(x)


def swiglu_quantized(x: torch.Tensor, codes: str, stream=None):
    """(codes, scales): what ``fp8.quantize_rows`` ("e4m3", N a multiple of 16) or
    ``fp4.quantize_rows`` ("mxfp4", of 32) would make of the unrounded y.  x is 16-byte
    aligned, its rows a multiple of 16 bytes apart; others are refused (:func:`swiglu` takes any)."""
    if stream is not None:
        return _on(stream, swiglu_quantized, x, codes)
    if codes not in CODES:
        raise ValueError("codes must be 'e4m3' or 'mxfp4'")
    return _front.swiglu_quantized(x, CODES[codes])


def swiglu_backward(dy: torch.Tensor, x: torch.Tensor, stream=None) -> torch.Tensor:
    """dx (rows, 2 N) from y's gradient dy (rows, N), both in x's type:
    ``dg = dy u s (1 + g (1 - s))`` and ``du = dy g s``."""
    if stream is not None:
        return _on(stream, swiglu_backward, dy, x)
    return _front.swiglu_backward(dy, x)
