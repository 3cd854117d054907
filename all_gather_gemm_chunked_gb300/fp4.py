"""Torch-tensor front end of the 4-bit products (include/ag_layer.h): microscaled operands,
e2m1 codes with a power-of-two scale (e8m0) for each 32 elements along K, for serving.  No
arithmetic here: tensors are checked and passed to libaggemm.so by the native module
``_front`` (csrc/front.cpp).

Weights are quantised once, rows within each step::

    wq, ws = quantize_weights(w)              # (E, K, N) or (K, N)
    layer = Fp4Linear(K, N, n_experts=E)
    xq, xs = quantize_rows(hidden, routing)   # gathers the experts' rows on the way
    y = layer.forward(xq, xs, wq, ws, routing.offsets)

A scale 2^E is the smallest power of two, from 2^-127 on, with its block's largest magnitude
below 7 * 2^E; the codes are x / 2^E, rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6
(ties to the even code), with a sign, two to a byte, the first in the low four bits.  An
infinity or NaN makes its whole block NaN.
"""
from __future__ import annotations

import torch

from . import binding as B_
from . import _front
from .moe import _ExpertsPlan, _on

E8M0 = torch.float8_e8m0fnu


def quantize_rows(x: torch.Tensor, routing=None, stream=None):
    """(codes (rows, K / 2) uint8, scales (ceil(K / 128), rows, 4) float8_e8m0fnu) of the rows
    of x (K a multiple of 32): the scale of row r and block b of 32 at [b // 4, r, b % 4].
    With a ``moe.Routing`` the rows are the experts' rows of x, as ``moe.gather`` gives them.
    x is 16-byte aligned, its rows a multiple of 16 bytes apart."""
    if stream is not None:
        return _on(stream, quantize_rows, x, routing)
    if routing is None:
        return _front.fp4_quantize_rows(x, None, None)
    return _front.fp4_quantize_rows(x, routing.order, routing.slots)


def quantize_weights(w: torch.Tensor, stream=None):
    """(codes (..., N, K / 2) uint8, scales (..., ceil(N / 128), ceil(K / 128), 32, 4, 4)
    float8_e8m0fnu) of contiguous, 16-byte aligned weights (E, K, N) or (K, N), K a multiple of 32 and N of 8, laid out as
    the product reads them: the scale of column n and block b of 32 along K at
    [n // 128, b // 4, n % 32, n % 128 // 32, b % 4]."""
    if stream is not None:
        return _on(stream, quantize_weights, w)
    return _front.fp4_quantize_weights(w)


class Fp4Linear(_ExpertsPlan):
    """y[r][n] = the sum over k of the values that the codes and scales of row r and of column
    n stand for, for one weight matrix or, with offsets, for the rows of ``n_experts`` experts.
    Sums in the tensor core's 32 bits, collected in 32-bit registers.  K is a multiple of 32,
    N of 8.  Forward only, without autograd: training goes through moe.Experts."""

    def __init__(self, K: int, N: int, n_experts: int = 1):
        super().__init__(n_experts, K, N, B_.E2M1)

    def forward(self, xq, xs, wq, ws, offsets=None, out=None, out_dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
        if stream is not None:
            return _on(stream, self.forward, xq, xs, wq, ws, offsets, out, out_dtype)
        return _front.fp4_product(self.handle, self.n_experts, self.K, self.N, xq, xs, wq, ws, offsets,
                                  out, out_dtype)
