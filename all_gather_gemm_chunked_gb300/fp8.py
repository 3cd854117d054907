"""Torch-tensor front end of the 8-bit products (include/ag_moe.h): operands in e4m3
with a scale for each block of 128, for serving.  No arithmetic here: tensors are
checked and passed to libaggemm.so by the native module ``_front`` (csrc/front.cpp).

Weights are quantised once, rows within each step::

    wq, ws = quantize_weights(w)              # (E, K, N) or (K, N)
    layer = Fp8Linear(K, N, n_experts=E)
    xq, xs = quantize_rows(hidden, routing)   # gathers the experts' rows on the way
    y = layer.forward(xq, xs, wq, ws, routing.offsets)
"""
from __future__ import annotations

import torch

from . import binding as B_
from . import _front
from .moe import _ExpertsPlan, _on

E4M3 = torch.float8_e4m3fn


def quantize_rows(x: torch.Tensor, routing=None, stream=None):
    """(codes (rows, K) e4m3, scales (ceil(K / 128), rows) float32) of the rows of x: in
    each 128 columns s = max(largest magnitude / 448, 2^-126) and code = e4m3(x * (1 / s)),
    rounded to float at each step, the code to the nearest, ties to even.  With a
    ``moe.Routing`` the rows are the experts' rows of x, as ``moe.gather`` gives them."""
    if stream is not None:
        return _on(stream, quantize_rows, x, routing)
    if routing is None:
        return _front.quantize_rows(x, None, None)
    return _front.quantize_rows(x, routing.order, routing.slots)


def quantize_weights(w: torch.Tensor, stream=None):
    """(codes (..., N, K) e4m3, scales (..., ceil(N / 128), ceil(K / 128)) float32) of
    weights (E, K, N) or (K, N): one scale for each 128 x 128 block, the codes laid out
    along K as the product reads them."""
    if stream is not None:
        return _on(stream, quantize_weights, w)
    return _front.quantize_weights(w)


class Fp8Linear(_ExpertsPlan):
    """y[r][n] = sum over the 128-blocks b of K of xs[b][r] * ws[e][n // 128][b] * (the
    block's sum of xq * wq), for one weight matrix or, with offsets, for the rows of
    ``n_experts`` experts.  Sums of a block in the tensor core's 32 bits, over the
    blocks in 32-bit registers.  K is a multiple of 16, N of 8.  Forward only, without
    autograd: training goes through moe.Experts."""

    def __init__(self, K: int, N: int, n_experts: int = 1):
        super().__init__(n_experts, K, N, B_.E4M3)

    def forward(self, xq, xs, wq, ws, offsets=None, out=None, out_dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
        if stream is not None:
            return _on(stream, self.forward, xq, xs, wq, ws, offsets, out, out_dtype)
        return _front.fp8_product(self.handle, self.n_experts, self.K, self.N, xq, xs, wq, ws, offsets,
                                  out, out_dtype)
