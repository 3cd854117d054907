"""Torch-tensor front end of the 8-bit products (include/ag_moe.h): operands in e4m3
with a scale for each block of 128, for serving.  Checks tensors and passes their
device pointers and the stream to libaggemm.so; no arithmetic here.

Weights are quantised once, rows within each step::

    wq, ws = quantize_weights(w)              # (E, K, N) or (K, N)
    layer = Fp8Linear(K, N, n_experts=E)
    xq, xs = quantize_rows(hidden, routing)   # gathers the experts' rows on the way
    y = layer.forward(xq, xs, wq, ws, routing.offsets)
"""
from __future__ import annotations

import torch

from . import binding as B_
from .moe import _current_stream, _ExpertsPlan, _on, _plain, _rows, _type, _TYPES

E4M3 = torch.float8_e4m3fn


def _blocks(n: int) -> int:
    return -(-n // B_.SCALE_BLOCK)


def quantize_rows(x: torch.Tensor, routing=None, stream=None):
    """(codes (rows, K) e4m3, scales (ceil(K / 128), rows) float32) of the rows of x: in
    each 128 columns s = max(largest magnitude / 448, 2^-126) and code = e4m3(x * (1 / s)),
    rounded to float at each step, the code to the nearest, ties to even.  With a
    ``moe.Routing`` the rows are the experts' rows of x, as ``moe.gather`` gives them."""
    if stream is not None:
        return _on(stream, quantize_rows, x, routing)
    code, ld = _type(x, "x"), _rows(x, "x")
    src, K = x.shape
    rows, order, k = src, None, 1
    if routing is not None:
        k = routing.slots.shape[1]
        rows = src * k
        order = _plain(routing.order, "routing.order", torch.int32, (rows,))
    q = torch.empty((rows, K), dtype=E4M3, device=x.device)
    s = torch.empty((_blocks(K), rows), dtype=torch.float32, device=x.device)
    B_.ag_fp8_quantize_rows(rows, K, code, x.data_ptr(), ld, src, order, k, q.data_ptr(), s.data_ptr(),
                            _current_stream(x.get_device()))
    return q, s


def quantize_weights(w: torch.Tensor, stream=None):
    """(codes (..., N, K) e4m3, scales (..., ceil(N / 128), ceil(K / 128)) float32) of
    weights (E, K, N) or (K, N): one scale for each 128 x 128 block, the codes laid out
    along K as the product reads them."""
    if stream is not None:
        return _on(stream, quantize_weights, w)
    code = _type(w, "w")
    if w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w must be a contiguous (E, K, N) or (K, N) tensor")
    E = w.shape[0] if w.dim() == 3 else 1
    K, N = w.shape[-2:]
    lead = tuple(w.shape[:-2])
    q = torch.empty(lead + (N, K), dtype=E4M3, device=w.device)
    s = torch.empty(lead + (_blocks(N), _blocks(K)), dtype=torch.float32, device=w.device)
    B_.ag_fp8_quantize_weights(E, K, N, code, w.data_ptr(), q.data_ptr(), s.data_ptr(),
                               _current_stream(w.get_device()))
    return q, s


class Fp8Linear(_ExpertsPlan):
    """y[r][n] = sum over the 128-blocks b of K of xs[b][r] * ws[e][n // 128][b] * (the
    block's sum of xq * wq), for one weight matrix or, with offsets, for the rows of
    ``n_experts`` experts.  Sums of a block in the tensor core's 32 bits, over the
    blocks in 32-bit registers.  Forward only: training goes through moe.Experts."""

    def __init__(self, K: int, N: int, n_experts: int = 1):
        self._xs_blocks = _blocks(K)
        self._w_shape, self._ws_shape = (N, K), (_blocks(N), _blocks(K))
        super().__init__(n_experts, K, N, B_.E4M3)

    def forward(self, xq, xs, wq, ws, offsets=None, out=None, out_dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
        if stream is not None:
            return _on(stream, self.forward, xq, xs, wq, ws, offsets, out, out_dtype)
        rows, N = xq.shape[0], self.N
        lead = () if self.n_experts == 1 and wq.dim() == 2 else (self.n_experts,)
        a = _plain(xq, "xq", E4M3, (rows, self.K))
        b = _plain(xs, "xs", torch.float32, (self._xs_blocks, rows))
        c = _plain(wq, "wq", E4M3, lead + self._w_shape)
        d = _plain(ws, "ws", torch.float32, lead + self._ws_shape)
        off = self._offsets(offsets)
        if out is None:
            out, ldo = torch.empty((rows, N), dtype=out_dtype, device=xq.device), N
        else:
            out = self._out(out, (rows, N), out_dtype, xq.device)
            ldo = _rows(out, "out")
        B_.ag_fp8_forward(self.handle, rows, a, b, off, c, d, out.data_ptr(), ldo,
                          _TYPES.get(out_dtype, -1), _current_stream(xq.get_device()))
        return out
