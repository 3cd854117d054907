"""Torch-tensor front end of the mixture-of-experts operators (include/ag_moe.h):
the router, the moves of rows between tokens and experts, and the products grouped
by expert, each with its gradient.  No arithmetic here: tensors are checked and passed
to libaggemm.so by the native module ``_front`` (csrc/front.cpp), which must be built.

A layer's forward pass::

    r = route(logits, top_k)                  # weights, experts and the rows' layout
    x = gather(hidden, r)                     # the experts' rows, sorted by expert
    h = up.forward(x, r.offsets, w_up)        # Experts
    y = down.forward(act(h), r.offsets, w_down)
    out = combine(y, r.slots, r.weights)

The functions know nothing of autograd: outputs carry no gradient, whatever the inputs
say; a backward pass calls the ``backward`` functions itself (examples/moe_layer.py).

The tensors of a call, its plan and its stream are on one device, which need not be the
current one.

``stream`` (every function): a torch stream, None for the current one.  Outputs are
allocated on it; inputs written on another stream need the caller's event, as in any
torch program.
"""
from __future__ import annotations

import re
from typing import NamedTuple, Optional

import torch

from . import binding as B_
from . import _front


def _same_torch(built: str, here: str) -> bool:
    return built == re.match(r"[0-9.]*[0-9]", here).group()


if not _same_torch(_front.torch_version, torch.__version__):
    raise ImportError(f"the native module was built for torch {_front.torch_version}, this is {torch.__version__}: "
                      "run the package's build again")
_front.init(B_._err)
_CODES = {"f16": (torch.float16, B_.F16), "bf16": (torch.bfloat16, B_.BF16)}


class Routing(NamedTuple):
    """What :func:`route` decides for T tokens and E experts."""
    weights: torch.Tensor  # (T, top_k) float32
    experts: torch.Tensor  # (T, top_k) int32, -1: no choice
    offsets: torch.Tensor  # (E + 1,) int32: expert e's rows are offsets[e]:offsets[e + 1]
    order: torch.Tensor    # (T * top_k,) int32: row -> token * top_k + j, -1: row not in use
    slots: torch.Tensor    # (T, top_k) int32: choice -> row, -1: none
    normalize: bool


def _on(stream, fn, *args):
    """fn(*args) with `stream` current: outputs are allocated on it."""
    first = next((a for a in args if isinstance(a, torch.Tensor)), None)
    if first is not None and first.is_cuda and first.device != stream.device:
        raise ValueError(f"stream is on device {stream.device}, the call's first tensor on {first.device}")
    with torch.cuda.stream(stream):
        return fn(*args)


# ---------------------------------------------------------------- router
def route(logits: torch.Tensor, top_k: int, normalize: bool = True, stream=None) -> Routing:
    """The ``top_k`` largest logits of each token (T x E; ties: the lowest expert; -inf
    is never chosen), their weights -- the softmax over the chosen ones, or with
    ``normalize=False`` the chosen entries of the softmax over all experts -- and the
    layout of the rows sorted by expert."""
    if stream is not None:
        return _on(stream, route, logits, top_k, normalize)
    return tuple.__new__(Routing, _front.route(logits, top_k, normalize))


def route_backward(logits: torch.Tensor, routing: Routing, dweights: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """Gradient of the logits (their type) from that of ``routing.weights``."""
    if stream is not None:
        return _on(stream, route_backward, logits, routing, dweights)
    return _front.route_backward(logits, routing.weights, routing.experts, dweights,
                                 routing.normalize)


# ---------------------------------------------------------------- rows
def gather(x: torch.Tensor, routing: Routing, stream=None) -> torch.Tensor:
    """The experts' rows: row s is x's row ``routing.order[s] // top_k`` (zeros where a
    row is not in use).  Its gradient is ``combine(dx, routing.slots)``."""
    if stream is not None:
        return _on(stream, gather, x, routing)
    return _front.gather(x, routing.order, routing.slots)


def combine(y: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """``out[t] = sum over j of weights[t, j] * y[slots[t, j]]``, summed in 32 bits
    (``weights`` None: 1 each)."""
    if stream is not None:
        return _on(stream, combine, y, slots, weights)
    return _front.combine(y, slots, weights)


def combine_backward(dout: torch.Tensor, y: torch.Tensor, slots: torch.Tensor,
                     weights: torch.Tensor, offsets: Optional[torch.Tensor] = None, stream=None):
    """(dy, dweights) of :func:`combine`.  With ``offsets`` the rows of dy that belong to
    no choice (from ``offsets[-1]`` on) become zeros; without it every row must belong
    to one."""
    if stream is not None:
        return _on(stream, combine_backward, dout, y, slots, weights, offsets)
    return _front.combine_backward(dout, y, slots, weights, offsets)


# ---------------------------------------------------------------- products by expert
class _ExpertsPlan:
    """Owns a library plan (workspace of split sums, status)."""

    def __init__(self, n_experts: int, K: int, N: int, code: int):
        self.n_experts, self.K, self.N = n_experts, K, N
        self.handle = B_.ag_moe_plan_create(n_experts, K, N, code)

    def close(self):
        if getattr(self, "handle", None):
            B_.ag_moe_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def tile_rows(self, rows: int, input_gradient: bool = False) -> int:
        """Rows of the tiles, 64 or 256, that a product of so many rows is cut into."""
        return B_.ag_moe_plan_tile_rows(self.handle, rows, input_gradient)

    def status(self) -> int:
        """Waits for the last run; 0, or binding.ERR_TIMEOUT / ERR_INVALID (offsets)."""
        return B_.ag_moe_plan_status(self.handle)

    def status_word(self) -> int:
        return B_.ag_moe_plan_status_word(self.handle)

    def reset(self, stream=None):
        stream = torch.cuda.current_stream() if stream is None else stream
        B_.ag_moe_plan_reset(self.handle, stream.cuda_stream)

    def set_timeout_ns(self, ns: int):
        B_.ag_moe_plan_set_timeout_ns(self.handle, ns)


class Experts(_ExpertsPlan):
    """Products of one layer's experts: ``n_experts`` weight matrices K x N ("f16" or
    "bf16"), for rows sorted by expert with ``offsets`` (n_experts + 1 int32 on the
    device; None: one expert, all rows).  Accumulation in 32 bits; outputs have the
    operands' type or float32.  Rows outside [offsets[0], offsets[-1]) are not written
    (an ``out`` of the caller's keeps them).

    K and N are multiples of 8.  Rows of any number from 0 on; x, dy and out may be column
    blocks of wider matrices, w may have its rows and its experts further apart than they
    are long (each expert's K rows behind the last one's); pitches are multiples of 16
    bytes."""

    def __init__(self, n_experts: int, K: int, N: int, dtype: str = "bf16"):
        if dtype not in _CODES:
            raise ValueError("dtype must be 'f16' or 'bf16'")
        self.dtype, code = _CODES[dtype]
        super().__init__(n_experts, K, N, code)

    def forward(self, x, offsets, w, out=None, out_dtype=None, stream=None) -> torch.Tensor:
        """y (rows x N): row r of expert e is x[r] w[e]."""
        if stream is not None:
            return _on(stream, self.forward, x, offsets, w, out, out_dtype)
        return _front.rows_product(self.handle, self.n_experts, self.K, self.N, self.dtype, False, x,
                                   offsets, w, out, out_dtype)

    def backward_input(self, dy, offsets, w, out=None, out_dtype=None, stream=None) -> torch.Tensor:
        """dx (rows x K): row r of expert e is dy[r] w[e]^T."""
        if stream is not None:
            return _on(stream, self.backward_input, dy, offsets, w, out, out_dtype)
        return _front.rows_product(self.handle, self.n_experts, self.K, self.N, self.dtype, True, dy,
                                   offsets, w, out, out_dtype)

    def backward_weight(self, x, dy, offsets, out=None, out_dtype=torch.float32,
                        stream=None) -> torch.Tensor:
        """dw (n_experts x K x N, float32 by default): x^T dy over each expert's rows,
        zeros for an expert without rows."""
        if stream is not None:
            return _on(stream, self.backward_weight, x, dy, offsets, out, out_dtype)
        return _front.weight_product(self.handle, self.n_experts, self.K, self.N, self.dtype, x, dy,
                                     offsets, out, out_dtype)
