"""Torch-tensor front end of the mixture-of-experts operators (include/ag_moe.h):
the router, the moves of rows between tokens and experts, and the products grouped
by expert, each with its gradient.  Checks tensors and passes their device pointers
and the stream to libaggemm.so; no arithmetic here.

A layer's forward pass::

    r = route(logits, top_k)                  # weights, experts and the rows' layout
    x = gather(hidden, r)                     # the experts' rows, sorted by expert
    h = up.forward(x, r.offsets, w_up)        # Experts
    y = down.forward(act(h), r.offsets, w_down)
    out = combine(y, r.slots, r.weights)

``stream`` (every function): a torch stream, None for the current one.  Outputs are
allocated on it; inputs written on another stream need the caller's event, as in any
torch program.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B_

_TYPES = {torch.float16: B_.F16, torch.bfloat16: B_.BF16, torch.float32: B_.F32}
_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


class Routing(NamedTuple):
    """What :func:`route` decides for T tokens and E experts."""
    weights: torch.Tensor  # (T, top_k) float32
    experts: torch.Tensor  # (T, top_k) int32, -1: no choice
    offsets: torch.Tensor  # (E + 1,) int32: expert e's rows are offsets[e]:offsets[e + 1]
    order: torch.Tensor    # (T * top_k,) int32: row -> token * top_k + j, -1: row not in use
    slots: torch.Tensor    # (T, top_k) int32: choice -> row, -1: none
    normalize: bool


# A call's host side is about as long as a small kernel, so the checks below take the
# passing case first and say what is wrong only once something is.

def _current_stream(device_index: int) -> int:
    return torch.cuda.current_stream(device_index).cuda_stream


# torch's own quick form of the same (3 us less a call), where this version has it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _on(stream, fn, *args):
    """fn(*args) with `stream` current: outputs are allocated on it."""
    with torch.cuda.stream(stream):
        return fn(*args)


def _refuse(t, name, dtype=None, shape=None):
    """Raises for what is wrong with a tensor that failed a check."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dtype is None and t.dtype not in _TYPES:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _type(t, name: str) -> int:
    code = _TYPES.get(getattr(t, "dtype", None))
    if code is None or not t.is_cuda:
        _refuse(t, name)
    return code


def _rows(t, name: str, cols: Optional[int] = None) -> int:
    """Row pitch of a matrix whose rows are contiguous (a column block of a wider
    matrix is one)."""
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must have shape (rows, {'columns' if cols is None else cols}), got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.shape[1]
    if t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0)


def _plain(t, name: str, dtype, shape) -> int:
    """Device pointer of a contiguous tensor of this type and shape."""
    if getattr(t, "dtype", None) != dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _refuse(t, name, dtype, shape)
    return t.data_ptr()


# ---------------------------------------------------------------- router
def route(logits: torch.Tensor, top_k: int, normalize: bool = True, stream=None) -> Routing:
    """The ``top_k`` largest logits of each token (T x E; ties: the lowest expert; -inf
    is never chosen), their weights -- the softmax over the chosen ones, or with
    ``normalize=False`` the chosen entries of the softmax over all experts -- and the
    layout of the rows sorted by expert."""
    if stream is not None:
        return _on(stream, route, logits, top_k, normalize)
    code, ld = _type(logits, "logits"), _rows(logits, "logits")
    T, E = logits.shape
    size = B_.ag_moe_route_workspace(T, E, top_k)
    dev, i32 = logits.device, torch.int32
    weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    experts = torch.empty((T, top_k), dtype=i32, device=dev)
    offsets = torch.empty(E + 1, dtype=i32, device=dev)
    order = torch.empty(T * top_k, dtype=i32, device=dev)
    slots = torch.empty((T, top_k), dtype=i32, device=dev)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    B_.ag_moe_route(T, E, top_k, code, logits.data_ptr(), ld, int(normalize),
                    weights.data_ptr(), experts.data_ptr(), offsets.data_ptr(),
                    order.data_ptr(), slots.data_ptr(), ws.data_ptr() if size else None,
                    _current_stream(logits.get_device()))
    return Routing(weights, experts, offsets, order, slots, normalize)


def route_backward(logits: torch.Tensor, routing: Routing, dweights: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """Gradient of the logits (their type) from that of ``routing.weights``."""
    if stream is not None:
        return _on(stream, route_backward, logits, routing, dweights)
    code, ld = _type(logits, "logits"), _rows(logits, "logits")
    T, E = logits.shape
    k = routing.weights.shape[1]
    w = _plain(routing.weights, "routing.weights", torch.float32, (T, k))
    e = _plain(routing.experts, "routing.experts", torch.int32, (T, k))
    dw = _plain(dweights, "dweights", torch.float32, (T, k))
    out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    B_.ag_moe_route_backward(T, E, k, code, logits.data_ptr(), ld, int(routing.normalize), w, e,
                             dw, out.data_ptr(), _current_stream(logits.get_device()))
    return out


# ---------------------------------------------------------------- rows
def gather(x: torch.Tensor, routing: Routing, stream=None) -> torch.Tensor:
    """The experts' rows: row s is x's row ``routing.order[s] // top_k`` (zeros where a
    row is not in use).  Its gradient is ``combine(dx, routing.slots)``."""
    if stream is not None:
        return _on(stream, gather, x, routing)
    code, ld = _type(x, "x"), _rows(x, "x")
    T, H = x.shape
    k = routing.slots.shape[1]
    order = _plain(routing.order, "routing.order", torch.int32, (T * k,))
    out = torch.empty((T * k, H), dtype=x.dtype, device=x.device)
    B_.ag_moe_gather(T, k, H, code, x.data_ptr(), ld, order, out.data_ptr(), _current_stream(x.get_device()))
    return out


def combine(y: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """``out[t] = sum over j of weights[t, j] * y[slots[t, j]]``, summed in 32 bits
    (``weights`` None: 1 each)."""
    if stream is not None:
        return _on(stream, combine, y, slots, weights)
    code, ld = _type(y, "y"), _rows(y, "y")
    T, k = slots.shape
    if y.shape[0] != T * k:
        raise ValueError(f"y must have {T * k} rows, got {y.shape[0]}")
    H = y.shape[1]
    s = _plain(slots, "slots", torch.int32, (T, k))
    w = None if weights is None else _plain(weights, "weights", torch.float32, (T, k))
    out = torch.empty((T, H), dtype=y.dtype, device=y.device)
    B_.ag_moe_combine(T, k, H, code, y.data_ptr(), ld, s, w, out.data_ptr(), _current_stream(y.get_device()))
    return out


def combine_backward(dout: torch.Tensor, y: torch.Tensor, slots: torch.Tensor,
                     weights: torch.Tensor, offsets: Optional[torch.Tensor] = None, stream=None):
    """(dy, dweights) of :func:`combine`.  With ``offsets`` the rows of dy that belong to
    no choice (from ``offsets[-1]`` on) become zeros; without it every row must belong
    to one."""
    if stream is not None:
        return _on(stream, combine_backward, dout, y, slots, weights, offsets)
    code, ld, ldd = _type(y, "y"), _rows(y, "y"), _rows(dout, "dout", y.shape[1])
    if dout.dtype != y.dtype or not dout.is_cuda:
        raise TypeError(f"dout must be {y.dtype} on a CUDA device, got {dout.dtype} on {dout.device}")
    T, k = slots.shape
    if y.shape[0] != T * k or dout.shape[0] != T:
        raise ValueError(f"y must have {T * k} rows and dout {T}, got {y.shape[0]} and {dout.shape[0]}")
    H = y.shape[1]
    s = _plain(slots, "slots", torch.int32, (T, k))
    w = _plain(weights, "weights", torch.float32, (T, k))
    end = None
    if offsets is not None:
        end = _plain(offsets, "offsets", torch.int32, (offsets.numel(),)) + 4 * (offsets.numel() - 1)
    dy = torch.empty((T * k, H), dtype=y.dtype, device=y.device)
    dw = torch.empty((T, k), dtype=torch.float32, device=y.device)
    B_.ag_moe_combine_backward(T, k, H, code, dout.data_ptr(), ldd, y.data_ptr(), ld, s, w, end,
                               dy.data_ptr(), dw.data_ptr(), _current_stream(y.get_device()))
    return dy, dw


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

    def _offsets(self, offsets):
        if offsets is None:
            return None
        return _plain(offsets, "offsets", torch.int32, (self.n_experts + 1,))

    def _out(self, out, shape, dtype, device):
        if out is None:
            return torch.empty(shape, dtype=dtype, device=device)
        if getattr(out, "dtype", None) != dtype or out.shape != shape or not out.is_cuda:
            _refuse(out, "out", dtype, shape)
        return out


class Experts(_ExpertsPlan):
    """Products of one layer's experts: ``n_experts`` weight matrices K x N ("f16" or
    "bf16"), for rows sorted by expert with ``offsets`` (n_experts + 1 int32 on the
    device; None: one expert, all rows).  Accumulation in 32 bits; outputs have the
    operands' type or float32.  Rows outside [offsets[0], offsets[-1]) are not written
    (an ``out`` of the caller's keeps them).

    Serves x rows of any number from 0 on; x, dy and out may be column blocks of wider
    matrices, w any (n_experts, K, N) tensor with contiguous rows."""

    def __init__(self, n_experts: int, K: int, N: int, dtype: str = "bf16"):
        if dtype not in _TORCH:
            raise ValueError("dtype must be 'f16' or 'bf16'")
        self.dtype = _TORCH[dtype]
        self._w_shape = (n_experts, K, N)
        super().__init__(n_experts, K, N, _TYPES[self.dtype])

    def _rows_of(self, t, name, cols):
        if getattr(t, "dtype", None) != self.dtype or not t.is_cuda:
            _refuse(t, name, self.dtype)
        return _rows(t, name, cols)

    def _weights(self, w):
        if getattr(w, "dtype", None) != self.dtype or not w.is_cuda or w.shape != self._w_shape:
            _refuse(w, "w", self.dtype, self._w_shape)
        if w.is_contiguous():
            return self.N, self.K * self.N
        if w.stride(2) != 1:
            raise ValueError("w must have contiguous rows")
        return w.stride(1), w.stride(0)

    def _product(self, call, name, t, offsets, w, cols, wide, out, out_dtype):
        ld = self._rows_of(t, name, cols)
        ldw, ldw_e = self._weights(w)
        off = self._offsets(offsets)
        dt = self.dtype if out_dtype is None else out_dtype
        rows = t.shape[0]
        if out is None:
            out, ldo = torch.empty((rows, wide), dtype=dt, device=t.device), wide
        else:
            out = self._out(out, (rows, wide), dt, t.device)
            ldo = _rows(out, "out")
        call(self.handle, rows, t.data_ptr(), ld, off, w.data_ptr(), ldw, ldw_e, out.data_ptr(), ldo,
             _TYPES.get(dt, -1), _current_stream(t.get_device()))
        return out

    def forward(self, x, offsets, w, out=None, out_dtype=None, stream=None) -> torch.Tensor:
        """y (rows x N): row r of expert e is x[r] w[e]."""
        if stream is not None:
            return _on(stream, self.forward, x, offsets, w, out, out_dtype)
        return self._product(B_.ag_moe_forward, "x", x, offsets, w, self.K, self.N, out, out_dtype)

    def backward_input(self, dy, offsets, w, out=None, out_dtype=None, stream=None) -> torch.Tensor:
        """dx (rows x K): row r of expert e is dy[r] w[e]^T."""
        if stream is not None:
            return _on(stream, self.backward_input, dy, offsets, w, out, out_dtype)
        return self._product(B_.ag_moe_backward_input, "dy", dy, offsets, w, self.N, self.K, out,
                             out_dtype)

    def backward_weight(self, x, dy, offsets, out=None, out_dtype=torch.float32,
                        stream=None) -> torch.Tensor:
        """dw (n_experts x K x N, float32 by default): x^T dy over each expert's rows,
        zeros for an expert without rows."""
        if stream is not None:
            return _on(stream, self.backward_weight, x, dy, offsets, out, out_dtype)
        ldx, ldd = self._rows_of(x, "x", self.K), self._rows_of(dy, "dy", self.N)
        if x.shape[0] != dy.shape[0]:
            raise ValueError(f"x and dy must have the same rows, got {x.shape[0]} and {dy.shape[0]}")
        off = self._offsets(offsets)
        out = self._out(out, self._w_shape, out_dtype, x.device)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        B_.ag_moe_backward_weight(self.handle, x.shape[0], x.data_ptr(), ldx, dy.data_ptr(), ldd, off,
                                  out.data_ptr(), _TYPES.get(out_dtype, -1),
                                  _current_stream(x.get_device()))
        return out
