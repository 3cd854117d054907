"""A mixture-of-experts layer behind a gathered product, as a model would use it.

    python examples/moe_layer.py [--tokens 512] [--hidden 1024] [--inner 512] [--experts 8] [--top-k 2]

The hidden states come out of a streamed AllGather+GEMM (two shards).  Then

* one training step of the layer in bf16: router, the experts' rows, two products by
  expert with an activation between them, the combination, and the whole way back;
* the same forward pass for serving, with the weights in e4m3 (a scale for each block
  of 128) and the rows quantised on their way to the experts.

Both are compared with the same layer written with torch operations in 64 bits.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from all_gather_gemm_chunked_gb300 import fp8, moe  # noqa: E402
from all_gather_gemm_chunked_gb300.plan import Plan  # noqa: E402


class Layer:
    """Weights of one layer and the plans of its products."""

    def __init__(self, hidden: int, inner: int, n_experts: int, top_k: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.top_k = top_k
        self.w_router = randn(hidden, n_experts) * hidden ** -0.5
        self.w_up = (randn(n_experts, hidden, inner) * hidden ** -0.5).bfloat16()
        self.w_down = (randn(n_experts, inner, hidden) * inner ** -0.5).bfloat16()
        self.up, self.down = moe.Experts(n_experts, hidden, inner), moe.Experts(n_experts, inner, hidden)
        # for serving: codes and scales, made once
        self.up8, self.down8 = fp8.quantize_weights(self.w_up), fp8.quantize_weights(self.w_down)
        self.low_up = fp8.Fp8Linear(hidden, inner, n_experts)
        self.low_down = fp8.Fp8Linear(inner, hidden, n_experts)

    def train_step(self, x: torch.Tensor, dout: torch.Tensor):
        """(out, gradients) for hidden states x and the gradient of the layer's output."""
        logits = x.float() @ self.w_router
        r = moe.route(logits, self.top_k)
        rows = moe.gather(x, r)
        h = self.up.forward(rows, r.offsets, self.w_up)
        a = torch.nn.functional.silu(h)
        y = self.down.forward(a, r.offsets, self.w_down)
        out = moe.combine(y, r.slots, r.weights)

        dy, dweights = moe.combine_backward(dout, y, r.slots, r.weights, r.offsets)
        da = self.down.backward_input(dy, r.offsets, self.w_down)
        dw_down = self.down.backward_weight(a, dy, r.offsets)
        s = torch.sigmoid(h.float())
        dh = (da.float() * s * (1 + h.float() * (1 - s))).to(h.dtype)
        drows = self.up.backward_input(dh, r.offsets, self.w_up)
        dw_up = self.up.backward_weight(rows, dh, r.offsets)
        dlogits = moe.route_backward(logits, r, dweights)
        dx = moe.combine(drows, r.slots).float() + dlogits @ self.w_router.t()
        return out, {"x": dx, "w_router": x.float().t() @ dlogits, "w_up": dw_up, "w_down": dw_down}

    def serve(self, x: torch.Tensor) -> torch.Tensor:
        r = moe.route(x.float() @ self.w_router, self.top_k)
        h = self.low_up.forward(*fp8.quantize_rows(x, r), *self.up8, r.offsets)
        a = torch.nn.functional.silu(h)
        y = self.low_down.forward(*fp8.quantize_rows(a), *self.down8, r.offsets)
        return moe.combine(y, r.slots, r.weights)

    def check_status(self):
        for p in (self.up, self.down, self.low_up, self.low_down):
            if p.status() != 0:
                raise RuntimeError("a product's device status is not OK")


def reference(layer: Layer, x: torch.Tensor, dout: torch.Tensor):
    """The layer in 64 bits by torch operations and autograd (every expert for every
    token, the chosen ones weighted)."""
    x, wr, wu, wd = (t.double().requires_grad_() for t in (x, layer.w_router, layer.w_up, layer.w_down))
    top, idx = torch.sort((x @ wr), dim=1, descending=True, stable=True)
    p = torch.softmax(top[:, :layer.top_k], 1)
    weight = torch.zeros(x.shape[0], wu.shape[0], dtype=torch.float64, device=x.device).scatter(1, idx[:, :layer.top_k], p)
    h = torch.nn.functional.silu(torch.einsum("tk,ekn->etn", x, wu))
    out = torch.einsum("te,etn,enk->tk", weight, h, wd)
    out.backward(dout.double())
    return out.detach(), {"x": x.grad, "w_router": wr.grad, "w_up": wu.grad, "w_down": wd.grad}


def error(got: torch.Tensor, want: torch.Tensor) -> float:
    return float((got.double() - want).norm() / want.norm())


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 512), ("hidden", 1024), ("inner", 512), ("experts", 8), ("top-k", 2)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # hidden states: the gathered rows of two shards times a weight matrix
    shards = [randn(a.tokens // 2, a.hidden).bfloat16() for _ in range(2)]
    with Plan(2, 2 * (a.tokens // 2), a.hidden, a.hidden, "bf16") as plan:
        x = plan.run(shards, (randn(a.hidden, a.hidden) * a.hidden ** -0.5).bfloat16()).bfloat16()
        if plan.status() != 0:
            raise RuntimeError("the gathered product's device status is not OK")
    dout = randn(x.shape[0], a.hidden).bfloat16()
    layer = Layer(a.hidden, a.inner, a.experts, a.top_k)
    out, grads = layer.train_step(x, dout)
    served = layer.serve(x)
    layer.check_status()
    want, want_grads = reference(layer, x, dout)
    errors = {"out": error(out, want), "served": error(served, want)}
    errors.update({"d" + k: error(v, want_grads[k]) for k, v in grads.items()})
    for k, v in errors.items():
        print(f"{k:10s} relative error against 64 bits {v:.1e}")
    return errors


if __name__ == "__main__":
    main()
