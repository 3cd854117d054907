"""A pre-norm layer with gated experts, as a model would use it.

    python examples/gated_layer.py [--tokens 384] [--hidden 512] [--inner 256] [--experts 6] [--top-k 2]

A layer takes the last layer's branch and the residual stream; it adds them, norms the sum, sends
it to experts whose up product makes gate and factor in one, and gives its own branch and the new
stream.  Here:

* one training step of the layer in bf16, forward and the whole way back, compared with the same
  layer in 64 bits by torch operations and autograd;
* the same forward pass for serving, with the experts' weights in e4m3 or in microscaled 4 bits:
  the gated activation hands its rows on as codes, and the norm behind the layer feeds a dense
  4-bit product (the model's head) the same way.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from all_gather_gemm_chunked_gb300 import act, fp4, fp8, moe, norm  # noqa: E402

EPS = 1e-6


class Layer:
    """Weights of one layer and of a head, and the plans of their products."""

    def __init__(self, hidden: int, inner: int, n_experts: int, top_k: int, vocabulary: int = 1000, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.top_k = top_k
        self.w_norm = (1 + 0.1 * randn(hidden)).bfloat16()
        self.w_router = randn(hidden, n_experts) * hidden ** -0.5
        self.w_up = (randn(n_experts, hidden, 2 * inner) * hidden ** -0.5).bfloat16()  # gate, factor
        self.w_down = (randn(n_experts, inner, hidden) * inner ** -0.5).bfloat16()
        self.up, self.down = moe.Experts(n_experts, hidden, 2 * inner), moe.Experts(n_experts, inner, hidden)
        # for serving: codes and scales, made once
        self.w_last = (1 + 0.1 * randn(hidden)).bfloat16()
        self.head4 = fp4.quantize_weights((randn(hidden, vocabulary) * hidden ** -0.5).bfloat16())
        self.head = fp4.Fp4Linear(hidden, vocabulary)
        self.low = {}
        for name, form, linear in (("e4m3", fp8, fp8.Fp8Linear), ("mxfp4", fp4, fp4.Fp4Linear)):
            self.low[name] = (form, linear(hidden, 2 * inner, n_experts), form.quantize_weights(self.w_up),
                              linear(inner, hidden, n_experts), form.quantize_weights(self.w_down))

    def train_step(self, branch, stream, dout, dstream):
        """(branch, stream, experts, gradients) of one layer for the gradients of its branch and of the stream behind it."""
        n = norm.rms_norm(branch, self.w_norm, EPS, residual=stream)
        logits = n.y.float() @ self.w_router
        r = moe.route(logits, self.top_k)
        rows = moe.gather(n.y, r)
        g = self.up.forward(rows, r.offsets, self.w_up)
        a = act.swiglu(g)
        z = self.down.forward(a, r.offsets, self.w_down)
        out = moe.combine(z, r.slots, r.weights)

        dz, dweights = moe.combine_backward(dout, z, r.slots, r.weights, r.offsets)
        da = self.down.backward_input(dz, r.offsets, self.w_down)
        dw_down = self.down.backward_weight(a, dz, r.offsets)
        dg = act.swiglu_backward(da, g)
        drows = self.up.backward_input(dg, r.offsets, self.w_up)
        dw_up = self.up.backward_weight(rows, dg, r.offsets)
        dlogits = moe.route_backward(logits, r, dweights)
        dy = (moe.combine(drows, r.slots).float() + dlogits @ self.w_router.t()).to(n.y.dtype)
        dx, dw_norm = norm.rms_norm_backward(dy, n.h, self.w_norm, n.rstd, dh=dstream)
        return out, n.h, r.experts, {"x": dx, "w_norm": dw_norm, "w_router": n.y.float().t() @ dlogits, "w_up": dw_up, "w_down": dw_down}

    def serve(self, branch, stream, form: str):
        """The head's logits behind the layer, all products of codes."""
        quantizer, up, w_up, down, w_down = self.low[form]
        n = norm.rms_norm(branch, self.w_norm, EPS, residual=stream)
        r = moe.route(n.y.float() @ self.w_router, self.top_k)
        g = up.forward(*quantizer.quantize_rows(n.y, r), *w_up, r.offsets)
        z = down.forward(*act.swiglu_quantized(g, form), *w_down, r.offsets)
        out = moe.combine(z, r.slots, r.weights)
        xq, xs, _ = norm.rms_norm_quantized(out, self.w_last, "mxfp4", EPS, residual=n.h)
        return self.head.forward(xq, xs, *self.head4)

    def check_status(self):
        for p in (self.up, self.down, self.head, *(q for low in self.low.values() for q in (low[1], low[3]))):
            if p.status() != 0:
                raise RuntimeError("a product's device status is not OK")


def reference(layer: Layer, branch, stream, experts, dout, dstream):
    """The layer in 64 bits by torch operations and autograd (every expert for every token, the
    chosen ones weighted); the stream as it is held, in 16 bits, and the experts that were chosen
    (which of two nearly equal ones a token takes is decided by the last bit of its rows)."""
    h = (branch.float() + stream.float()).to(branch.dtype).double().requires_grad_()
    wn, wr, wu, wd = (t.double().requires_grad_() for t in (layer.w_norm, layer.w_router, layer.w_up, layer.w_down))
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * wn
    p = torch.softmax((y @ wr).gather(1, experts.long()), 1)
    weight = torch.zeros(y.shape[0], wu.shape[0], dtype=torch.float64, device=y.device).scatter(1, experts.long(), p)
    gate, factor = torch.einsum("tk,ekn->etn", y, wu).chunk(2, dim=2)
    out = torch.einsum("te,etn,enk->tk", weight, torch.nn.functional.silu(gate) * factor, wd)
    torch.autograd.backward([out, h], [dout.double(), dstream.double()])
    return out.detach(), {"x": h.grad, "w_norm": wn.grad, "w_router": wr.grad, "w_up": wu.grad, "w_down": wd.grad}


def error(got: torch.Tensor, want: torch.Tensor) -> float:
    return float((got.double() - want).norm() / want.norm())


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 384), ("hidden", 512), ("inner", 256), ("experts", 6), ("top-k", 2)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    branch, stream, dout, dstream = (torch.randn((a.tokens, a.hidden), generator=g, device="cuda").bfloat16() for _ in range(4))
    layer = Layer(a.hidden, a.inner, a.experts, a.top_k)
    out, _, experts, grads = layer.train_step(branch, stream, dout, dstream)
    served = {form: layer.serve(branch, stream, form) for form in layer.low}
    layer.check_status()
    want, want_grads = reference(layer, branch, stream, experts, dout, dstream)
    errors = {"out": error(out, want)}
    errors.update({"d" + k: error(v, want_grads[k]) for k, v in grads.items()})
    for k, v in errors.items():
        print(f"{k:10s} relative error against 64 bits {v:.1e}")
    print(f"head's logits behind 4-bit experts, against e4m3 ones: {error(served['mxfp4'], served['e4m3'].double()):.1e}")
    return {"errors": errors, "served": served}


if __name__ == "__main__":
    main()
