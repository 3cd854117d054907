"""The example of a gated layer: a training step's output and gradients against 64 bits, and that serving runs."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [[], ["--tokens", "45", "--hidden", "160", "--inner", "96", "--experts", "9", "--top-k", "4"]])
def test_layer(args):
    spec = importlib.util.spec_from_file_location("gated_layer", os.path.join(ROOT, "examples", "gated_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    found = m.main(args)
    # bf16: every value passes up to nine roundings of at most 2^-8 (norm, gather's product, activation, product,
    # combination and, back, gradients of rows, activation, product, sum)
    for k, v in found["errors"].items():
        assert v <= 9 * 2.0 ** -8, (k, v)
    for v in found["served"].values():
        assert v.shape[1] == 1000 and bool(torch.isfinite(v).all()) and bool(v.any())
