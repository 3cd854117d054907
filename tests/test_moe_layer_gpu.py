"""The example of a whole layer: training step and serving against 64 bits."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [[], ["--tokens", "70", "--hidden", "256", "--inner", "384", "--experts", "12", "--top-k", "5"]])
def test_layer(args):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    errors = m.main(args)
    # bf16: every value passes up to six roundings of at most 2^-8; e4m3: two products of
    # operands that are each off by at most 2^-4, and mostly by less than 2^-5
    for k, v in errors.items():
        assert v <= (2.0 ** -3 if k == "served" else 6 * 2.0 ** -8), (k, v)
