"""The router's layout where one block places very many tokens, and in its two-kernel form
for every number of experts a lane holds."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from all_gather_gemm_chunked_gb300 import moe  # noqa: E402
from moe_util import randn, rng, route_ref  # noqa: E402


def _check_layout(r, E):
    """offsets, order and slots of the choices r.experts, by a stable sort."""
    flat = torch.where(r.experts >= 0, r.experts, E).reshape(-1)
    order = torch.sort(flat, stable=True)[1].int()
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    used = int(counts.sum())
    assert torch.equal(r.offsets[1:].long(), counts.cumsum(0)) and int(r.offsets[0]) == 0
    order[used:] = -1
    assert torch.equal(r.order, order)
    slots = torch.full_like(flat, -1)
    slots[order[:used].long()] = torch.arange(used, dtype=torch.int32, device="cuda")
    assert torch.equal(r.slots.reshape(-1), slots)


# more tokens on one expert than 16 bits count in a block: nearly all on one of two, all
# on the only one, every token on both
@pytest.mark.parametrize("T,E,k", [((1 << 24) + 5, 2, 1), (10_500_001, 1, 1), ((1 << 24) - 3, 2, 2)])
def test_many_tokens_on_one_expert(T, E, k):
    logits = torch.zeros((T, E), dtype=torch.float16, device="cuda")
    if k < E:
        logits[::1000, 1] = 1.0
    r = moe.route(logits, k)
    if k < E:
        assert torch.equal(r.experts[:, 0], (torch.arange(T, device="cuda") % 1000 == 0).int())
    _check_layout(r, E)


@pytest.mark.parametrize("T,E,k", [(700, 600, 6), (650, 1024, 32), (5000, 513, 3), (40000, 900, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_kernels_of_many_experts(T, E, k, dtype):
    logits = randn(rng(T + E), (T, E), dtype)
    logits[::7] = logits[::7].masked_fill(torch.rand((1, E), generator=rng(1), device="cuda") < 0.98, float("-inf"))
    r = moe.route(logits, k)
    _check_layout(r, E)
    some = np.arange(0, T, max(1, T // 300))
    ref = route_ref(logits[torch.from_numpy(some).cuda()], k)
    assert np.array_equal(r.experts.cpu().numpy()[some], ref[1])
