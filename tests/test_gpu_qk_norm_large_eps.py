"""Head norms with an eps near the end of fp32's range: one rule, whatever the number of rows."""
import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_qk_norm import run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


@pytest.mark.parametrize("eps", [2.0 ** 120, 2.0 ** 124, 2.0 ** 126, 3e38])
@pytest.mark.parametrize("size", [1.0, 1e10, 1e18, 1e19, 1e25])
def test_large_eps(eps, size):
    """Heads far below the root of eps, near it and far above: a few rows, and whole tokens to a warp."""
    for M in (7, 5100):
        run(1, M, 9, 2, 64, torch.float32, size=size, eps=eps, seed=8)
        run(1, M, 5, 1, 128, torch.bfloat16, size=size, eps=eps, seed=9, inplace=True)


def test_the_same_head_in_calls_of_any_length():
    x = torch.randn((1, 5100, 8, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 1e18
    for eps in (1e-6, 1e30, 1e38):
        many, few = dtree.qk_norm(x, None, eps=eps)[0], dtree.qk_norm(x[:, :3], None, eps=eps)[0]
        assert torch.allclose(many[:, :3], few, rtol=2.0 ** -20, atol=0.0)
