"""Tree attention over caches whose value scales lie far apart."""
import math

import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_attention import make_cache
from test_gpu_attention_edges import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


@pytest.mark.parametrize("M,G", [(1, 1), (3, 4), (20, 2), (300, 1)])
@pytest.mark.parametrize("low,high", [(-48, 0), (-48, 48), (0, 96), (-100, -20), (24, 120), (-100, -60)])
def test_value_scales_far_apart(M, G, low, high):
    """Pages with large and with small values beside each other, up to 2^96: each keeps its weight in the sum."""
    cache = make_cache([300, 45], 16, 2, 128, 6)
    some = torch.rand(cache.v_scale.shape, generator=torch.Generator().manual_seed(3)).cuda() < 0.5
    e = torch.where(some, float(low), float(high))
    cache.v_scale.copy_(torch.where(cache.v_scale.isfinite(), torch.exp2(e), math.nan))
    x = torch.randn((2, M, 2 * G + 4, 128), generator=torch.Generator().manual_seed(M)).cuda()
    x[:, :, 2 * G + 2:] *= 2.0 ** max(low, -50)
    x = x.to(torch.bfloat16)
    q, k, v = x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:]
    compare(cache, q, k, v, dtree.tree_attention(cache, q, k, v))


@pytest.mark.parametrize("M,G", [(1, 1), (3, 4), (20, 2)])
def test_scales_that_are_no_powers_of_two(M, G):
    cache = make_cache([300, 45], 16, 2, 64, 6)
    g = torch.Generator().manual_seed(4)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_(1.0 + torch.rand(s.shape, generator=g).cuda())
    x = torch.randn((2, M, 2 * G + 4, 64), generator=g).to(torch.bfloat16).cuda()
    q, k, v = x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:]
    compare(cache, q, k, v, dtree.tree_attention(cache, q, k, v))
