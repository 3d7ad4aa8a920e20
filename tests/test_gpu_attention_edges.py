"""Tree attention where its scales could fail: zeros, tiny and spread scales, large neighbours
behind masks, and divisions of the work that small batches do not reach."""
import math

import pytest
import torch

import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_attention import make_cache, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def compare(cache, q, k, v, out, sees=None, scale=None, rows=None):
    """out against the definition (a chain when sees is None); rows: bool [M], the rows to compare."""
    B, M = q.shape[:2]
    sees = torch.ones((M, M), dtype=torch.bool).tril() if sees is None else sees
    at = torch.arange(M, device="cuda")
    rows = torch.ones(M, dtype=torch.bool, device="cuda") if rows is None else rows
    scale = 1.0 / math.sqrt(cache.D) if scale is None else scale
    for b in range(B):
        want, tol = ref.attention(cache, b, q[b], k[b], v[b], sees.cuda(), at, None, scale)
        # bf16 rounds to half a step, 2^-8 of a number just above a power of two: twice what the bound holds for it
        tol = tol + 2.0 ** -9 * want.abs()
        got = out[b].double()
        assert torch.isfinite(got[rows]).all(), (b, int(cache.len[b]))
        worst = ((got - want).abs() / tol)[rows].max().item()
        assert worst <= 1.0, (b, int(cache.len[b]), worst)


SHAPES = [(1, 1), (1, 4), (16, 1), (17, 1), (5, 8), (300, 1)]  # rows, query heads per key head


@pytest.mark.parametrize("M,G", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("zero", ["queries", "keys", "both"])
def test_zero_queries_and_keys(M, G, D, zero):
    """Equal scores: the mean of the values that a row sees.  Cached zero keys as append writes them."""
    lens, Hkv, page = [0, 5, 130, 256], 2, 16
    B, g = len(lens), torch.Generator(device="cuda").manual_seed(M + G)
    cache = dtree.PagedCache.empty(B * 17, page, Hkv, D, B, 17)
    cache.table.copy_(torch.arange(B * 17).view(B, 17))
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    on = 0.0 if zero != "queries" else 1.0
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dtree.kv_append(cache, rnd(B, max(lens), Hkv, D) * on, rnd(B, max(lens), Hkv, D), count=n)
    cache.len.copy_(n)
    q, k, v = rnd(B, M, G * Hkv, D) * (1.0 - on if zero == "keys" else 0.0), rnd(B, M, Hkv, D) * on, rnd(B, M, Hkv, D)
    compare(cache, q, k, v, dtree.tree_attention(cache, q, k, v))


@pytest.mark.parametrize("M,G", SHAPES)
@pytest.mark.parametrize("key_scale,scale", [(2.0 ** -120, None), (2.0 ** -126, None), (2.0 ** -6, 1e-37)])
def test_factors_that_underflow(M, G, key_scale, scale):
    """Tiny cached key scales, or a tiny softmax scale: scores of nearly zero."""
    cache = make_cache([37, 130], 16, 2, 64, 3)
    cache.k_scale[cache.k_scale.isfinite()] = key_scale
    x = torch.randn((2, M, 2 * G + 4, 64), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    x[:, :, :2 * G] *= 2.0 ** -30
    q, k, v = x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:]
    compare(cache, q, k, v, dtree.tree_attention(cache, q, k, v, scale=scale), scale=scale)


@pytest.mark.parametrize("M,G", SHAPES)
def test_queries_near_the_largest_number(M, G):
    """Queries of 2^127 and more over keys as small: ordinary scores.  No new row is seen."""
    cache = make_cache([37, 130], 16, 2, 64, 3)
    cache.k_scale[cache.k_scale.isfinite()] = 2.0 ** -126
    x = torch.randn((2, M, 2 * G + 4, 64), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    x[:, :, :2 * G, 7] = 2.5e38
    q, k, v = x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:]
    mask = torch.zeros((2, M, (M + 31) // 32), dtype=torch.int32, device="cuda")
    compare(cache, q, k, v, dtree.tree_attention(cache, q, k, v, mask=mask), torch.zeros((M, M), dtype=torch.bool))
