"""Tree attention beside rows of another magnitude: what a row does not see does not matter to it."""
import math

import pytest
import torch

import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_attention import make_cache
from test_gpu_attention_edges import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def tree_sees(M):
    return ref.path_bits([-1] + [max(0, i - 2) for i in range(1, M)])


SHAPES = [(6, 1), (6, 2), (16, 1), (70, 4), (200, 1), (300, 2)]  # rows, query heads per key head


@pytest.mark.parametrize("M,G", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [3.0e38, -1.7e38, 1e20, 40000.0])
@pytest.mark.parametrize("size", [1.0, 1e-6])
def test_large_neighbours(M, G, D, value, size):
    """A node with a large finite element among ordinary (or small) ones: the rows that do not see it are
    as exact as ever; with values that fp16 holds beside each other those that do are too."""
    cache = make_cache([37], 16, 1, D, 4)
    x = torch.randn((1, M, G + 2, D), generator=torch.Generator().manual_seed(M)).cuda()
    x[:, :, G:] *= size
    x = x.to(torch.bfloat16)
    sees, bad = tree_sees(M), 4
    mask = ref.pack(sees, M)[None].cuda()
    for head in (G, G + 1):
        y = x.clone()
        y[0, bad, head, 11] = value
        q, k, v = y[:, :, :G], y[:, :, G:G + 1], y[:, :, G + 1:]
        out = dtree.tree_attention(cache, q, k, v, mask=mask)
        every = head == G + 1 and abs(value) <= 40000.0
        compare(cache, q, k, v, out, sees, rows=None if every else ~sees[:, bad].cuda())


@pytest.mark.parametrize("M,G", SHAPES)
def test_large_later_rows_of_a_chain(M, G):
    """The rows ahead of a large one, and of a whole run of rows with magnitudes of their own."""
    cache = make_cache([130], 32, 1, 128, 5)
    x = torch.randn((1, M, G + 2, 128), generator=torch.Generator().manual_seed(M)).cuda()
    x[:, M // 2:, G:] *= torch.exp2(torch.arange(M - M // 2, device="cuda") % 97 + 20.0)[None, :, None, None]
    x = x.to(torch.bfloat16)
    q, k, v = x[:, :, :G], x[:, :, G:G + 1], x[:, :, G + 1:]
    rows = torch.arange(M, device="cuda") < M // 2
    compare(cache, q, k, v, dtree.tree_attention(cache, q, k, v), rows=rows)


@pytest.mark.parametrize("M,G", SHAPES)
def test_rows_of_many_magnitudes(M, G):
    """Each row sees itself alone, over an empty cache: its output is its value, at any magnitude
    from 2^-40 to 2^126, zero rows among them."""
    cache = dtree.PagedCache.empty(1, 16, 1, 128, 1, 1)
    x = torch.randn((1, M, G + 2, 128), generator=torch.Generator().manual_seed(M))
    e = (torch.arange(M) * 37 % 164 - 40).float()
    x[:, :, G + 1] *= torch.exp2(e)[None, :, None] * 0.25
    x[:, 3::7, G + 1] = 0.0
    x = x.to(torch.bfloat16).cuda()
    sees = torch.eye(M, dtype=torch.bool)
    mask = ref.pack(sees, M)[None].cuda()
    q, k, v = x[:, :, :G], x[:, :, G:G + 1], x[:, :, G + 1:]
    out = dtree.tree_attention(cache, q, k, v, mask=mask)
    want = v.expand(1, M, G, 128).double()
    # fp16 of the scaled value: 11 bits of it, or 2^-25 of a largest element in [1, 2) or above; then bf16
    tol = want.abs() * (2.0 ** -11 + 2.0 ** -9) * 1.01 + want.abs().amax(-1, keepdim=True) * 2.0 ** -24
    assert ((out.double() - want).abs() <= tol).all()
