"""Calls that are not given status words return theirs: what the device refused can be told from data."""
import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


I32 = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("form", [dtree.PagedCache, dtree.PagedCache4])
def test_read_back(form):
    """A request longer than the outputs is refused as a whole; a row number out of range is one zero row."""
    cache = form.empty(16, 32, 2, 64, 3, 7)
    cache.table.copy_(torch.arange(16, dtype=torch.int32)[:3, None])
    cache.len.copy_(torch.tensor([20, 200, 0]))
    got = dtree.kv_read(cache, N=100)
    k, v = got
    assert got.status.tolist() == [0, dtree.DT_DEV_BAD_CACHE, 0] and k is got[0] and v is got[1] and len(got) == 2
    rows = torch.tensor([[0, 19], [0, 1], [0, 0]], **I32)
    assert dtree.kv_read(cache, rows=rows).status.tolist() == [0, 0, dtree.DT_DEV_BAD_CACHE]
    mine = torch.zeros(3, **I32)
    assert dtree.kv_read(cache, N=100, status=mine).status is mine


@pytest.mark.parametrize("M", [2, 3000])
def test_head_norms(M):
    """A position past the tables."""
    x = torch.randn((2, M, 4, 64), device="cuda")
    rope = dtree.Rope(torch.ones((M + 5, 32), device="cuda"), torch.zeros((M + 5, 32), device="cuda"))
    got = dtree.qk_norm(x, x, rope=rope, len=torch.tensor([5, 6], **I32))
    q, k = got
    assert got.status.tolist() == [0, dtree.DT_DEV_BAD_CACHE] and q is got[0] and k is got[1]
    mine = torch.zeros(2, **I32)
    assert dtree.qk_norm(x, None, status=mine).status is mine and mine.tolist() == [0, 0]
