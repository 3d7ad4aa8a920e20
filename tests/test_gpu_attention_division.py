"""Tree attention's division of the work: more than 32 requests, units in many parts, wide groups."""
import pytest
import torch

from test_gpu_attention import run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


@pytest.mark.parametrize("B", [33, 70, 200])
@pytest.mark.parametrize("M,G", [(1, 4), (3, 2), (20, 2), (150, 2)])
def test_many_requests(B, M, G):
    """Groups of 32 requests in the shares and in the zeros past n_nodes, empty ones among them."""
    g = torch.Generator().manual_seed(B + M)
    lens = torch.randint(0, 400, (B,), generator=g).tolist()
    n_nodes = torch.randint(0, M + 1, (B,), generator=g).tolist()
    lens[5], n_nodes[B - 1], n_nodes[7] = 0, M, 0
    run(lens, M, G, 1, 64, 16, n_nodes=n_nodes, seed=B)


@pytest.mark.parametrize("M", [1, 16, 17, 300])
def test_units_in_many_parts(M):
    """One request and key head over 65536 tokens: some hundred parts to a unit."""
    run([65536], M, 1, 1, 128 if M < 300 else 64, 128, seed=M)


@pytest.mark.parametrize("M,G", [(1, 128), (3, 128), (1, 100), (9, 33)])
def test_wide_groups(M, G):
    run([200, 1, 0], M, 2 * G, 2, 128, 64, seed=G)


def test_long_chain():
    run([70], 2100, 2, 1, 64, 64, tree=False, seed=2)
