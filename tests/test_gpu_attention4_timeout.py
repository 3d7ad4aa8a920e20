"""The timeout path of tree attention on the tensor cores over 4 bits, whose softmax has loops of its own: a wait that
runs out stops every role, sets DT_DEV_TIMEOUT and leaves the context usable."""
import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_attention4 import make_cache

pytestmark = pytest.mark.gpu

BUDGET = 2_000_000  # SM clock cycles, about a millisecond


@pytest.fixture(autouse=True)
def _hook_off(cuda_lib):
    dtree.set_test_wait_fault(())
    yield
    dtree.set_test_wait_fault(())


# one short unit; both slots with other rows; slots that share rows; long units in many parts; many requests;
# size: of the new values, which then have a scale for their tile, or one for each row
@pytest.mark.parametrize("lens,M,G,D,size", [([0], 17, 1, 64, 0), ([300, 5], 257, 2, 128, -20), ([700], 40, 2, 64, 30),
                                             ([9000, 3], 40, 4, 128, 0), ([5000, 40], 300, 1, 128, 30), ([50] * 40, 20, 2, 64, -20)])
def test_timeout_stops_every_role(lens, M, G, D, size):
    B = len(lens)
    cache = make_cache(lens, 32, 2, D, 7)
    x = torch.randn((B, M, 2 * G + 4, D), generator=torch.Generator().manual_seed(M))
    x[:, ::2, 2 * G + 2:] *= 2.0 ** size
    x = x.to(torch.bfloat16).cuda()
    q, k, v = x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:]
    ws, st = dtree.attention_workspace(cache, M, 2 * G), torch.zeros(B, dtype=torch.int32, device="cuda")
    want = dtree.tree_attention(cache, q, k, v, workspace=ws, status=st)
    assert not st.any()
    dtree.set_test_wait_fault(("attention",), BUDGET)
    dtree.tree_attention(cache, q, k, v, workspace=ws, status=st)
    torch.cuda.synchronize()
    assert all(s & dtree.DT_DEV_TIMEOUT for s in st.tolist())
    # hook off, workspace zeroed: the same call on the same context is as it was
    dtree.set_test_wait_fault(())
    ws[0].zero_()
    st.zero_()
    again = dtree.tree_attention(cache, q, k, v, workspace=ws, status=st)
    assert not st.any() and torch.equal(again, want)
