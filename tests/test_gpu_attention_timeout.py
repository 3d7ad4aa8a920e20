"""The timeout path of tree attention on the tensor cores: a wait that runs out stops every role of the
kernel, sets DT_DEV_TIMEOUT and leaves the context usable (dt_test_wait_fault makes one run out on a
barrier that nothing completes; no copy or product is skipped by it)."""
import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_attention import make_cache

pytestmark = pytest.mark.gpu

BUDGET = 2_000_000  # SM clock cycles, about a millisecond


@pytest.fixture(autouse=True)
def _hook_off(cuda_lib):
    dtree.set_test_wait_fault(())
    yield
    dtree.set_test_wait_fault(())


# lengths, rows, query heads per key head, D: one short unit; both slots with other rows; slots that share
# rows; long units in many parts that are joined; more requests than a warp looks at
@pytest.mark.parametrize("lens,M,G,D", [([0], 17, 1, 64), ([300, 5], 257, 2, 128), ([700], 40, 2, 64), ([9000, 3], 40, 4, 128),
                                        ([5000, 40], 300, 1, 128), ([50] * 40, 20, 2, 64)])
def test_timeout_stops_every_role(lens, M, G, D):
    B = len(lens)
    cache = make_cache(lens, 32, 2, D, 7)
    x = torch.randn((B, M, 2 * G + 4, D), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
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


def test_hook_leaves_small_calls_alone():
    """Up to 16 rows per key head: another kernel, without such waits."""
    cache = make_cache([100], 16, 1, 64, 3)
    x = torch.randn((1, 4, 4, 64), device="cuda").to(torch.bfloat16)
    want = dtree.tree_attention(cache, x[:, :, :2], x[:, :, 2:3], x[:, :, 3:])
    dtree.set_test_wait_fault(("attention",), BUDGET)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(dtree.tree_attention(cache, x[:, :, :2], x[:, :, 2:3], x[:, :, 3:], status=st), want) and not st.any()
