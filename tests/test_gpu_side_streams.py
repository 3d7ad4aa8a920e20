"""Calls on a stream that is not the current one, with nothing brought by the caller: what they
allocate and fill for themselves belongs to the stream that they run on."""
import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_attention import make_cache

pytestmark = pytest.mark.gpu

CLOCKS = 200_000_000  # some 100 ms


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def calls():
    """name: a call that takes a stream and returns its outputs."""
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = make_cache([700, 40], 32, 2, 128, 21)
    x = torch.randn((2, 40, 12, 128), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :, :8], x[:, :, 8:10], x[:, :, 10:]
    logits = torch.randn((2, 40, 5003), generator=g, device="cuda")
    tok = torch.randint(0, 5003, (2, 40), generator=g, device="cuda").to(torch.int32)
    new = make_cache([5, 1], 32, 2, 128, 22)
    new.table.fill_(-1)  # no page to append to
    p = dtree.Params(mode="ddtree", batch=1, L=4, V=5003, dtype="f32", K=4, B=8)
    tree = dtree.TreeBuffers.for_params(p)
    dtree.build_tree(p, logits[:1, :4].contiguous(), tree)
    target = logits[:1, :tree.max_nodes].contiguous()

    def logprobs(stream):
        o = dtree.token_logprobs(logits, tok, top=7, stream=stream)
        return [o.logprob, o.entropy, o.rank, o.top_id, o.top_logprob]

    return {"attention of trees": lambda s: [dtree.tree_attention(cache, q, k, v, stream=s)],
            "attention of tokens": lambda s: [dtree.tree_attention(cache, q[:, :1], k[:, :1], v[:, :1], stream=s)],
            "append": lambda s: [dtree.kv_append(new, k, v, stream=s)],
            "logprobs": logprobs,
            "verify": lambda s: list(dtree.verify(tree, target, stream=s))}


NAMES = ["attention of trees", "attention of tokens", "append", "logprobs", "verify"]


@pytest.mark.parametrize("name", NAMES)
def test_while_the_current_stream_is_busy(name):
    call = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(CLOCKS)
    got = call(side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # nothing waited for the current stream
    torch.cuda.synchronize()
    assert len(want) == len(got) and all(torch.equal(a, b) for a, b in zip(want, got))
    if name == "append":
        assert got[0].tolist() == [dtree.DT_DEV_BAD_CACHE] * 2


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_holds_is_not_handed_out(name):
    """The call is queued on the side stream; meanwhile the current stream fills all memory that is free."""
    call = calls()[name]
    want = call(None)
    del want
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CLOCKS)
    got = call(side)
    others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in [1 << 26, 1 << 25, 1 << 24] + [512] * 200]
    torch.cuda.current_stream().synchronize()
    assert not side.query()
    side.synchronize()
    assert all(bool((t == 7).all()) for t in others)
    assert all(torch.equal(a, b) for a, b in zip(call(None), got))
