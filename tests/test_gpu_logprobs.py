"""Log-probabilities, ranks, entropies and alternatives against their definitions in 64 bits."""
import math

import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def check(x, rows, tokens, top, o):
    """x [B, M, V]; entries with a negative row are padding."""
    B, M, V = x.shape
    N = tokens.shape[1]
    pick = torch.arange(N, device=x.device).expand(B, N) if rows is None else rows.long()
    used, named = pick >= 0, (pick >= 0) & (tokens >= 0)
    y = x.double().gather(1, pick.clamp(min=0)[..., None].expand(B, N, V))
    lp = torch.log_softmax(y, -1)
    t = tokens.long().clamp(min=0)[..., None]
    want = torch.where(named, lp.gather(-1, t)[..., 0], 0.0)
    # fp32 sums of V positive terms in parts of a few hundred, the terms within 2^-21; then two
    # roundings of a number of the size of the largest logit
    size = torch.where(y.isinf(), 0.0, y).abs().amax(-1)
    tol = 4e-6 + 2.0 ** -22 * size
    assert ((o.logprob.double() - want).abs() <= tol + 2.0 ** -22 * want.abs()).all()
    p = lp.exp()
    ent = torch.where(used, -torch.where(p > 0, p * lp, 0.0).sum(-1), 0.0)
    # the terms p log p add up like p, weighted by at most log V + 4
    assert ((o.entropy.double() - ent).abs() <= 4e-6 * (math.log(V) + 4)).all()
    at = y.gather(-1, t)
    rank = ((y > at) | ((y == at) & (torch.arange(V, device=x.device) < t))).sum(-1)
    assert torch.equal(o.rank.long(), torch.where(named, rank, -1))
    if top:
        best, ids = torch.sort(y, dim=-1, descending=True, stable=True)
        assert torch.equal(o.top_id.long(), torch.where(used[..., None], ids[..., :top], -1))
        got = torch.where(used[..., None], best[..., :top] - torch.logsumexp(y, -1, keepdim=True), 0.0)
        close = (o.top_logprob.double() - got).abs() <= (tol + 2.0 ** -22 * size)[..., None] * 1.0001 + 2.0 ** -22 * got.abs()
        assert (close | (got == o.top_logprob.double())).all()
    else:
        assert o.top_id is None


def logits(shape, dtype, seed, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype), g


@pytest.mark.parametrize("V", [1, 2, 7, 31, 32, 33, 255, 1000, 4099, 32768, 50257, 151936, 151937])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_vocabularies(V, dtype):
    x, g = logits((2, 3, V), dtype, V)
    tok = torch.randint(0, V, (2, 3), generator=g, device="cuda").to(torch.int32)
    top = min(V, 20)
    check(x, None, tok, top, dtree.token_logprobs(x, tok, top=top))


@pytest.mark.parametrize("top", [0, 1, 2, 5, 31, 32])
@pytest.mark.parametrize("B,N", [(1, 1), (3, 17), (40, 5), (1, 330)])
def test_counts(top, B, N):
    x, g = logits((B, N, 5003), torch.bfloat16, top + B)
    tok = torch.randint(0, 5003, (B, N), generator=g, device="cuda").to(torch.int32)
    check(x, None, tok, top, dtree.token_logprobs(x, tok, top=top))


def test_rows_and_padding():
    x, g = logits((3, 40, 9001), torch.float32, 5)
    rows = torch.tensor([[0, 4, 39, -1, -1], [7, -1, -1, -1, -1], [3, 3, 2, 1, 0]], dtype=torch.int32, device="cuda")
    tok = torch.tensor([[1, -1, 9000, -1, 5], [0, 3, -1, -1, 2], [77, 77, -1, 8, 8999]], dtype=torch.int32, device="cuda")
    check(x, rows, tok, 4, dtree.token_logprobs(x, tok, top=4, rows=rows))


def test_rows_and_tokens_out_of_range():
    x, _ = logits((1, 4, 3001), torch.bfloat16, 6)
    rows = torch.tensor([[0, 4, 10 ** 9, 3]], dtype=torch.int32, device="cuda")
    tok = torch.tensor([[3001, 1, 1, 2 ** 30]], dtype=torch.int32, device="cuda")
    o = dtree.token_logprobs(x, tok, top=2, rows=rows)
    assert o.logprob.isnan().all() and (o.rank == -1).all()
    assert o.entropy[0, 1:3].isnan().all() and torch.isfinite(o.entropy[0, [0, 3]]).all()
    assert (o.top_id[0, 1:3] == -1).all() and o.top_logprob[0, 1:3].isnan().all() and (o.top_id[0, [0, 3]] >= 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["flat", "few", "rising", "falling", "ruled out", "one left", "hot", "offset", "zeros"])
def test_hard_rows(dtype, kind):
    """Ties, sorted rows, rows of -inf but for some, a single certain token, a large common offset."""
    V = 20011
    x, g = logits((2, 4, V), torch.float32, 7)
    if kind == "flat":
        x.fill_(1.25)
    elif kind == "few":
        x = x.clamp(-1, 1).round()
    elif kind == "rising":
        x = x.sort(-1).values
    elif kind == "falling":
        x = x.sort(-1, descending=True).values
    elif kind == "ruled out":
        x[..., torch.rand(V, generator=g, device="cuda") < 0.97] = -math.inf
    elif kind == "one left":
        keep = x[..., 12345].clone()
        x.fill_(-math.inf)
        x[..., 12345] = keep
    elif kind == "hot":
        x *= 40
    elif kind == "offset":
        x += 3000
    elif kind == "zeros":
        x = torch.where(x > 0, 0.0, -0.0)
    x = x.to(dtype)
    tok = torch.tensor([[0, 1, 12345, V - 1]] * 2, dtype=torch.int32, device="cuda")
    top = 1 if kind == "one left" else 32
    if kind in ("ruled out", "one left"):  # a token that cannot be drawn: -inf, in the place its id gives it
        tok.fill_(int(x[0, 0].argmax()))
    check(x, None, tok, top, dtree.token_logprobs(x, tok, top=top))


def test_impossible_token():
    x, _ = logits((1, 1, 1000), torch.float32, 8)
    x[..., 10:20] = -math.inf
    o = dtree.token_logprobs(x, torch.tensor([[13]], dtype=torch.int32, device="cuda"))
    assert o.logprob.item() == -math.inf and o.rank.item() == 993 and torch.isfinite(o.entropy).all()


def test_rows_without_a_number():
    """NaN, +inf or no finite value: the figures are not finite, and the call returns."""
    x, _ = logits((1, 3, 4000), torch.float32, 9)
    x[0, 0, 77] = math.nan
    x[0, 1, 78] = math.inf
    x[0, 2] = -math.inf
    o = dtree.token_logprobs(x, torch.tensor([[1, 1, 1]], dtype=torch.int32, device="cuda"), top=32)
    assert not torch.isfinite(o.logprob).any() and not torch.isfinite(o.entropy).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padded_rows_and_odd_starts(dtype):
    """Rows of a wider table, starting off any vector boundary."""
    wide, g = logits((2, 5, 3020), dtype, 10)
    for first in (0, 1, 3, 7):
        x = wide[:, :, first:first + 3001]
        tok = torch.randint(0, 3001, (2, 5), generator=g, device="cuda").to(torch.int32)
        check(x, None, tok, 7, dtree.token_logprobs(x, tok, top=7))


def test_same_bits_every_time_and_other_stream():
    x, g = logits((1, 9, 151936), torch.bfloat16, 11)
    tok = torch.randint(0, 151936, (1, 9), generator=g, device="cuda").to(torch.int32)
    a = dtree.token_logprobs(x, tok, top=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = dtree.alloc_logprobs(1, 9, 9)
    torch.cuda.synchronize()
    dtree.token_logprobs(x, tok, top=9, out=b, stream=side)
    side.synchronize()
    for f in ("logprob", "entropy", "rank", "top_id", "top_logprob"):
        assert torch.equal(getattr(a, f), getattr(b, f))


def test_offsets_past_32_bits():
    x = torch.zeros((1, 15000, 151936), dtype=torch.bfloat16, device="cuda")
    x[0, 14999], _ = logits((151936,), torch.bfloat16, 12)
    rows, tok = (torch.tensor([[v]], dtype=torch.int32, device="cuda") for v in (14999, 151935))
    o = dtree.token_logprobs(x, tok, top=5, rows=rows)
    check(x[:, 14999:], None, tok, 5, o)


def test_refusals():
    x, _ = logits((2, 3, 100), torch.float32, 1)
    tok = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        dtree.token_logprobs(x.half(), tok)
    with pytest.raises(TypeError):
        dtree.token_logprobs(x, tok.long())
    with pytest.raises(ValueError):
        dtree.token_logprobs(x[0], tok)
    with pytest.raises(ValueError):
        dtree.token_logprobs(x.transpose(1, 2), tok)
    with pytest.raises(ValueError):
        dtree.token_logprobs(x, tok, rows=tok[:1])
    with pytest.raises(ValueError):
        dtree.token_logprobs(x, tok, top=2, out=dtree.alloc_logprobs(2, 3))
    with pytest.raises(dtree.DtError):  # more tokens than rows
        dtree.token_logprobs(x[:, :2], tok)
    for top in (-1, 33):
        with pytest.raises(dtree.DtError):
            dtree.token_logprobs(x, tok, top=top)


@pytest.mark.parametrize("level", [-200.0, -4096.0, 512.0])
@pytest.mark.parametrize("ruled_out", [5000, 40000, 150000])
@pytest.mark.parametrize("dtype,rows", [(torch.bfloat16, 1), (torch.float32, 2), (torch.bfloat16, 700)])
def test_far_values_behind_ruled_out_ones(dtype, rows, ruled_out, level):
    """The first tokens ruled out, the others' logits far from zero: a common offset changes nothing."""
    V = 151936
    x, g = logits((1, rows, V), dtype, 5, scale=2.0)
    x = (x.float() + level).to(dtype)
    x[..., :ruled_out] = -math.inf
    tok = torch.randint(ruled_out, V, (1, rows), generator=g, device="cuda").to(torch.int32)
    pick = torch.arange(min(rows, 5), device="cuda")  # the 64-bit check of a few rows
    o = dtree.token_logprobs(x, tok, top=4)
    few = dtree.Logprobs(*(getattr(o, f)[:, pick] for f in ("logprob", "entropy", "rank", "top_id", "top_logprob")))
    check(x[:, pick], None, tok[:, pick], 4, few)
    assert torch.isfinite(o.logprob).all()
