"""Log-probabilities of rows with mask constants and logits far from zero, against 64 bits."""
import math

import pytest
import torch

from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu

V = 151936


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def check(x, tok, top, o):
    """x [1, M, V], the first rows of a call's logits.  The bound goes by the row's largest logit: what
    lies far below it has no weight.  lse = largest + log(sum): its product with the two constants
    log2(e) and ln(2), its own rounding and the subtraction's, each within 2^-24 of what it is applied
    to; the sum's terms within 2^-21."""
    M = x.shape[1]
    y, t = x.double(), tok[:, :M].long()[..., None]
    lp = torch.log_softmax(y, -1)
    size = y.amax(-1).abs()
    want = lp.gather(-1, t)[..., 0]
    got = o.logprob[:, :M].double()
    close = (got - want).abs() <= 4e-6 + 2.0 ** -22 * (size + want.abs())
    assert (close | (got == want.float().double())).all(), (got, want)  # -inf for what fp32 does not hold
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    assert ((o.entropy[:, :M].double() - ent).abs() <= 4e-6 * (math.log(x.shape[2]) + 4)).all()
    at = y.gather(-1, t)
    rank = ((y > at) | ((y == at) & (torch.arange(x.shape[2], device=x.device) < t))).sum(-1)
    assert torch.equal(o.rank[:, :M].long(), rank)
    best, ids = torch.sort(y, dim=-1, descending=True, stable=True)
    assert torch.equal(o.top_id[:, :M].long(), ids[..., :top])
    ref = lp.gather(-1, ids[..., :top])
    close = (o.top_logprob[:, :M].double() - ref).abs() <= 4e-6 + 2.0 ** -22 * (size[..., None] + ref.abs())
    assert (close | (o.top_logprob[:, :M] == ref.float())).all()


def make(rows, dtype, seed, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((1, rows, V), generator=g, device="cuda") * scale).to(dtype), g


KINDS = [(torch.bfloat16, 1), (torch.float32, 2), (torch.bfloat16, 700)]  # a cluster to a row, few threads to a row


@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e30, -1e37, -1e38, -1.7e38, "lowest"])
@pytest.mark.parametrize("where", ["most", "first", "all but one"])
@pytest.mark.parametrize("dtype,rows", KINDS)
def test_mask_constants(dtype, rows, mask, where):
    """Tokens ruled out by a large negative number: no weight, ranks and order as they are."""
    x, g = make(rows, dtype, 3)
    mask = torch.finfo(dtype).min if mask == "lowest" else mask
    off = torch.rand(V, generator=g, device="cuda") < 0.97
    if where != "most":
        off = torch.arange(V, device="cuda") < (150000 if where == "first" else V)
        off[77777] = False
    x[..., off] = mask
    tok = torch.randint(0, V, (1, rows), generator=g, device="cuda").to(torch.int32)
    tok[0, 0] = 77777
    o = dtree.token_logprobs(x, tok, top=4)
    assert torch.isfinite(o.logprob).all() and torch.isfinite(o.entropy).all()
    check(x[:, :5], tok, 4, o)


@pytest.mark.parametrize("level", [-3.0e38, -1e38, -1e30, -1e9, -1e6, 1e6, 1e9, 1e30, 1.0e38, 3.0e38])
@pytest.mark.parametrize("dtype,rows", KINDS)
def test_flat_rows_far_from_zero(dtype, rows, level):
    """Every token at one number, as in a row whose mask leaves nothing: all equally likely."""
    x = torch.full((1, rows, V), level, device="cuda").to(dtype)
    tok = torch.full((1, rows), 5, dtype=torch.int32, device="cuda")
    o = dtree.token_logprobs(x, tok, top=3)
    # below 2^30 the sum's logarithm joins a number of the logits' size; past it there is nothing but ties
    tol = 4e-6 + (2.0 ** -22 * abs(level) if abs(level) < 2.0 ** 29 else 0.0)
    assert ((o.logprob.double() + math.log(V)).abs() <= tol + 2.0 ** -22 * math.log(V)).all()
    assert ((o.entropy.double() - math.log(V)).abs() <= 4e-6 * (math.log(V) + 4)).all()
    assert (o.rank == 5).all() and (o.top_id == torch.arange(3, device="cuda")).all()


@pytest.mark.parametrize("high", [1e7, 3e8, 1e9, 1e12, 1e37, 1.0e38, 1.7e38, 3.3e38])
@pytest.mark.parametrize("dtype,rows", KINDS)
def test_few_tokens_far_above(dtype, rows, high):
    """One, two or three equal tokens far above the rest, with mask constants below."""
    x, g = make(rows, dtype, 4)
    x[..., 1000:60000] = -1e38
    at = torch.tensor([31, 90000, V - 1], device="cuda")
    for r in range(rows):
        x[0, r, at[:1 + r % 3]] = high
    tok = torch.randint(0, V, (1, rows), generator=g, device="cuda").to(torch.int32)
    tok[0, ::2] = 31
    o = dtree.token_logprobs(x, tok, top=4)
    held = x.double().gather(-1, tok.long()[..., None])[..., 0] - high > -3.4e38  # a difference that fp32 holds
    assert torch.isfinite(o.logprob[held]).all() and torch.isfinite(o.entropy).all()
    check(x[:, :6], tok, 4, o)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_levels_around_the_limit(dtype):
    """Largest logits between 2^20 and 2^36 with neighbours one step of the type below."""
    x, g = make(17, dtype, 6)
    for r in range(17):
        top = torch.tensor(2.0 ** (20 + r) * 1.03, device="cuda").to(dtype)
        bits = top.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
        x[0, r, 500:520], x[0, r, 140000:140003] = top, top
        x[0, r, 30000:60000] = (bits - 1).view(dtype)
    tok = torch.full((1, 17), 510, dtype=torch.int32, device="cuda")
    check(x, tok, 4, dtree.token_logprobs(x, tok, top=4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_entropy_of_certain_rows(dtype):
    """Two numbers in one thread's share, the later one up to 30 above the earlier: the reference that
    a thread keeps may lag its largest value, and what that costs the entropy stays below 2e-6 (log and
    quotient of some 6 each, to 2^-23 of it, and an exponential to 2^-22); it is not negative."""
    rows = 400  # a CTA to a row
    x = torch.full((1, rows, V), -math.inf, device="cuda")
    x[0, :, 3] = torch.linspace(-40.0, 10.0, rows, device="cuda")
    x[0, :, 3 + 512 * 8 * 12] = x[0, :, 3] + torch.linspace(0.0, 30.0, rows, device="cuda")
    x = x.to(dtype)
    o = dtree.token_logprobs(x, torch.full((1, rows), 3, dtype=torch.int32, device="cuda"), top=2)
    lp = torch.log_softmax(x.double(), -1)
    ent = -torch.where(lp > -700, lp.exp() * lp, 0.0).sum(-1)
    assert (o.entropy >= 0).all()
    worst = (o.entropy.double() - ent).abs().max().item()
    assert worst <= 2e-6, worst
