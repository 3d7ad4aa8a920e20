"""Tree attention over 4 bits beside new rows with a large element: the other columns are the other tokens'."""
import pytest
import torch

import target4_ref as ref4
import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree
from test_gpu_attention4 import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


SHAPES = [(1, 4), (2, 1), (2, 4), (8, 2), (16, 1), (40, 1), (150, 1), (300, 2)]  # rows, query heads per key head


def compare(cache, b, v, sees, out, G):
    """Against the mean of the values that a row sees: keys are zeros, so that all weights are equal and exact.  Values
    are exact in fp16 down to 2^-20 of a row's largest; sums of fp32 take 2^-23 per step, the output half a step of bf16."""
    n, m = v.shape[0], int(cache.len[b])
    vc = ref4.held(cache.v, cache.v_scale, cache.table[b], m, cache.page)
    w = torch.cat((torch.ones((n, m), dtype=torch.double, device=v.device), sees.double()), 1)
    w = w / w.sum(-1, keepdim=True)
    for h in range(cache.Hkv):
        x = torch.cat((vc[:, h], v[:, h].double()))
        want = w @ x
        low = torch.cat((torch.zeros(m, device=v.device).double(), v[:, h].double().abs().amax(-1) * 2.0 ** -20))
        low = torch.where(low < 2.0 ** -10, low, 0.0)           # of ordinary rows; the large ones hold one element
        tol = 2.0 ** -8 * 1.01 * want.abs() + (w @ x.abs()) * (m + n) * 2.0 ** -22 + (w @ low)[:, None] + 1e-30
        got = out[:, h * G:(h + 1) * G].double()
        assert torch.isfinite(got).all()
        worst = ((got - want[:, None]).abs() / tol[:, None]).max().item()
        assert worst <= 1.0, (b, h, worst)


def make(M, G, D, lens, e, among, seed):
    """Rows of which every seventh holds 2^e in one column and nothing else; among: the others hold
    ordinary values, which rows see too, else nobody sees those others."""
    g = torch.Generator().manual_seed(seed)
    B, Hkv = len(lens), 2
    cache = make_cache(lens, 32, Hkv, D, 3)
    for b, n in enumerate(lens):                       # keys of zeros
        for j in range(n):
            cache.k[int(cache.table[b, j // 32]), :, j % 32] = 0
            cache.k_scale[int(cache.table[b, j // 32]), :, j % 32] = 1
    q, k = torch.randn((B, M, Hkv * G, D), generator=g), torch.zeros((B, M, Hkv, D))
    v = torch.randn((B, M, Hkv, D), generator=g)
    v = torch.where(v.abs() < 2.0 ** -6, torch.full_like(v, 0.25), v)
    large = torch.arange(M) % 7 == M // 2 % 7
    v[:, large] = 0.0
    v[:, large, :, 5] = 2.0 ** e
    if not among:
        v[:, ~large] *= 2.0 ** -3
    sees = torch.ones((M, M), dtype=torch.bool).tril()
    sees[:, int(large.nonzero()[0])] = True            # all rows see a large one
    if not among:
        sees &= large[None]
    return cache, *(t.to(torch.bfloat16).cuda() for t in (q, k, v)), sees


def run(M, G, D, lens, e, among, turn):
    cache, q, k, v, sees = make(M, G, D, lens, e, among, M + e)
    rope = dtree.Rope(torch.ones((8000, D // 2), device="cuda"), torch.zeros((8000, D // 2), device="cuda")) if turn else None
    mask = ref.pack(sees, M)[None].expand(len(lens), -1, -1).contiguous().cuda()
    status = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    out = dtree.tree_attention(cache, q, k, v, mask=mask, rope=rope, status=status)
    assert (status == 0).all()
    for b in range(len(lens)):
        compare(cache, b, v[b], sees.cuda(), out[b], G)


@pytest.mark.parametrize("M,G", SHAPES)
@pytest.mark.parametrize("e", [14, 16, 22, 30, 44, 60, 89])
@pytest.mark.parametrize("turn", [False, True])
def test_cached_tokens_beside_a_large_new_value(M, G, e, turn):
    run(M, G, 128 if M % 4 else 64, [100, 0, 33, 300], e, False, turn)


@pytest.mark.parametrize("M,G", SHAPES[1:])
@pytest.mark.parametrize("e", [14, 16, 22, 30])
@pytest.mark.parametrize("turn", [False, True])
def test_new_rows_beside_a_large_new_value(M, G, e, turn):
    run(M, G, 64 if M % 4 else 128, [100, 0, 33, 300], e, True, turn)


@pytest.mark.parametrize("M,G", [(2, 4), (40, 1), (300, 2)])
@pytest.mark.parametrize("e", [20, 60])
def test_parts_of_long_contexts(M, G, e):
    """Units that several CTAs share: parts with large rows and parts without."""
    run(M, G, 64, [6000], e, False, False)
    run(M, G, 128, [3000, 5, 0], e, e < 31, True)


@pytest.mark.parametrize("M,G", SHAPES)
@pytest.mark.parametrize("e", [91, 104, 127])
def test_near_the_end_of_the_range(M, G, e):
    """Larger values still: the column is right, and nothing becomes infinite or NaN."""
    cache, q, k, v, sees = make(M, G, 128, [100, 0, 300], e, True, e)
    v[..., 5] = v[..., 5].clamp(min=0.0)
    mask = ref.pack(sees, M)[None].expand(3, -1, -1).contiguous().cuda()
    out = dtree.tree_attention(cache, q, k, v, mask=mask)
    assert torch.isfinite(out).all()
    for b, n in enumerate((100, 0, 300)):
        large = (v[b, :, 0, 5] > 2.0 ** 90).double()
        w = sees.cuda().double()
        want = (w @ large) / (n + w.sum(-1)) * 2.0 ** e
        got = out[b, :, :, 5].double()
        assert ((got - want[:, None]).abs() <= want[:, None] * (2.0 ** -8 * 1.01 + (M + n) * 2.0 ** -22)).all()
