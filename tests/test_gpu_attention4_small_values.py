"""Tree attention over 4 bits of new rows with small values whose weights lie far below a cached token's."""
import math

import pytest
import torch

import target4_ref as ref4
from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def weighted(cache, b, s, v, sees):
    """Outputs [n, Hq, D] of rows whose scores [n, m + n] are alike for all heads, and a bound on the kernel's error.

    Queries and keys are exact in fp16 here, and so are their products.  A score times its factor, both
    rounded to fp32, is off by a few times 2^-24 of at most 16 octaves: a weight by 2^-17 of itself at most.  It is
    rounded to fp16 (half a step, 2^-11), sums of fp32 take 2^-23 per step, the output half a step of bf16.
    A new value below 2^-8 may lose what lies under half of fp16's smallest number, 2^-25."""
    n, m = v.shape[0], int(cache.len[b])
    vc = ref4.held(cache.v, cache.v_scale, cache.table[b], m, cache.page)
    see = torch.cat((torch.ones((n, m), dtype=torch.bool, device=v.device), sees), 1)
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
    out, a = (torch.stack([p @ torch.cat((vc[:, h], w[:, h])) for h in range(cache.Hkv)], 1)
              for vc, w in ((vc, v.double()), (vc.abs(), v.double().abs())))
    lost = p[:, m:].sum(-1)[:, None, None] * 2.0 ** -25
    return out, 2.0 ** -8 * 1.01 * out.abs() + a * 1.01 * (2.0 ** -11 + 2.0 ** -16 + (m + n) * 2.0 ** -23) + lost


@pytest.mark.parametrize("M,G,D", [(40, 1, 128), (40, 1, 64), (300, 2, 64), (300, 1, 128), (3, 8, 128), (8, 2, 128), (16, 1, 64), (2, 3, 128)])
@pytest.mark.parametrize("size", [-5, -9, -14, -20])
@pytest.mark.parametrize("turn", [False, True])
def test_small_values_beside_a_token_that_leads(M, G, D, size, turn):
    """A first token ahead of all others by 10 to 16 octaves, whose value is zero: what is left of the output is the
    others' values, each with a weight of its own.  turn: by angles of zero, so that rows are as they were."""
    g = torch.Generator().manual_seed(M + size)
    lens, page, Hkv = [200, 1, 129], 16, 2
    x = torch.zeros((2, 40, Hkv, page, D))
    x[1] = torch.randn(x[1].shape, generator=g) * 2.0 ** size
    lead = [6.75, 7.5, 9.0, 9.75, 10.5, 11.25]          # numbers of the cache's format: six times a scale
    key = torch.randint(-8, 9, (40, Hkv, page), generator=g) / 16.0
    table = torch.randperm(40, generator=g)[:39].view(3, 13).to(torch.int32)
    top = [lead[(M + i) % 6] for i in range(3)]
    for b in range(3):
        x[0, int(table[b, 0]), :, 0, 0] = top[b]
        x[1, int(table[b, 0]), :, 0] = 0.0
    x[0, ..., 16] = key                                  # other tokens' keys: one element, exact in the format
    for b in range(3):
        x[0, int(table[b, 0]), :, 0, 16] = 0.0
    codes, scales = ref4.quantised(x.cuda().double())
    cache = dtree.PagedCache4(codes[0], codes[1], scales[0], scales[1], table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    held = ref4.values4(codes[0], scales[0])
    assert torch.equal(held[..., 0], x[0, ..., 0].cuda().double())
    q = torch.zeros((3, M, Hkv * G, D))
    q[..., 0], q[..., 16] = 4.0, 4.0
    k = torch.zeros((3, M, Hkv, D))
    k[..., 0] = (torch.arange(M) * 37 % 64 - 32)[None, :, None] / 64.0
    v = torch.randn((3, M, Hkv, D), generator=g) * 2.0 ** size
    q, k, v = (t.to(torch.bfloat16).cuda() for t in (q, k, v))
    rope = dtree.Rope(torch.ones((600, D // 2), device="cuda"), torch.zeros((600, D // 2), device="cuda")) if turn else None
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = dtree.tree_attention(cache, q, k, v, rope=rope, scale=0.25, status=status)
    assert (status == 0).all()
    sees = torch.ones((M, M), dtype=torch.bool, device="cuda").tril()
    for b in range(3):
        kc = ref4.held(cache.k, cache.k_scale, cache.table[b], lens[b], page)
        # the heads' scores differ in their cached keys
        for h in range(Hkv):
            s = torch.cat((kc[:, h, 0] + kc[:, h, 16], k[b, :, h, 0].double()))[None].expand(M, -1)
            want, tol = weighted(cache, b, s, v[b], sees)
            got = out[b, :, h * G:(h + 1) * G].double()
            worst = ((got - want[:, h:h + 1]).abs() / tol[:, h:h + 1]).max().item()
            assert worst <= 1.0, (b, h, worst)
