"""Tree attention over 4 bits of new rows whose values change their magnitude every 128 rows, under masks that leave
some of those runs out."""
import math

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


def check(cache, q, k, v, sees, rope, scale, out):
    """The reference's bound, and what fp16 loses of a value: of a row, what lies 2^-20 below its largest, or half of
    fp16's smallest number."""
    M = q.shape[1]
    at = torch.arange(M, device="cuda")
    for b in range(q.shape[0]):
        m = int(cache.len[b])
        want, tol = ref4.attention(cache, b, q[b], k[b], v[b], sees.cuda(), at + m, rope, scale)
        lost = (v[b].double().abs().amax(-1).amax(-1) * 2.0 ** -20).clamp(min=2.0 ** -25)
        for h in range(q.shape[2]):
            g = h // (q.shape[2] // cache.Hkv)
            kc = ref4.held(cache.k, cache.k_scale, cache.table[b], m, cache.page)[:, g]
            kn = ref.rotate(k[b].double(), at + m, rope)[:, g]
            s = ref.rotate(q[b].double(), at + m, rope)[:, h] @ torch.cat((kc, kn)).T * scale
            see = torch.cat((torch.ones((M, m), dtype=torch.bool, device="cuda"), sees.cuda()), 1)
            p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
            got = out[b, :, h].double()
            assert torch.isfinite(got).all()
            worst = ((got - want[:, h]).abs() / (tol[:, h] + (p[:, m:] @ lost)[:, None])).max().item()
            assert worst <= 1.0, (b, h, worst)


@pytest.mark.parametrize("M,G,D", [(700, 1, 64), (513, 2, 128), (1025, 1, 128), (260, 4, 64), (120, 1, 128)])
@pytest.mark.parametrize("sizes", [(0, -30, 20, -5, 45, -12, 3), (60, -7, -50, 14, -20), (-9, -8, -4, 15, 0), (-25, 88, 14, -3)])
@pytest.mark.parametrize("lens", [[300, 0], [4000, 77]])
def test_runs_of_other_magnitudes(M, G, D, sizes, lens):
    g = torch.Generator().manual_seed(M + sizes[0])
    cache = make_cache(lens, 64, 2, D, 6)
    x = torch.randn((2, M, 2 * G + 4, D), generator=g)
    x[:, :, 2 * G + 2:] *= torch.exp2(torch.tensor([float(sizes[i // 128 % len(sizes)]) for i in range(M)]))[None, :, None, None]
    x = x.to(torch.bfloat16).cuda()
    q, k, v = x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:]
    n, m = torch.arange(M)[:, None], torch.arange(M)[None]
    sees = (m <= n) & ((n // 3 >> (m // 128 % 4)) & 1 > 0) | (m == n)
    mask = ref.pack(sees, M)[None].expand(2, -1, -1).contiguous().cuda()
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    tabs = ref.rope_tables(6000, D, "cuda") if M % 2 else None
    rope = dtree.Rope(*tabs) if tabs else None
    out = dtree.tree_attention(cache, q, k, v, mask=mask, rope=rope, status=status)
    again = dtree.tree_attention(cache, q, k, v, mask=mask, rope=rope, status=status)
    assert (status == 0).all() and torch.equal(out, again)
    check(cache, q, k, v, sees, (*tabs, False) if tabs else None, 1.0 / math.sqrt(D), out)


@pytest.mark.parametrize("M,G", [(16, 1), (5, 3), (2, 8), (1, 7)])
@pytest.mark.parametrize("size", [-40, -20, -9, 0, 14, 16, 60])
def test_few_rows_of_any_magnitude(M, G, size):
    g = torch.Generator().manual_seed(M + size)
    cache = make_cache([300, 0, 77], 32, 2, 128, 6)
    x = torch.randn((3, M, 2 * G + 4, 128), generator=g)
    x[:, :, 2 * G + 2:] *= 2.0 ** size * torch.exp2(-(torch.arange(M) % 3).float() * 5)[None, :, None, None]
    x = x.to(torch.bfloat16).cuda()
    q, k, v = x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:]
    tabs = ref.rope_tables(600, 64, "cuda")
    sees = torch.ones((M, M), dtype=torch.bool).tril()
    for rope in (None, tabs):
        out = dtree.tree_attention(cache, q, k, v, rope=dtree.Rope(*rope) if rope else None)
        check(cache, q, k, v, sees, (*rope, False) if rope else None, 1.0 / math.sqrt(128), out)
