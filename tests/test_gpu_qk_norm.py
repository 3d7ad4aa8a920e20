"""Norms of query and key heads with their rotation against the definition in 64 bits."""
import math

import pytest
import torch

import target4_ref as ref4
import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


I32 = dict(dtype=torch.int32, device="cuda")


def run(B, M, Hq, Hk, D, dtype, rot=None, interleaved=False, heads=False, lens=None, n_nodes=None, tree=False, weights=True,
        inplace=False, size=1.0, eps=1e-6, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((B, M, Hq + 2 * Hk, D), generator=g) * size).to(dtype).cuda()
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    qw, kw = ((1 + 0.3 * torch.randn((H, D) if heads else (D,), generator=g)).cuda() if weights else None for H in (Hq, Hk))
    rot = D if rot is None else rot
    lens = [0] * B if lens is None else lens
    n_nodes = [M] * B if n_nodes is None else n_nodes
    pos = torch.randint(0, 17, (B, M), generator=g).to(torch.int32) if tree else None
    tabs = ref.rope_tables(max(lens) + max(M, 17) + 1, rot, "cuda") if rot else None
    before = x.clone()
    status = torch.zeros(B, **I32)
    qo, ko = (q, k) if inplace else (torch.full((B, M, Hq, D), 5.0, dtype=dtype, device="cuda"),
                                     torch.full((B, M, Hk, D), 5.0, dtype=dtype, device="cuda"))
    got = dtree.qk_norm(q, k if Hk else None, qw, kw if Hk else None, eps=eps, rope=dtree.Rope(*tabs, interleaved) if rot else None,
                        len=torch.tensor(lens, **I32), pos=None if pos is None else pos.cuda(),
                        n_nodes=torch.tensor(n_nodes, **I32), q_out=qo, k_out=ko if Hk else None, status=status)
    assert (status == 0).all() and got[0] is qo and (Hk == 0 or got[1] is ko)
    for b in range(B):
        n = n_nodes[b]
        at = (lens[b] + (pos[b, :n].long() if tree else torch.arange(n))).cuda()
        for y, w, o, c in ((before[b, :n, :Hq], qw, qo, 0), (before[b, :n, Hq:Hq + Hk], kw, ko, Hq)):
            if not o.shape[2]:
                continue
            want, tol = ref4.normed(y, w, eps, at, (*tabs, interleaved) if rot else None, dtype)
            worst = ((o[b, :n].double() - want).abs() / tol).max().item() if n else 0.0
            assert worst <= 1.0, (b, n, worst)
            rest = before[b, n:, c:c + o.shape[2]] if inplace else torch.full_like(o[b, n:], 5.0)
            assert torch.equal(o[b, n:], rest)
    assert torch.equal(x[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    if not inplace:
        assert torch.equal(x, before)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (48, False), (64, False), (64, True), (None, False), (None, True)])
def test_rotations(D, dtype, rot, interleaved):
    run(3, 9, 6, 2, D, dtype, rot, interleaved, lens=[0, 77, 1000], n_nodes=[9, 4, 0], seed=D)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (3, 0), (7, 1), (14, 2), (16, 16), (40, 8), (64, 8)])
@pytest.mark.parametrize("heads", [False, True])
def test_head_layouts(Hq, Hk, heads):
    run(2, 5, Hq, Hk, 128, torch.bfloat16, heads=heads, tree=True, lens=[3, 0], seed=Hq)
    run(2, 5, Hq, Hk, 64, torch.float32, heads=heads, tree=True, lens=[3, 0], seed=Hq, weights=not heads)


@pytest.mark.parametrize("M", [1, 17, 700, 4100])
def test_lengths(M):
    run(2, M, 6, 2, 128, torch.bfloat16, lens=[5, 0], n_nodes=[M, M // 2], seed=M)
    run(1, M, 3, 1, 64, torch.float32, seed=M)


def test_in_place():
    run(3, 33, 6, 2, 128, torch.bfloat16, lens=[0, 4, 9], n_nodes=[33, 1, 20], inplace=True)
    run(3, 33, 6, 2, 64, torch.float32, rot=32, lens=[0, 4, 9], n_nodes=[33, 1, 20], inplace=True)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-5, 1e4, 1e18, 1e25, 1e37])
def test_magnitudes(size):
    """Rows of zeros, below eps, and with squares past fp32's range."""
    run(2, 7, 5, 1, 128, torch.float32, size=size, seed=3)
    run(2, 7, 5, 1, 64, torch.bfloat16, size=size, eps=0.1, seed=4)


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -110])
@pytest.mark.parametrize("size", [1e-14, 1e-16, 1e-19, 1e-25, 1e-38, 1e-43])
def test_squares_below_the_range(size, eps):
    """Heads whose squares, and eps, are below what fp32 holds, denormal numbers among them."""
    run(2, 7, 5, 1, 128, torch.float32, size=size, eps=eps, seed=5)
    run(2, 9, 7, 3, 64, torch.float32, size=size, eps=eps, heads=True, inplace=True, seed=6)
    run(1, 5100, 9, 2, 64, torch.float32, size=size, eps=eps, seed=8)  # whole tokens to a warp
    if size > 1e-39:  # numbers of bf16
        run(2, 7, 5, 1, 64, torch.bfloat16, size=size, eps=eps, tree=True, seed=7)


def test_values_that_are_not_finite_stay_in_their_head():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((1, 3, 4, 128), generator=g).to(torch.bfloat16).cuda()
    y = x.clone()
    y[0, 1, 2, 5], y[0, 2, 0, 3] = math.inf, math.nan
    a, _ = dtree.qk_norm(x, None)
    b, _ = dtree.qk_norm(y, None)
    bad = torch.zeros((1, 3, 4, 128), dtype=torch.bool, device="cuda")
    bad[0, 1, 2, 5] = bad[0, 2, 0] = True
    assert torch.equal(torch.isnan(b), bad)
    same = torch.ones((1, 3, 4), dtype=torch.bool, device="cuda")
    same[0, 1, 2] = same[0, 2, 0] = False
    assert torch.equal(a[same], b[same])
    assert (b[0, 1, 2][~bad[0, 1, 2]] == 0).all()


def test_positions_and_counts_out_of_range():
    """Flagged, and left alone."""
    x = torch.randn((4, 5, 2, 64), device="cuda")
    cos, sin = ref.rope_tables(20, 64, "cuda")
    lens, pos = torch.tensor([0, 18, -3, 0], **I32), torch.arange(5, **I32).repeat(4, 1)
    n = torch.tensor([5, 5, 5, 6], **I32)
    status, out = torch.zeros(4, **I32), torch.full_like(x, 9.0)
    dtree.qk_norm(x, None, rope=dtree.Rope(cos, sin), len=lens, pos=pos, n_nodes=n, q_out=out, status=status)
    bad = dtree.DT_DEV_BAD_CACHE
    assert status.tolist() == [0, bad, bad, bad]
    left = (out == 9.0).all(-1).all(-1)
    assert left.tolist() == [[False] * 5, [False] * 2 + [True] * 3, [True] * 3 + [False] * 2, [True] * 5]


def test_refusals():
    x = torch.zeros((1, 2, 4, 64), device="cuda")
    with pytest.raises(TypeError):
        dtree.qk_norm(x, x.bfloat16())
    with pytest.raises(TypeError):
        dtree.qk_norm(x.half(), None)
    with pytest.raises(ValueError):
        dtree.qk_norm(x, None, q_weight=torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        dtree.qk_norm(x, None, k_out=x)
    with pytest.raises(ValueError):
        dtree.qk_norm(x, None, q_out=x[:, :, :2])
    with pytest.raises(ValueError):
        dtree.qk_norm(x, None, len=torch.zeros(0, **I32))
    for kw in (dict(eps=-1.0), dict(eps=math.inf)):
        with pytest.raises(dtree.DtError):
            dtree.qk_norm(x, None, **kw)
    with pytest.raises(dtree.DtError):
        dtree.qk_norm(torch.zeros((1, 2, 4, 32), device="cuda"), None)
    cos, sin = ref.rope_tables(8, 128, "cuda")
    with pytest.raises(dtree.DtError):
        dtree.qk_norm(x, None, rope=dtree.Rope(cos, sin))
