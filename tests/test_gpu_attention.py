"""Tree attention over the paged e4m3 cache against its definition in 64 bits."""
import math

import pytest
import torch

import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def make_cache(lens, page, Hkv, D, seed, extra_pages=2, spread=True):
    """A filled cache: random codes of every exponent, a scale per block over a few octaves, pages in
    no order, and NaN codes wherever no token lies."""
    g = torch.Generator().manual_seed(seed)
    max_pages = max(1, max(-(-n // page) for n in lens)) + 1
    n_pages = len(lens) * max_pages + extra_pages
    x = torch.randn((n_pages, 2, Hkv, page, D), generator=g) * 60
    codes = x.to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.exp2(torch.randint(-9, -4, (2, n_pages, Hkv), generator=g).float())
    if not spread:
        scales.fill_(2.0 ** -6)
    table = torch.randperm(n_pages, generator=g)[:len(lens) * max_pages].view(len(lens), max_pages).to(torch.int32)
    for b, n in enumerate(lens):
        for p in range(max_pages):
            lo = min(page, max(0, n - p * page))
            codes[int(table[b, p]), :, :, lo:] = 0x7F
            if lo == 0:
                scales[:, int(table[b, p])] = math.nan
                if p > -(-n // page):
                    table[b, p] = -1
    codes = codes.cuda()
    return dtree.PagedCache(codes[:, 0].contiguous(), codes[:, 1].contiguous(), scales[0].cuda(), scales[1].cuda(),
                            table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())


def random_tree(n, g, levels=16):
    parents, depth = [-1], [0]
    for i in range(1, n):
        p = int(torch.randint(0, i, (1,), generator=g))
        if depth[p] >= levels:
            p = 0
        parents.append(p)
        depth.append(depth[p] + 1)
    return parents, depth


def check(cache, q, k, v, sees, depth, n_nodes, rope, scale, out):
    """out [B, M, Hq, D] against the reference; rows past n_nodes are zero."""
    for b in range(q.shape[0]):
        n = n_nodes[b]
        at = int(cache.len[b]) + depth[b][:n]
        if n:
            want, tol = ref.attention(cache, b, q[b, :n], k[b, :n], v[b, :n], sees[b].cuda(), at.cuda(), rope, scale)
            err = (out[b, :n].double() - want).abs()
            worst = (err / tol).max().item()
            assert torch.isfinite(out[b, :n]).all() and worst <= 1.0, (b, n, int(cache.len[b]), worst)
        assert (out[b, n:] == 0).all()


def run(lens, M, Hq, Hkv, D, page, tree=True, rot=None, interleaved=False, layout="fused", n_nodes=None, seed=0, hot=1.0):
    g = torch.Generator().manual_seed(seed + 1)
    B = len(lens)
    cache = make_cache(lens, page, Hkv, D, seed)
    H = Hq + 2 * Hkv
    x = torch.randn((B, M, H, D), generator=g) * hot
    if layout == "fused":
        x = x.to(torch.bfloat16).cuda()
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    else:  # heads before rows
        x = x.to(torch.bfloat16).cuda().transpose(1, 2).contiguous().transpose(1, 2)
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    n_nodes = [M] * B if n_nodes is None else n_nodes
    sees, depth, mask, pos = [], [], None, None
    if tree:
        mask = torch.full((B, M, (M + 31) // 32), -1, dtype=torch.int32)
        pos = torch.full((B, M), -7, dtype=torch.int32)
        for b in range(B):
            parents, d = random_tree(max(1, n_nodes[b]), g)
            anc = ref.path_bits(parents)
            mask[b, :len(parents)] = ref.pack(anc, M)[:len(parents)]
            pos[b, :len(parents)] = torch.tensor(d)
            sees.append(anc[:n_nodes[b], :n_nodes[b]])
            depth.append(torch.tensor(d))
        mask, pos = mask.cuda(), pos.cuda()
    else:
        for b in range(B):
            sees.append(torch.ones((n_nodes[b], n_nodes[b]), dtype=torch.bool).tril())
            depth.append(torch.arange(M))
    rot = D if rot is None else rot
    tabs = ref.rope_tables(max(lens) + M + 1, rot, "cuda") if rot else None
    rope = dtree.Rope(tabs[0], tabs[1], interleaved) if rot else None
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(D)
    nn = torch.tensor(n_nodes, dtype=torch.int32).cuda()
    out = dtree.tree_attention(cache, q, k, v, mask=mask, pos=pos, n_nodes=nn, rope=rope, scale=scale, status=status)
    again = dtree.tree_attention(cache, q, k, v, mask=mask, pos=pos, n_nodes=nn, rope=rope, scale=scale, status=status)
    assert (status == 0).all()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time
    check(cache, q, k, v, sees, depth, n_nodes, (tabs[0], tabs[1], interleaved) if rot else None, scale, out)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens_at_every_kind_of_length(page, D):
    lens = [0, 1, 15, 16, 17, page - 1, page, page + 1, 127, 128, 129, 255, 2 * page + 3, 700]
    run(lens, 1, 8, 2, D, page, tree=False)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 12, 16, 17])
def test_head_groups(G):
    run([200, 1], 1, 2 * G, 2, 128, 64, tree=False, seed=G)
    run([130, 33], 6, 2 * G, 2, 128, 32, tree=True, seed=G + 100)


@pytest.mark.parametrize("M", [2, 5, 16, 17, 31, 32, 33, 61, 65, 127, 129])
@pytest.mark.parametrize("D", [64, 128])
def test_trees(M, D):
    run([0, 1, 100, 515], M, 4, 2, D, 64, n_nodes=[M, M - 1, 1, (M + 1) // 2], seed=M)


@pytest.mark.parametrize("M,Hq,Hkv", [(257, 8, 2), (300, 3, 3), (513, 4, 4), (1025, 2, 1)])
def test_large_trees(M, Hq, Hkv):
    run([190, 0], M, Hq, Hkv, 128, 16, n_nodes=[M, M // 2], seed=M)


@pytest.mark.parametrize("M", [1, 7, 64, 130, 400])
def test_chains(M):
    run([0, 77, 300], M, 4, 1, 64, 32, tree=False, n_nodes=[M, M, (M + 1) // 2], seed=M)


@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (64, True), (96, False), (128, True)])
@pytest.mark.parametrize("layout", ["fused", "heads"])
def test_rotations_and_strides(rot, interleaved, layout):
    run([40, 333], 9, 6, 2, 128, 64, rot=rot, interleaved=interleaved, layout=layout, seed=rot)


def test_long_context_is_split():
    run([9000, 5, 3001], 1, 16, 2, 128, 64, tree=False, seed=5)
    run([7001], 40, 16, 2, 128, 128, seed=6)
    run([5000, 12], 257, 4, 1, 64, 64, seed=7)


def test_requests_without_rows():
    run([50, 0, 128], 3, 4, 2, 64, 32, n_nodes=[0, 0, 3], seed=9)


def test_hot_scores():
    """Scores far apart: single keys dominate, the running maximum keeps moving."""
    run([600], 5, 8, 2, 128, 64, hot=12.0, seed=11)
    run([600], 150, 4, 2, 128, 64, hot=12.0, seed=12)


def test_rows_that_see_nothing():
    """An empty cache and a mask without a bit: zeros, not NaN."""
    for M, G in ((3, 2), (90, 4)):
        cache = make_cache([0, 20], 16, 2, 64, 3)
        x = torch.randn((2, M, 2 * G + 4, 64), device="cuda").to(torch.bfloat16)
        mask = torch.zeros((2, M, (M + 31) // 32), dtype=torch.int32, device="cuda")
        out = dtree.tree_attention(cache, x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:], mask=mask)
        assert (out[0] == 0).all()
        sees = torch.zeros((M, M), dtype=torch.bool)
        want, tol = ref.attention(cache, 1, x[1, :, :2 * G], x[1, :, 2 * G:2 * G + 2], x[1, :, 2 * G + 2:], sees.cuda(),
                                  None, None, 1 / 8.0)
        assert ((out[1].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("M,G", [(6, 2), (70, 4)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, 3.0e38])
def test_what_is_masked_does_not_matter(M, G, value):
    """A node's keys or values reach its descendants and nobody else."""
    cache = make_cache([37], 16, 1, 64, 4)
    x = torch.randn((1, M, G + 2, 64), device="cuda").to(torch.bfloat16)
    anc = ref.path_bits([-1] + [max(0, i - 2) for i in range(1, M)])
    mask = ref.pack(anc, M)[None].cuda()
    bad = 4
    clean = dtree.tree_attention(cache, x[:, :, :G], x[:, :, G:G + 1], x[:, :, G + 1:], mask=mask)
    touched = anc[:, bad].cuda()
    for head in (G, G + 1):
        y = x.clone()
        y[0, bad, head, 11] = value
        out = dtree.tree_attention(cache, y[:, :, :G], y[:, :, G:G + 1], y[:, :, G + 1:], mask=mask)
        # a large finite neighbour may cost the others precision in fp16's range, nothing more
        assert torch.isfinite(out[0, ~touched]).all()
        if not math.isfinite(value):
            assert torch.equal(out[0, ~touched], clean[0, ~touched])
            assert out[0, touched].isnan().flatten(1).any(1).all()


def test_nan_scale_reaches_the_rows_of_its_head():
    cache = make_cache([100, 100], 16, 2, 64, 8)
    cache.k_scale[cache.table[0, 2].long(), 1] = math.nan
    for M in (2, 80):
        x = torch.randn((2, M, 8, 64), device="cuda").to(torch.bfloat16)
        out = dtree.tree_attention(cache, x[:, :, :4], x[:, :, 4:6], x[:, :, 6:])
        assert out[0, :, 2:].isnan().all() and torch.isfinite(out[0, :, :2]).all() and torch.isfinite(out[1]).all()


def test_offsets_past_32_bits():
    """Pages that lie more than 2^32 bytes into the cache."""
    page, Hkv, D, n_pages = 128, 8, 128, 34000
    k = torch.zeros((n_pages, Hkv, page, D), dtype=torch.uint8, device="cuda")
    v, ks = torch.zeros_like(k), torch.full((n_pages, Hkv), 2.0 ** -6, device="cuda")
    ids = torch.tensor([[33999, 3, 33001]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (k, v):
        t[ids[0].long()] = (torch.randn((3, Hkv, page, D), generator=g, device="cuda") * 60).to(
            torch.float8_e4m3fn).view(torch.uint8)
    cache = dtree.PagedCache(k, v, ks, ks.clone(), ids, torch.tensor([300], dtype=torch.int32, device="cuda"))
    for M in (1, 40):
        x = torch.randn((1, M, 32, D), generator=g, device="cuda").to(torch.bfloat16)
        q, kn, vn = x[:, :, :16], x[:, :, 16:24], x[:, :, 24:]
        out = dtree.tree_attention(cache, q, kn, vn)
        want, tol = ref.attention(cache, 0, q[0], kn[0], vn[0], torch.ones((M, M), dtype=torch.bool).tril().cuda(), None,
                                  None, 1 / math.sqrt(D))
        assert ((out[0].double() - want).abs() <= tol).all()


def test_other_stream_and_graph():
    """A call on a side stream, and a captured one replayed with new lengths and queries."""
    cache = make_cache([300, 40], 32, 2, 128, 21)
    x = torch.randn((2, 3, 12, 128), device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :, :8], x[:, :, 8:10], x[:, :, 10:]
    ws, st = dtree.attention_workspace(cache, 3, 8), torch.zeros(2, dtype=torch.int32, device="cuda")
    want = dtree.tree_attention(cache, q, k, v, workspace=ws, status=st)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dtree.tree_attention(cache, q, k, v, out=out, workspace=ws, status=st, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dtree.tree_attention(cache, q, k, v, out=out, workspace=ws, status=st)
    for n in (299, 12, 0):
        cache.len.fill_(min(n, 40))
        cache.len[0] = n
        x.copy_(torch.randn_like(x.float()).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dtree.tree_attention(cache, q, k, v))


def test_out_of_range_requests_are_flagged():
    """A length, page or position out of range: the status bit, and the other request as always."""
    cache = make_cache([100, 60], 16, 1, 64, 5)
    rope = dtree.Rope(*ref.rope_tables(120, 64, "cuda"))
    for M in (2, 100):
        x = torch.randn((2, M, 4, 64), device="cuda").to(torch.bfloat16)
        q, k, v = x[:, :, :2], x[:, :, 2:3], x[:, :, 3:]
        pos = torch.zeros((2, M), dtype=torch.int32, device="cuda")
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        want = dtree.tree_attention(cache, q, k, v, pos=pos, rope=rope, status=st)
        assert st.tolist() == [0, 0]

        def flagged(**kw):
            st.zero_()
            out = dtree.tree_attention(cache, q, k, v, pos=pos, rope=rope, status=st, **kw)
            assert st.tolist() == [dtree.DT_DEV_BAD_CACHE, 0]
            assert torch.equal(out[1], want[1])

        for n in (-1, 10 ** 6):
            cache.len[0] = n
            flagged()
        cache.len[0] = 100
        for bad in (-5, 10 ** 8):
            keep = cache.table[0, 3].clone()
            cache.table[0, 3] = bad
            flagged()
            cache.table[0, 3] = keep
        for bad in (-101, 50):
            pos[0, 1] = bad
            flagged()
        pos[0, 1] = 0
        flagged(n_nodes=torch.tensor([M + 1, M], dtype=torch.int32, device="cuda"))


def test_refusals():
    cache = make_cache([10], 16, 2, 64, 1)
    x = torch.randn((1, 3, 8, 64), device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    with pytest.raises(TypeError):
        dtree.tree_attention(cache, q.float(), k, v)
    with pytest.raises(ValueError):  # another number of key heads
        dtree.tree_attention(cache, q, x[:, :, 4:5], x[:, :, 5:6])
    with pytest.raises(ValueError):  # a mask for fewer rows
        dtree.tree_attention(cache, q, k, v, mask=torch.zeros((1, 2, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):  # head elements apart
        dtree.tree_attention(cache, q, k, x.transpose(2, 3).contiguous().transpose(2, 3)[:, :, 6:])
    with pytest.raises(ValueError):
        dtree.tree_attention(cache, q, k, v, out=torch.empty((1, 3, 3, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dtree.DtError):  # three query heads to two key heads
        dtree.tree_attention(cache, x[:, :, :3], k, v)
    with pytest.raises(dtree.DtError):
        dtree.tree_attention(cache, q, k, v, scale=-1.0)
    y = torch.randn((1, 3, 8, 66), device="cuda").to(torch.bfloat16)[..., 1:65]
    with pytest.raises(dtree.DtError):  # head vectors off the 16-byte boundary
        dtree.tree_attention(cache, y[:, :, :4], k, v)
    with pytest.raises(ValueError):
        dtree.PagedCache(cache.k, cache.v[:1], cache.k_scale, cache.v_scale, cache.table, cache.len)
