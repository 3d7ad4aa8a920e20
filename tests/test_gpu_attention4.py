"""Tree attention over the paged 4-bit cache against its definition in 64 bits."""
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


def make_cache(lens, page, Hkv, D, seed, octaves=4, extra_pages=2):
    """A filled cache: blocks over a few octaves, pages in no order, any codes and NaN scales wherever no
    token lies, and no page at all behind the last token's next one."""
    g = torch.Generator().manual_seed(seed)
    max_pages = max(1, max(-(-n // page) for n in lens)) + 1
    n_pages = len(lens) * max_pages + extra_pages
    x = torch.randn((2, n_pages, Hkv, page, D), generator=g)
    x = x * torch.exp2(torch.randint(-octaves, 1, (2, n_pages, Hkv, page, D // 16), generator=g).float()).repeat_interleave(16, -1)
    codes, scales = ref4.quantised(x.cuda().double())
    table = torch.randperm(n_pages, generator=g)[:len(lens) * max_pages].view(len(lens), max_pages).to(torch.int32)
    for b, n in enumerate(lens):
        for p in range(max_pages):
            lo = min(page, max(0, n - p * page))
            codes[:, int(table[b, p]), :, lo:] = torch.randint(0, 256, codes[:, int(table[b, p]), :, lo:].shape, generator=g, dtype=torch.uint8).cuda()
            scales[:, int(table[b, p]), :, lo:] = 255
            if lo == 0 and p > -(-n // page):
                table[b, p] = -1
    return dtree.PagedCache4(codes[0].contiguous(), codes[1].contiguous(), scales[0].contiguous(), scales[1].contiguous(),
                             table.cuda(), torch.tensor(lens, **I32))


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
        if n:
            at = int(cache.len[b]) + depth[b][:n]
            want, tol = ref4.attention(cache, b, q[b, :n], k[b, :n], v[b, :n], sees[b].cuda(), at.cuda(), rope, scale)
            worst = ((out[b, :n].double() - want).abs() / tol).max().item()
            assert torch.isfinite(out[b, :n]).all() and worst <= 1.0, (b, n, int(cache.len[b]), worst)
        assert (out[b, n:] == 0).all()


def inputs(B, M, Hq, Hkv, D, g, layout="fused", hot=1.0):
    x = (torch.randn((B, M, Hq + 2 * Hkv, D), generator=g) * hot).to(torch.bfloat16).cuda()
    if layout == "heads":  # heads before rows
        x = x.transpose(1, 2).contiguous().transpose(1, 2)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]


def run(lens, M, Hq, Hkv, D, page, tree=True, rot=None, interleaved=False, layout="fused", n_nodes=None, seed=0, hot=1.0,
        octaves=4):
    g = torch.Generator().manual_seed(seed + 1)
    B = len(lens)
    cache = make_cache(lens, page, Hkv, D, seed, octaves)
    q, k, v = inputs(B, M, Hq, Hkv, D, g, layout, hot)
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
    status = torch.zeros(B, **I32)
    scale = 1.0 / math.sqrt(D)
    kw = dict(mask=mask, pos=pos, n_nodes=torch.tensor(n_nodes, **I32), rope=rope, scale=scale, status=status)
    out = dtree.tree_attention(cache, q, k, v, **kw)
    again = dtree.tree_attention(cache, q, k, v, **kw)
    assert (status == 0).all()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time
    check(cache, q, k, v, sees, depth, n_nodes, (tabs[0], tabs[1], interleaved) if rot else None, scale, out)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens_at_every_kind_of_length(page, D):
    lens = [0, 1, 7, 8, 9, 15, 16, 17, page - 1, page, page + 1, 127, 128, 129, 255, 2 * page + 3, 700]
    run(lens, 1, 8, 2, D, page, tree=False)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 12, 16, 17])
def test_head_groups(G):
    run([200, 1], 1, 2 * G, 2, 128, 64, tree=False, seed=G)
    run([130, 33], 6, 2 * G, 2, 128, 32, tree=True, seed=G + 100)
    run([77, 140], 2, 2 * G, 2, 64, 16, tree=True, seed=G + 200)


@pytest.mark.parametrize("M", [2, 5, 16, 17, 31, 32, 33, 61, 65, 127, 129])
@pytest.mark.parametrize("D", [64, 128])
def test_trees(M, D):
    run([0, 1, 100, 515], M, 4, 2, D, 64, n_nodes=[M, M - 1, 1, (M + 1) // 2], seed=M)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_trees_over_every_kind_of_length(page, D):
    run([0, 1, 15, 16, 17, page + 1, 127, 128, 129, 300], 20, 4, 1, D, page, seed=page)


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
    run([40, 333], 3, 6, 2, 128, 64, rot=rot, interleaved=interleaved, layout=layout, seed=rot + 1)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_are_rotated_already(page, D):
    """Without a rotation new rows take shorter paths: single tokens, small trees, large ones, chains."""
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 300]
    for G in (1, 4, 7, 12):
        run(lens, 1, 2 * G, 2, D, page, tree=False, rot=0, seed=G)
    run(lens, 5, 6, 2, D, page, rot=0, n_nodes=[5, 1, 2, 0, 5, 1, 3, 4, 5], seed=20)
    run(lens, 61, 6, 2, D, page, rot=0, n_nodes=[61, 1, 2, 0, 60, 33, 32, 31, 61], seed=21)
    run([100, 0], 290, 2, 1, D, page, rot=0, n_nodes=[290, 257], seed=22)
    run([100, 0], 150, 3, 1, D, page, tree=False, rot=0, seed=23)


def test_single_tokens_among_many():
    """Enough units that every CTA has work (shares of two sizes), with more and fewer rows than one."""
    lens = [(577 * i) % 3000 for i in range(48)]
    run(lens, 1, 8, 8, 64, 16, tree=False, rot=0, seed=31)
    run(lens, 3, 8, 4, 128, 64, rot=0, n_nodes=[(i % 3) + 1 for i in range(48)], seed=32)


@pytest.mark.parametrize("G", [2, 12])
def test_a_single_row_of_its_own(G):
    """One new row: not finite, hidden by its mask, or far from the cache's magnitudes."""
    cache = make_cache([100, 0, 30], 32, 2, 128, 5)
    g = torch.Generator().manual_seed(G)
    q, k, v = inputs(3, 1, 2 * G, 2, 128, g)
    see, none = [torch.ones((1, 1), dtype=torch.bool)] * 3, [torch.zeros((1, 1), dtype=torch.bool)] * 3
    at = [torch.arange(1)] * 3
    for size in (2.0 ** -30, 2.0 ** -12, 1.0, 2.0 ** 12):
        out = dtree.tree_attention(cache, q, k, v * size)
        check(cache, q, k, v * size, see, at, [1] * 3, None, 1 / math.sqrt(128), out)
    bad = v.clone()
    bad[:, 0, 0, 7], bad[:, 0, 1, 100] = math.nan, -math.inf
    hidden = torch.zeros((3, 1, 1), **I32)
    out = dtree.tree_attention(cache, q, bad, bad, mask=hidden)
    assert (out[1] == 0).all()  # sees nothing at all
    for b in (0, 2):
        one = dtree.PagedCache4(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table[b:b + 1].contiguous(), cache.len[b:b + 1].contiguous())
        check(one, q[b:b + 1], k[b:b + 1], v[b:b + 1], none[:1], at[:1], [1], None, 1 / math.sqrt(128), out[b:b + 1])
    for kk, vv in ((bad, v), (k, bad)):
        assert torch.isnan(dtree.tree_attention(cache, q, kk, vv)).all()
    qn = q.clone()
    qn[0, 0, 0, 3] = math.nan
    out = dtree.tree_attention(cache, qn, k, v)
    nan = torch.isnan(out).all(-1)
    assert nan[0, 0, 0] and int(nan.sum()) == 1


@pytest.mark.parametrize("G", [2, 12])
@pytest.mark.parametrize("rot", [0, 64])
def test_a_single_row_near_the_end_of_the_range(G, rot):
    """Its values up to 3e38, and keys whose products with the query cancel, each far past fp32's range in
    part.  With a rotation, position 0 (the empty context) turns nothing."""
    cache = make_cache([100, 0, 30] if rot == 0 else [0, 0, 0], 32, 2, 64, 5)
    g = torch.Generator().manual_seed(G)
    q, k, v = (x.clone() for x in inputs(3, 1, 2 * G, 2, 64, g))
    tabs = ref.rope_tables(200, rot, "cuda") if rot else None
    rope = dtree.Rope(*tabs, False) if rot else None
    see, at = [torch.ones((1, 1), dtype=torch.bool)] * 3, [torch.arange(1)] * 3
    for size in (2.0 ** 90, 2.0 ** 99, 2.0 ** 101, 2.0 ** 110, 2.0 ** 122, 2.0 ** 125):
        far = v * size
        assert torch.isfinite(far).all()
        out = dtree.tree_attention(cache, q, k, far, rope=rope)
        check(cache, q, k, far, see, at, [1] * 3, (*tabs, False) if rot else None, 1 / math.sqrt(64), out)
    # q of ones, keys of +x and -x in halves: every score is zero, whatever x, and the row's weight that of
    # a key of zeros
    one, zero = torch.ones_like(q), torch.zeros_like(k)
    for x in (2.0 ** 100, 2.0 ** 124, 2.0 ** 127):
        half = torch.cat((torch.full_like(k[..., :32], x), torch.full_like(k[..., :32], -x)), -1)
        got = dtree.tree_attention(cache, one, half, v, rope=rope)
        check(cache, one, zero, v, see, at, [1] * 3, (*tabs, False) if rot else None, 1 / math.sqrt(64), got)


def test_long_contexts_are_split():
    run([9000, 5, 3001], 1, 16, 2, 128, 64, tree=False, seed=5)
    run([7001], 40, 16, 2, 128, 128, seed=6)
    run([5000, 12], 257, 4, 1, 64, 64, seed=7)
    run([12000], 1, 8, 1, 64, 16, tree=False, seed=8)


def test_more_requests_than_a_warp_looks_at():
    run([(37 * i) % 500 for i in range(70)], 2, 4, 2, 128, 16, seed=21)
    run([(37 * i) % 300 for i in range(40)], 17, 2, 1, 64, 32, seed=22)


def test_requests_without_rows():
    run([50, 0, 128], 3, 4, 2, 64, 32, n_nodes=[0, 0, 3], seed=9)


def test_hot_scores():
    """Scores far apart: single keys dominate, the running maximum keeps moving."""
    run([600], 5, 8, 2, 128, 64, hot=12.0, seed=11)
    run([600], 150, 4, 2, 128, 64, hot=12.0, seed=12)


def test_blocks_of_very_different_magnitudes():
    run([300, 40], 1, 8, 2, 128, 64, tree=False, octaves=14, seed=13)
    run([300, 40], 30, 8, 2, 64, 64, octaves=14, seed=14)


@pytest.mark.parametrize("M,Hq", [(1, 4), (40, 4)])
@pytest.mark.parametrize("byte", [1, 7, 8, 225, 226])
def test_values_at_the_ends_of_the_scales(M, Hq, byte):
    """Values whose scales are the format's smallest and largest; subnormal ones, too."""
    cache = make_cache([200, 3], 32, 2, 128, 4)
    cache.v_scale.copy_(torch.where(cache.v_scale == 255, 255, byte).to(torch.uint8))
    g = torch.Generator().manual_seed(byte)
    q, k, v = inputs(2, M, Hq, 2, 128, g)
    v = v * float(ref4.scale_values(torch.tensor(byte)))
    out = dtree.tree_attention(cache, q, k, v)
    sees = [torch.ones((M, M), dtype=torch.bool).tril()] * 2
    check(cache, q, k, v, sees, [torch.arange(M)] * 2, [M, M], None, 1 / math.sqrt(128), out)


@pytest.mark.parametrize("M,Hq", [(1, 4), (8, 4), (40, 4)])
@pytest.mark.parametrize("small", [-4, -8, -12, -16])
def test_new_rows_count_beside_a_cache_of_small_values(M, Hq, small):
    """Values far below 1 in the cache and in the new rows, which get most of the weight."""
    cache = make_cache([200, 3], 32, 2, 128, 4)
    cache.v_scale.copy_(torch.where(cache.v_scale == 255, 255, 8 * (15 + small) + 4 if small > -15 else 2).to(torch.uint8))
    g = torch.Generator().manual_seed(M)
    q, k, v = inputs(2, M, Hq, 2, 128, g)
    k = torch.nn.functional.normalize(q[:, :, ::2].float(), dim=-1).to(torch.bfloat16) * 8  # near each row's own query
    v = v * 2.0 ** small
    out = dtree.tree_attention(cache, q, k, v)
    sees = [torch.ones((M, M), dtype=torch.bool).tril()] * 2
    check(cache, q, k, v, sees, [torch.arange(M)] * 2, [M, M], None, 1 / math.sqrt(128), out)


def test_rows_that_see_nothing():
    """An empty cache and a mask without a bit: zeros, not NaN."""
    for M, G in ((3, 2), (90, 4)):
        cache = make_cache([0, 20], 16, 2, 64, 3)
        x = torch.randn((2, M, 2 * G + 4, 64), device="cuda").to(torch.bfloat16)
        mask = torch.zeros((2, M, (M + 31) // 32), **I32)
        out = dtree.tree_attention(cache, x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:], mask=mask)
        assert (out[0] == 0).all()
        none = [torch.zeros((M, M), dtype=torch.bool)] * 2
        check(cache, x[:, :, :2 * G], x[:, :, 2 * G:2 * G + 2], x[:, :, 2 * G + 2:], none, [torch.arange(M)] * 2, [0, M],
              None, 1 / 8, torch.cat((torch.zeros_like(out[:1]), out[1:])))


@pytest.mark.parametrize("M", [2, 70])
def test_not_finite_reaches_the_rows_that_see_it(M):
    """A NaN block of the cache: every row of its request and key head.  NaN and infinity in new rows that a
    row does not see: nothing."""
    g = torch.Generator().manual_seed(M)
    q, k, v = inputs(2, M, 4, 2, 128, g)
    for which in ("k_scale", "v_scale"):
        cache = make_cache([100, 90], 32, 2, 128, 5)
        getattr(cache, which)[int(cache.table[1, 1]), 0, 3, 2] = 255  # token 35 of request 1, key head 0
        out = dtree.tree_attention(cache, q, k, v)
        nan = torch.isnan(out)
        assert not nan[0].any() and not nan[1, :, 2:].any()
        want = torch.ones((M, 2, 128), dtype=torch.bool, device="cuda")
        if which == "v_scale":  # a NaN value block: its 16 columns
            want[:] = False
            want[..., 32:48] = True
            assert nan[1, :, :2][want].all()
        else:
            assert torch.equal(nan[1, :, :2], want)
    cache = make_cache([100, 90], 32, 2, 128, 5)
    k2, v2 = k.clone(), v.clone()
    k2[:, M - 1], v2[:, M - 1] = math.inf, math.nan
    a, b = dtree.tree_attention(cache, q, k, v), dtree.tree_attention(cache, q, k2, v2)
    assert torch.equal(a[:, :M - 1], b[:, :M - 1]) and torch.isnan(b[:, M - 1]).all()


@pytest.mark.parametrize("M", [1, 40])
def test_out_of_range(M):
    """Lengths, counts, pages and positions: flagged; the other requests are right."""
    cache = make_cache([50, 50, 50, 50, 20], 16, 2, 64, 7)
    cache.len[0], cache.len[1] = -1, 10 ** 6
    cache.table[2, 1] = cache.n_pages
    g = torch.Generator().manual_seed(1)
    q, k, v = inputs(5, M, 8, 2, 64, g)
    tabs = ref.rope_tables(60 + M, 64, "cuda")
    pos = torch.arange(M, **I32).repeat(5, 1)
    pos[3, M - 1] = 1000
    n = [M] * 5
    status = torch.zeros(5, **I32)
    out = dtree.tree_attention(cache, q, k, v, pos=pos, n_nodes=torch.tensor(n, **I32), rope=dtree.Rope(*tabs), status=status)
    assert status.tolist() == [dtree.DT_DEV_BAD_CACHE] * 4 + [0]
    one = dtree.PagedCache4(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table[4:].contiguous(), cache.len[4:].contiguous())
    check(one, q[4:], k[4:], v[4:], [torch.ones((M, M), dtype=torch.bool).tril()], [torch.arange(M)], [M], (*tabs, False), 1 / 8, out[4:])


def test_pages_past_32_bit_offsets():
    """A pool whose last pages lie past 2^32 bytes, of codes and of scales alike."""
    page, Hkv, D = 128, 16, 128
    n = (1 << 32) // (Hkv * page * D // 16) + 3   # 34 GB of codes
    small = make_cache([200], page, Hkv, D, 9)
    one = lambda w, fill: torch.full((n, Hkv, page, w), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
    k, ks = one(D // 2, 0), one(D // 16, 255)
    for i in range(2):
        p = int(small.table[0, i])
        k[n - 1 - i], ks[n - 1 - i] = small.k[p], small.k_scale[p]
    cache = dtree.PagedCache4(k, k, ks, ks, torch.tensor([[n - 1, n - 2]], **I32), small.len)
    small = dtree.PagedCache4(small.k, small.k, small.k_scale, small.k_scale, small.table, small.len)
    for M in (1, 40):
        q, kn, vn = inputs(1, M, 32, Hkv, D, torch.Generator().manual_seed(M))
        a, b = dtree.tree_attention(cache, q, kn, vn), dtree.tree_attention(small, q, kn, vn)
        assert torch.equal(a, b) and torch.isfinite(a).all()


def test_calls_in_graphs_and_on_streams():
    """A captured call replayed after its inputs changed; two streams with workspaces of their own; a workspace
    that calls of both cache forms share."""
    cache = make_cache([300, 70, 1000], 64, 2, 128, 1)
    eight = dtree.PagedCache.empty(8, 64, 2, 128, 3, 1)
    g = torch.Generator().manual_seed(3)
    for M in (1, 50):
        sets = [inputs(3, M, 16, 2, 128, g) for _ in range(3)]
        want = [dtree.tree_attention(cache, *x) for x in sets]
        ws, status = dtree.attention_workspace(cache, M, 16), torch.zeros(3, **I32)
        buf = [t.clone() for t in sets[0]]
        out = torch.empty_like(want[0])
        call = lambda w=ws, o=out: dtree.tree_attention(cache, *buf, out=o, workspace=w, status=status)  # noqa: E731
        call()
        dtree.tree_attention(eight, *buf, workspace=ws, status=status)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for x, y in zip(sets, want):
            for t, s in zip(buf, x):
                t.copy_(s)
            graph.replay()
            assert torch.equal(out, y)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = []
        for s, x in zip(streams, sets[1:]):
            with torch.cuda.stream(s):
                for _ in range(20):
                    o = dtree.tree_attention(cache, *x)
                got.append(o)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[1:])) and (status == 0).all()
