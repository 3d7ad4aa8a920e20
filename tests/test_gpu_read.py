"""Reading tokens back out of both forms of the paged cache, bit for bit."""
import pytest
import torch

import target4_ref as ref4
from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def make(bits, lens, page, Hkv, D, seed):
    """A cache of random codes and scales (of e4m3 not only powers of two)."""
    g = torch.Generator().manual_seed(seed)
    max_pages = max(-(-max(lens) // page), 1) + 1
    form = dtree.PagedCache4 if bits == 4 else dtree.PagedCache
    cache = form.empty(len(lens) * max_pages + 2, page, Hkv, D, len(lens), max_pages)
    cache.table.copy_(torch.randperm(cache.n_pages, generator=g)[:len(lens) * max_pages].view(len(lens), max_pages))
    cache.len.copy_(torch.tensor(lens))
    for t in (cache.k, cache.v):
        c = torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8)
        if bits == 8:
            c[(c & 127) == 127] = 0x3A
        t.copy_(c)
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.randint(1, 227, s.shape, generator=g) if bits == 4 else torch.exp2(torch.randn(s.shape, generator=g) * 4))
    return cache, g


def values(cache, b):
    """fp32 values [len, Hkv, D] of a request's keys and values: code times scale, rounded once."""
    return [ref4.held(c, s, cache.table[b], int(cache.len[b]), cache.page).float()
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("page,D", [(16, 64), (16, 128), (32, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_whole_contexts(bits, page, D, dtype):
    lens = [0, 1, page - 1, page, page + 1, 3 * page + 7, 300]
    cache, _ = make(bits, lens, page, 3, D, page + D)
    status = torch.zeros(7, dtype=torch.int32, device="cuda")
    k, v = dtree.kv_read(cache, N=max(lens) + 1, dtype=dtype, status=status)
    assert (status == 0).all() and k.dtype == v.dtype == dtype
    for b, m in enumerate(lens):
        for got, want in zip((k, v), values(cache, b)):
            assert torch.equal(got[b, :m], want.to(dtype)) and not got[b, m:].any()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shift", [0, 8])
def test_ranges_into_strided_outputs(bits, shift):
    """start and count + count_add; outputs that are slices of a larger tensor, starting on 16 bytes only."""
    lens, start, count = [90, 5, 33, 200], [80, 0, 33, 7], [9, 4, -1, 149]
    cache, _ = make(bits, lens, 32, 2, 64, 4)
    whole = torch.full((4, 160, 5, 64 + shift), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = whole[:, 3:153, 0:2, shift:], whole[:, 3:153, 2:5:2, shift:]
    i32 = dict(dtype=torch.int32, device="cuda")
    status = torch.zeros(4, **i32)
    dtree.kv_read(cache, start=torch.tensor(start, **i32), count=torch.tensor(count, **i32), count_add=1, k=k, v=v, status=status)
    assert (status == 0).all()
    want = torch.full_like(whole, 7.0)
    for b, (m, n) in enumerate(zip(start, count)):
        x, y = values(cache, b)
        want[b, 3:4 + n, 0:2, shift:] = x[m:m + n + 1].to(torch.bfloat16)
        want[b, 3:4 + n, 2:5:2, shift:] = y[m:m + n + 1].to(torch.bfloat16)
    assert torch.equal(whole, want)


@pytest.mark.parametrize("bits", [4, 8])
def test_picked_tokens(bits):
    """Any order, the same token several times, and entries behind the count that name nothing."""
    lens, count = [700, 1, 40, 0], [77, 30, 0, 0]
    cache, g = make(bits, lens, 64, 4, 128, 8)
    rows = torch.full((4, 77), -9, dtype=torch.int32)
    for b, (m, n) in enumerate(zip(lens, count)):
        if n:
            rows[b, :n] = torch.randint(0, m, (n,), generator=g)
    i32 = dict(dtype=torch.int32, device="cuda")
    status = torch.zeros(4, **i32)
    k, v = dtree.kv_read(cache, rows=rows.cuda(), count=torch.tensor(count, **i32), dtype=torch.float32, status=status)
    assert (status == 0).all()
    for b, n in enumerate(count):
        for got, want in zip((k, v), values(cache, b)):
            assert torch.equal(got[b, :n], want[rows[b, :n].long().cuda()]) and not got[b, n:].any()


def test_what_is_not_finite_comes_back_as_nan():
    """A block that held infinity is NaN as a whole; its neighbours are as they were."""
    for bits, D in ((4, 128), (8, 128)):
        cache, g = make(bits, [0], 16, 1, D, 3)
        x = torch.randn((1, 20, 1, D), generator=g).cuda()
        x[0, 17, 0, 40] = -torch.inf
        new = torch.empty((1,), dtype=torch.int32, device="cuda")
        dtree.kv_append(cache, x, x, len_out=new)
        cache.len.copy_(new)
        k, _ = dtree.kv_read(cache, N=20)
        bad = torch.isnan(k[0, :, 0])
        want = torch.zeros((20, D), dtype=torch.bool, device="cuda")
        if bits == 4:
            want[17, 32:48] = True
        else:
            want[16:] = True  # the page's block
        assert torch.equal(bad, want)


@pytest.mark.parametrize("bits", [4, 8])
def test_requests_out_of_range(bits):
    """Lengths, starts and counts out of range leave a request alone; a bad row or page makes a row zeros."""
    cache, _ = make(bits, [40] * 8, 16, 2, 64, 6)
    good = values(cache, 0)[0][3:8]
    cache.len[1], cache.len[2] = -1, 1000
    cache.table[6, 0], cache.table[7, 0] = cache.n_pages, -1
    i32 = dict(dtype=torch.int32, device="cuda")
    start = torch.tensor([3, 3, 3, -1, 38, 3, 14, 14], **i32)
    count = torch.tensor([5, 5, 5, 5, 5, 7, 5, 5], **i32)
    status = torch.zeros(8, **i32)
    k = torch.full((8, 6, 2, 64), 3.0, device="cuda")
    dtree.kv_read(cache, start=start, count=count, k=k, v=k.clone(), status=status)
    assert status.tolist() == [0] + [dtree.DT_DEV_BAD_CACHE] * 7
    assert torch.equal(k[0, :5], good) and (k[1:6] == 3.0).all()
    assert (k[6:, :2] == 0).all() and (k[6:, 5] == 3.0).all() and (k[6:, 2:5] != 0).any()
    rows = torch.tensor([[0, 40, 2], [-1, 0, 1]], **i32)
    two = type(cache)(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table[[0, 3]].contiguous(), torch.tensor([40, 40], **i32))
    status = torch.zeros(2, **i32)
    k, _ = dtree.kv_read(two, rows=rows, status=status)
    assert status.tolist() == [dtree.DT_DEV_BAD_CACHE] * 2
    for b, bad in ((0, 1), (1, 0)):
        want = values(two, b)[0][rows[b].clamp(0, 39).long()].to(torch.bfloat16)
        want[bad] = 0
        assert torch.equal(k[b], want)


def test_refusals():
    cache, _ = make(4, [10], 16, 2, 64, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        dtree.kv_read(cache)
    with pytest.raises(ValueError):
        dtree.kv_read(cache, rows=torch.zeros((1, 3), **i32), start=torch.zeros(1, **i32))
    with pytest.raises(ValueError):
        dtree.kv_read(cache, N=4, rows=torch.zeros((1, 3), **i32))
    with pytest.raises(TypeError):
        dtree.kv_read(cache, N=4, dtype=torch.float16)
    k = torch.zeros((1, 4, 2, 64), device="cuda")
    with pytest.raises(TypeError):
        dtree.kv_read(cache, k=k, v=k.bfloat16())
    with pytest.raises(ValueError):
        dtree.kv_read(cache, k=k, v=k[:, :, :1])
    with pytest.raises(dtree.DtError):
        dtree.kv_read(cache, k=torch.zeros(1 + 4 * 2 * 64, device="cuda")[1:].view(1, 4, 2, 64), v=k)
    with pytest.raises(ValueError):
        dtree.PagedCache4(cache.k, cache.v, cache.k_scale, cache.v_scale[..., :2].contiguous(), cache.table, cache.len)
