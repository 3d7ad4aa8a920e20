"""Appending to the paged 4-bit cache, bit for bit."""
import pytest
import torch

import target4_ref as ref4
import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def make(lens, grow, page, Hkv, D, seed):
    """A cache of random bytes."""
    g = torch.Generator().manual_seed(seed)
    max_pages = max(-(-(n + grow) // page) for n in lens) + 1
    cache = dtree.PagedCache4.empty(len(lens) * max_pages + 2, page, Hkv, D, len(lens), max_pages)
    cache.table.copy_(torch.randperm(cache.n_pages, generator=g)[:len(lens) * max_pages].view(len(lens), max_pages))
    cache.len.copy_(torch.tensor(lens))
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    return cache, g


def snapshot(c):
    return [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]


def check(cache, before, lens, counts, k, v, rows, rope):
    """Every byte of the cache: the new tokens' by the definition, all others as they were."""
    want = [t.clone() for t in before]
    for b, (m, n) in enumerate(zip(lens, counts)):
        at = torch.arange(m, m + n, device="cuda")
        pick = torch.arange(n, device="cuda") if rows is None else rows[b, :n].long()
        ids, slot = cache.table[b, at // cache.page].long(), at % cache.page
        for i, x in enumerate((ref4.rotated32(k[b][pick], at, rope), v[b][pick].float())):
            codes, scales = ref4.quantised(x.double())
            want[i][ids, :, slot], want[2 + i][ids, :, slot] = codes, scales
    for got, w, name in zip((cache.k_scale, cache.v_scale, cache.k, cache.v), (want[2], want[3], want[0], want[1]),
                            ("k_scale", "v_scale", "k", "v")):
        assert torch.equal(got, w), (name, int((got != w).sum()))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompts(page, D, dtype):
    lens = [0, 1, page - 1, page, page + 5, 3 * page - 2]
    counts = [150, 1, 2, page, 0, 77]
    cache, g = make(lens, 150, page, 3, D, page + D)
    kv = (torch.randn((len(lens), 150, 6, D), generator=g) * 3).to(dtype).cuda()
    k, v = kv[:, :, :3], kv[:, :, 3:]
    cos, sin = ref.rope_tables(600, D, "cuda")
    before = snapshot(cache)
    out = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    st = dtree.kv_append(cache, k, v, rope=dtree.Rope(cos, sin), count=torch.tensor(counts, dtype=torch.int32).cuda(),
                         len_out=out)
    assert (st == 0).all() and out.tolist() == [a + b for a, b in zip(lens, counts)]
    assert cache.len.tolist() == lens
    check(cache, before, lens, counts, k, v, None, (cos, sin, False))


@pytest.mark.parametrize("D,rot,interleaved", [(128, 0, False), (128, 16, True), (128, 16, False), (128, 48, False),
                                               (128, 64, False), (128, 80, True), (128, 96, False), (128, 112, False),
                                               (128, 128, True), (64, 16, False), (64, 32, False), (64, 48, False),
                                               (64, 48, True), (64, 64, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotations_of_accepted_paths(D, rot, interleaved, dtype):
    """Rows picked by the walk's outputs: the root and the accepted nodes, -1 after them."""
    lens, acc = [0, 5, 60, 63, 700], [8, 0, 3, 1, 5]
    cache, g = make(lens, 9, 64, 2, D, rot)
    kv = torch.randn((5, 41, 4, D), generator=g).to(dtype).cuda()
    k, v = kv[:, :, 1:3], kv[:, :, :4:3]
    rows = torch.full((5, 9), -1, dtype=torch.int32)
    for b, a in enumerate(acc):
        rows[b, :a + 1] = torch.randperm(41, generator=g)[:a + 1].sort().values
    rows = rows.cuda()
    tabs = ref.rope_tables(709, rot, "cuda") if rot else None
    before = snapshot(cache)
    st = dtree.kv_append(cache, k, v, rope=dtree.Rope(*tabs, interleaved) if rot else None, rows=rows,
                         count=torch.tensor(acc, dtype=torch.int32).cuda(), count_add=1)
    assert (st == 0).all()
    check(cache, before, lens, [a + 1 for a in acc], k, v, rows, (*tabs, interleaved) if rot else None)


def edge_blocks():
    """Blocks of 16 at and around every border of the format, fp32: for each scale s, magnitudes up to 6 s,
    borders between codes and their neighbours in fp32, with signs."""
    s = ref4.scale_values(torch.arange(1, ref4.TOP + 1)).float()
    out = []
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for x in s:
        e = edges * x
        up, down = torch.nextafter(e, torch.tensor(torch.inf)), torch.nextafter(e, torch.tensor(0.0))
        sign = torch.tensor([1.0, -1.0] * 8)
        out.append(torch.cat((6 * x[None], e, up, torch.zeros(1))) * sign)
        out.append(torch.cat((6 * x[None], down, e, -torch.zeros(1))) * sign)
        out.append(torch.cat((torch.nextafter(6 * x, torch.tensor(torch.inf))[None], up, down, 6 * x[None])) * sign)
        out.append(torch.cat((torch.nextafter(6 * x, torch.tensor(0.0))[None], e, up, x[None])) * sign)
    least = 2.0 ** -149
    out += [torch.zeros(16), -torch.zeros(16), torch.full((16,), least), torch.full((16,), 2.0 ** -126),
            torch.linspace(-3e38, 3e38, 16), torch.linspace(-7e4, 7e4, 16), torch.full((16,), 61440.0),
            torch.tensor([2.0 ** -17, -2.0 ** -19] * 8)]
    for odd in (torch.inf, -torch.inf, torch.nan):
        x = torch.linspace(-1, 1, 16)
        x[5] = odd
        out.append(x)
    return torch.stack(out)


@pytest.mark.parametrize("D", [64, 128])
def test_every_border_of_the_format(D):
    blocks = edge_blocks()
    per = D // 16
    n = -(-len(blocks) // per)
    x = torch.zeros((n * per, 16))
    x[:len(blocks)] = blocks
    x = x.view(1, n, 1, D).cuda()
    cache, _ = make([7], n, 64, 1, D, 3)
    before = snapshot(cache)
    st = dtree.kv_append(cache, x, x.flip(-1).contiguous())
    assert (st == 0).all()
    check(cache, before, [7], [n], x, x.flip(-1), None, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_magnitudes_from_smallest_to_largest(dtype):
    g = torch.Generator().manual_seed(5)
    x = torch.randn((2, 600, 4, 128), generator=g) * torch.exp2(torch.randint(-60, 30, (2, 600, 4, 8), generator=g).float()).repeat_interleave(16, -1)
    x = x.to(dtype).cuda()
    cache, _ = make([3, 0], 600, 32, 4, 128, 9)
    before = snapshot(cache)
    assert (dtree.kv_append(cache, x, x.flip(1).contiguous()) == 0).all()
    check(cache, before, [3, 0], [600, 600], x, x.flip(1), None, None)


def test_requests_out_of_range_are_left_alone():
    """Bad lengths, counts, rows, pages and positions: flagged, nothing written, others unharmed."""
    lens = [3, -1, 500, 3, 3, 3, 40, 2]
    cache, g = make([64] * 8, 40, 16, 2, 64, 1)
    cache.len.copy_(torch.tensor(lens))
    cache.table[6, 2] = cache.n_pages    # first page written
    cache.table[7, 0] = -1
    counts = torch.tensor([2, 1, 1, -1, 10, 2, 9, 3], dtype=torch.int32).cuda()
    kv = torch.randn((8, 30, 4, 64), generator=g).to(torch.bfloat16).cuda()
    rows = torch.arange(9, dtype=torch.int32).repeat(8, 1)
    rows[5, 1] = 30
    rows = rows.cuda()
    cos, sin = ref.rope_tables(49, 64, "cuda")
    before = snapshot(cache)
    out = torch.full((8,), -5, dtype=torch.int32, device="cuda")
    st = dtree.kv_append(cache, kv[:, :, :2], kv[:, :, 2:], rope=dtree.Rope(cos, sin), rows=rows, count=counts, len_out=out)
    assert st.tolist() == [0] + [dtree.DT_DEV_BAD_CACHE] * 7
    assert out.tolist() == [5, -1, 500, 3, 3, 3, 40, 2]
    check(cache, before, [3] + [0] * 7, [2] + [0] * 7, kv[:, :, :2], kv[:, :, 2:], rows, (cos, sin, False))


def test_pages_past_32_bit_offsets():
    """A pool whose last pages lie past 2^32 bytes."""
    page, Hkv, D = 128, 16, 128
    n = (1 << 32) // (Hkv * page * D // 2) + 3
    cache = dtree.PagedCache4(*(torch.zeros((n, Hkv, page, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2)),
                              *(torch.zeros((n, Hkv, page, D // 16), dtype=torch.uint8, device="cuda") for _ in range(2)),
                              torch.tensor([[n - 1, n - 2]], dtype=torch.int32).cuda(), torch.tensor([100], dtype=torch.int32).cuda())
    g = torch.Generator().manual_seed(2)
    kv = torch.randn((1, 60, 2 * Hkv, D), generator=g).to(torch.bfloat16).cuda()
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:]
    new = torch.empty((1,), dtype=torch.int32, device="cuda")
    assert (dtree.kv_append(cache, k, v, len_out=new) == 0).all()
    assert int(cache.k[:n - 2].any()) == 0
    cache.len.copy_(new)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = dtree.kv_read(cache, N=60, start=torch.tensor([100], dtype=torch.int32).cuda(), dtype=torch.float32, status=status)
    assert int(status) == 0
    for got, x in ((a, k), (b, v)):
        assert torch.equal(got.double(), ref4.values4(*ref4.quantised(x.double())))
