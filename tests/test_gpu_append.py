"""Appending to the paged e4m3 cache against its definition in 64 bits."""
import math

import pytest
import torch

import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu

TOP = 448.0


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def exponent(amax):
    """Smallest e >= -48 with amax <= 448 * 2^e."""
    f, x = math.frexp(amax)
    return max(-48, (x - 9 if f <= 0.875 else x - 8) if amax > 0 else -48)


def make(lens, grow, page, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    max_pages = max(-(-(n + grow) // page) for n in lens) + 1
    cache = dtree.PagedCache.empty(len(lens) * max_pages + 2, page, Hkv, D, len(lens), max_pages)
    perm = torch.randperm(cache.n_pages, generator=g)[:len(lens) * max_pages]
    cache.table.copy_(perm.view(len(lens), max_pages))
    cache.len.copy_(torch.tensor(lens))
    codes = torch.randint(0, 256, (2, *cache.k.shape), generator=g, dtype=torch.uint8)
    codes[(codes & 127) == 127] = 0x3A  # no NaN codes
    cache.k.copy_(codes[0])
    cache.v.copy_(codes[1])
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.exp2(torch.randint(-12, -2, s.shape, generator=g).float()))
    return cache, g


def snapshot(c):
    return [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]


def check(cache, before, lens, counts, k, v, rows, rope):
    """Every byte of the cache: what was appended, what was rescaled, what had to stay."""
    page, D = cache.page, cache.D
    touched = set()
    for b, (m, n) in enumerate(zip(lens, counts)):
        if n == 0:
            continue
        at = torch.arange(m, m + n, device="cuda")
        pick = torch.arange(n, device="cuda") if rows is None else rows[b, :n].long()
        new = (ref.rotate(k[b][pick].double(), at, rope), v[b][pick].double())
        for p in range(m // page, (m + n - 1) // page + 1):
            i = int(cache.table[b, p])
            touched.add(i)
            lo, hi = max(m, p * page), min(m + n, (p + 1) * page)
            for which, x in enumerate(new):
                codes, scale = (cache.k, cache.v)[which][i], (cache.k_scale, cache.v_scale)[which][i]
                old, was = before[which][i], before[2 + which][i]
                y = x[lo - m:hi - m].transpose(0, 1)  # [Hkv, rows, D]
                for h in range(cache.Hkv):
                    amax = y[h].abs().max().item()
                    # the rotation's two rounded products and sum put amax within 2^-22 of the kernel's
                    want = {exponent(amax * f) for f in (1 - 2.0 ** -22, 1.0, 1 + 2.0 ** -22)}
                    if lo > p * page:
                        want = {max(e, round(math.log2(was[h].item()))) for e in want}
                    s = scale[h].item()
                    assert s in {2.0 ** e for e in want}, (b, p, h, s, want)
                    got = ref.e4m3_values(codes[h, lo - p * page:hi - p * page]) * s
                    # half a step: 2^-4 of the magnitude, or of the smallest normal 2^-6; and the rotation's rounding
                    tol = torch.maximum(y[h].abs() * 2.0 ** -4, torch.tensor(s * 2.0 ** -10)) + amax * 2.0 ** -21
                    assert ((got - y[h]).abs() <= tol).all()
                    kept = slice(0, lo - p * page)
                    f = was[h].double() / s
                    z = ref.e4m3_values(old[h, kept]) * f
                    d = (ref.e4m3_values(codes[h, kept]) - z).abs()
                    assert (d <= torch.maximum(z.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))).all()
                    if f == 1:
                        assert torch.equal(codes[h, kept], old[h, kept])
                    assert torch.equal(codes[h, hi - p * page:], old[h, hi - p * page:])
    rest = torch.tensor([i for i in range(cache.n_pages) if i not in touched], device="cuda")
    for now, old in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(now[rest], old[rest])


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


@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, True), (64, False), (128, True)])
def test_accepted_paths(rot, interleaved):
    """Rows picked by the walk's outputs: the root and the accepted nodes, -1 after them."""
    lens, acc = [5, 90, 31, 64], [0, 16, 3, 7]
    cache, g = make(lens, 17, 32, 2, 128, rot)
    rows = torch.full((4, 17), -1, dtype=torch.int32)
    for b, a in enumerate(acc):
        rows[b, :a + 1] = torch.randperm(40, generator=g)[:a + 1].sort().values
    rows = rows.cuda()
    k = torch.randn((4, 2, 41, 128), generator=g).cuda().transpose(1, 2)  # heads before rows
    v = torch.randn((4, 41, 2, 128), generator=g).cuda()
    tabs = ref.rope_tables(128, rot, "cuda") if rot else None
    before = snapshot(cache)
    st = dtree.kv_append(cache, k, v, rope=dtree.Rope(*tabs, interleaved) if rot else None, rows=rows,
                         count=torch.tensor(acc, dtype=torch.int32).cuda(), count_add=1)
    assert (st == 0).all()
    check(cache, before, lens, [a + 1 for a in acc], k, v, rows, (*tabs, interleaved) if rot else None)


def test_all_rows_of_one_token():
    cache, g = make([16, 3], 1, 16, 1, 64, 3)
    k, v = torch.randn((2, 1, 1, 64), generator=g).cuda(), torch.randn((2, 1, 1, 64), generator=g).cuda()
    before = snapshot(cache)
    dtree.kv_append(cache, k, v)
    check(cache, before, [16, 3], [1, 1], k, v, None, None)


def test_token_by_token_reads_back():
    """A page filled one token at a time, growing: every token within half a step at the final scale,
    plus what one rescaling may cost (subnormals only: half of 2^-9 per growth of the scale)."""
    cache, g = make([0], 40, 32, 1, 64, 12)
    x = torch.randn((40, 2, 64), generator=g).cuda() * torch.exp2(torch.arange(40) / 4).cuda()[:, None, None]
    for j in range(40):
        cache.len.fill_(j)
        dtree.kv_append(cache, x[j, 0].view(1, 1, 1, 64), x[j, 1].view(1, 1, 1, 64))
    cache.len.fill_(40)
    for i, (codes, scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        got = ref.held(codes, scale, cache.table[0], 40, 32)[:, 0]
        s = scale[cache.table[0].long(), 0].double().repeat_interleave(32)[:40, None]
        want = x[:, i].double()
        assert ((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) + s * 2.0 ** -9).all()


def test_extreme_values():
    """Zeros, the smallest and the largest numbers, exact ties of the scale."""
    for value in (0.0, 1e-40, 2.0 ** -60, 7.0, 7.0000005, 448.0, 449.0, 3.3e38):
        cache, _ = make([0], 2, 16, 1, 64, 1)
        x = torch.zeros((1, 2, 1, 64), device="cuda")
        x[0, 1, 0, 5] = -value
        dtree.kv_append(cache, x, x)
        e = exponent(float(x.abs().max()))
        i = int(cache.table[0, 0])
        assert cache.k_scale[i, 0].item() == cache.v_scale[i, 0].item() == 2.0 ** e
        got = ref.e4m3_values(cache.k[i, 0, 1, 5]).item() * 2.0 ** e
        assert abs(got + float(x.abs().max())) <= max(2.0 ** -4 * value, 2.0 ** (e - 10))


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_values_that_are_not_finite(value):
    """Their block's scale is NaN, then and for later tokens of the block; other blocks are untouched."""
    cache, g = make([8], 20, 16, 2, 64, 6)
    k, v = torch.randn((1, 16, 2, 64), generator=g).cuda(), torch.randn((1, 16, 2, 64), generator=g).cuda()
    k[0, 10, 1, 3] = value
    dtree.kv_append(cache, k, v)
    t = cache.table[0].tolist()
    assert torch.isfinite(cache.k_scale[t[0]]).all() and torch.isfinite(cache.v_scale[t[:2]]).all()
    assert torch.isfinite(cache.k_scale[t[1], 0]) and cache.k_scale[t[1], 1].isnan()
    cache.len.fill_(24)
    dtree.kv_append(cache, k[:, :1], v[:, :1])
    assert cache.k_scale[t[1], 1].isnan() and torch.isfinite(cache.k_scale[t[1], 0])


def test_requests_that_do_not_fit_are_left_alone():
    def attempt(change, expect, **kw):
        cache, g = make([10, 20, 5], 8, 16, 1, 64, 4)
        k, v = torch.randn((3, 8, 1, 64), generator=g).cuda(), torch.randn((3, 8, 1, 64), generator=g).cuda()
        rows = torch.arange(8, dtype=torch.int32).repeat(3, 1).cuda()
        count = torch.full((3,), 8, dtype=torch.int32).cuda()
        rope = dtree.Rope(*ref.rope_tables(40, 64, "cuda"))
        change(cache, rows, count)
        before, lens = snapshot(cache), cache.len.clone()
        out = torch.full((3,), -9, dtype=torch.int32, device="cuda")
        st = dtree.kv_append(cache, k, v, rope=rope, rows=rows, count=count, len_out=out, **kw)
        assert st.tolist() == [0, expect, 0]
        assert out[1] == lens[1] and out[0] == 18
        ids = cache.table[1]
        ids = ids[(ids >= 0) & (ids < cache.n_pages)].long()
        for now, old in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
            assert torch.equal(now[ids], old[ids])

    BAD = dtree.DT_DEV_BAD_CACHE
    attempt(lambda c, r, n: c.len[1:2].fill_(-1), BAD)
    attempt(lambda c, r, n: c.len[1:2].fill_(c.max_pages * 16 - 7), BAD)  # one slot short
    attempt(lambda c, r, n: c.len[1:2].fill_(33), BAD)                    # one position past the tables
    attempt(lambda c, r, n: n[1:2].fill_(9), BAD)
    attempt(lambda c, r, n: n[1:2].fill_(-2), BAD)
    attempt(lambda c, r, n: r[1, 7:].fill_(8), BAD)
    attempt(lambda c, r, n: r[1, 2:3].fill_(-1), BAD)
    attempt(lambda c, r, n: c.table[1, 1:2].fill_(c.n_pages), BAD)
    attempt(lambda c, r, n: n[1:2].fill_(0), 0)                           # nothing to append is fine


def test_pages_past_32_bits():
    """Pages that lie more than 2^32 bytes into the cache."""
    cache = dtree.PagedCache.empty(34000, 128, 8, 128, 1, 2)
    cache.table.copy_(torch.tensor([[33990, 7]]))
    cache.len.fill_(100)
    k = torch.randn((1, 60, 8, 128), device="cuda")
    before = snapshot(cache)
    dtree.kv_append(cache, k, -k)
    check(cache, before, [100], [60], k, -k, None, None)


def test_refusals():
    cache, g = make([0, 0], 4, 16, 2, 64, 2)
    k = torch.randn((2, 4, 2, 64), device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        dtree.kv_append(cache, k, k.to(torch.bfloat16))
    with pytest.raises(TypeError):
        dtree.kv_append(cache, k.half(), k.half())
    with pytest.raises(ValueError):
        dtree.kv_append(cache, k[:, :, :1], k[:, :, :1])
    with pytest.raises(ValueError):
        dtree.kv_append(cache, k, k, rows=torch.zeros((1, 4), **i32))
    with pytest.raises(ValueError):
        dtree.kv_append(cache, k, k, count=torch.zeros((1,), **i32))
    with pytest.raises(dtree.DtError):  # the lengths the call reads are not its output
        dtree.kv_append(cache, k, k, len_out=cache.len)
    with pytest.raises(dtree.DtError):  # rotates more than the head holds
        dtree.kv_append(cache, k, k, rope=dtree.Rope(*ref.rope_tables(8, 128, "cuda")))
    odd = torch.randn((2, 4, 2, 65), device="cuda")[..., 1:]
    with pytest.raises(dtree.DtError):  # off the 16-byte boundary
        dtree.kv_append(cache, odd, odd)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotation_rounds_every_step(dtype, interleaved):
    """Each product and each sum of the rotation is rounded once: with 2^24 keys the codes would
    show some of the last-bit differences that a contracted product and sum makes."""
    n, H, D, page = 8192, 16, 128, 128
    g = torch.Generator(device="cuda").manual_seed(7)
    k = torch.randn((1, n, H, D), generator=g, device="cuda").to(dtype)
    cos, sin = ref.rope_tables(n, D, "cuda")
    cache = dtree.PagedCache.empty(n // page, page, H, D, 1, n // page)
    cache.table.copy_(torch.arange(n // page).view(1, -1))
    assert not dtree.kv_append(cache, k, k, rope=dtree.Rope(cos, sin, interleaved)).any()
    x = k[0].float()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :D // 2], x[..., D // 2:])
    c, s = cos[:, None], sin[:, None]
    p, q, r, t = a * c, b * s, b * c, a * s
    first, second = p - q, r + t
    x = torch.stack((first, second), -1).flatten(-2) if interleaved else torch.cat((first, second), -1)
    for codes, scale, y in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, k[0].float())):
        y = y.view(n // page, page, H, D).transpose(1, 2)
        f, e = torch.frexp(y.abs().amax((2, 3)))
        e = torch.where(f <= 0.875, e - 9, e - 8)
        assert torch.equal(scale, torch.exp2(e.float()))
        assert torch.equal(codes, (y / torch.exp2(e.float())[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8))
