"""The target-side calls together: the example's rounds of draft, verify and append."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("decode_rounds", os.path.join(ROOT, "examples", "decode_rounds.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def prompts_of(ex, lengths):
    p = torch.full((len(lengths), max(lengths)), -1, device="cuda")
    for i, n in enumerate(lengths):
        p[i, :n] = torch.randint(0, ex.V, (n,), generator=torch.Generator().manual_seed(10 + i)).cuda()
    return p


@pytest.mark.parametrize("lengths", [(1,), (1, 17, 50), (33, 16, 2, 9)])
def test_rounds(ex, lengths):
    """Lengths add up, greedy emits tokens of rank 0, and what was emitted is what the contexts hold:
    a fresh prefill of prompt and emitted tokens gives the first layer's cache again, up to the
    rounding of codes that were appended in other portions."""
    model, rounds = ex.Model(), 5
    prompts = prompts_of(ex, lengths)
    got, caches, status = ex.decode(model, prompts, rounds)
    assert not status.any()
    for i, n in enumerate(lengths):
        assert rounds <= len(got[i]) <= rounds * (ex.L + 1)
        assert caches[0].len[i] == caches[1].len[i] == n - 1 + len(got[i])
        assert all(rank == 0 for _, _, rank in got[i])
        assert all(lp <= 0.0 for _, lp, _ in got[i])
    # some request got more than plain decoding's one token per round
    assert max(len(g) for g in got) > rounds
    # the whole sequences as prompts of their own
    full = torch.full((len(lengths), max(n + len(g) for n, g in zip(lengths, got))), -1, device="cuda")
    for i, n in enumerate(lengths):
        full[i, :n] = prompts[i, :n]
        full[i, n:n + len(got[i])] = torch.tensor([t for t, _, _ in got[i]], device="cuda")
    again = ex.new_caches(len(lengths), full.shape[1])
    st = torch.zeros((len(lengths),), dtype=torch.int32, device="cuda")
    assert torch.equal(ex.prefill(model, full, again, st), full.gather(1, (full >= 0).sum(1, keepdim=True) - 1)[:, 0])
    assert not st.any() and torch.equal(again[0].len, caches[0].len)
    # the first layer's keys and values are a function of the tokens alone
    for i in range(len(lengths)):
        m = int(again[0].len[i])
        for name in ("k", "v"):
            a, b = (held(c, name, i, m) for c in (again[0], caches[0]))
            # two roundings of one value: half a step of e4m3 (2^-4) each, and the coarser of two scales
            # (at most 2^8 apart below the block's largest number 448 * scale): absolute 2^-9 of it
            top = a.abs().amax()
            assert ((a - b).abs() <= a.abs() * 2.0 ** -3 + top * 2.0 ** -9).all()


def held(cache, name, i, m):
    codes = getattr(cache, name).view(torch.float8_e4m3fn).float()
    x = codes * getattr(cache, name + "_scale")[:, :, None, None]
    x = x[cache.table[i].clamp(min=0).long()]  # [pages, Hkv, page, D]
    return x.transpose(1, 2).reshape(-1, cache.Hkv, cache.D)[:m]


def test_one_node_trees_are_plain_decoding(ex):
    """A tree of one node and a chain of one row are the same call."""
    model = ex.Model(1)
    prompts = prompts_of(ex, (20, 3))
    st = torch.zeros((2,), dtype=torch.int32, device="cuda")
    caches = ex.new_caches(2, 64)
    last = ex.prefill(model, prompts, caches, st)
    ws = ex.dtree.attention_workspace(caches[0], 1, ex.HQ)
    mask, pos = (torch.ones((2, 1, 1), dtype=torch.int32, device="cuda"), torch.zeros((2, 1), dtype=torch.int32, device="cuda"))
    a, _ = model.forward(last[:, None], caches, ws, st)
    b, _ = model.forward(last[:, None], caches, ws, st, mask=mask, pos=pos)
    assert torch.equal(a, b) and not st.any()
