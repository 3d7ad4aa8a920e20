"""Norms, attention, append and read-back together: rounds of the example with a 4-bit context and a
model that normalises its heads, and a layer's calls captured into one graph."""
import importlib.util
import os

import pytest
import torch

import target4_ref as ref4
import target_ref as ref
from speculative_decoding_draft_bf16_gb300 import dtree

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I32 = dict(dtype=torch.int32, device="cuda")


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


@pytest.mark.parametrize("bits,normed", [(4, True), (4, False), (8, True)])
@pytest.mark.parametrize("lengths", [(1,), (33, 16, 2, 9)])
def test_rounds(ex, bits, normed, lengths):
    """Lengths add up, greedy emits tokens of rank 0, and a fresh prefill of prompt and emitted tokens
    gives the first layer's context again."""
    model, rounds = ex.Model(normed=normed), 5
    prompts = prompts_of(ex, lengths)
    got, caches, status = ex.decode(model, prompts, rounds, bits=bits)
    assert not status.any()
    for i, n in enumerate(lengths):
        assert rounds <= len(got[i]) <= rounds * (ex.L + 1)
        assert caches[0].len[i] == caches[1].len[i] == n - 1 + len(got[i])
        assert all(rank == 0 and lp <= 0.0 for _, lp, rank in got[i])
    full = torch.full((len(lengths), max(n + len(g) for n, g in zip(lengths, got))), -1, device="cuda")
    for i, n in enumerate(lengths):
        full[i, :n] = prompts[i, :n]
        full[i, n:n + len(got[i])] = torch.tensor([t for t, _, _ in got[i]], device="cuda")
    again = ex.new_caches(len(lengths), full.shape[1], bits=bits)
    st = torch.zeros((len(lengths),), **I32)
    ex.prefill(model, full, again, st)
    assert not st.any() and torch.equal(again[0].len, caches[0].len)
    N = int(again[0].len.max())
    if bits != 4 or N == 0:
        return
    for a, b in zip(dtree.kv_read(again[0], N=N, dtype=torch.float32), dtree.kv_read(caches[0], N=N, dtype=torch.float32)):
        # the first layer's rows are a function of the tokens alone, up to the products' roundings in bf16
        # (2^-6 of a value at most); both sides lie within half a step of them: a quarter of the value, or
        # of the scale, so a third of what is held, or a quarter of the scale, which is at most a quarter
        # of the block's largest held number
        top = a.unflatten(-1, (-1, 16)).abs().amax(-1).repeat_interleave(16, -1)
        assert ((a - b).abs() <= 2 * torch.maximum(a.abs() / 3, top / 16) + a.abs() * 2.0 ** -6).all()
        assert a.any()


@pytest.mark.parametrize("M", [1, 6, 90])
def test_a_layer_in_one_graph(M):
    """Norms, attention over 4 bits, append and read-back, captured together: replays on new inputs give
    what the calls give one by one."""
    B, Hq, Hkv, D = 3, 8, 2, 128
    lens = torch.tensor([70, 0, 400], **I32)
    cos, sin = ref.rope_tables(600, D, "cuda")
    rope, w = dtree.Rope(cos, sin), torch.rand((D,), device="cuda") + 0.5
    count = torch.tensor([M, (M + 1) // 2, M], **I32)
    g = torch.Generator().manual_seed(M)

    def fresh():
        cache = dtree.PagedCache4.empty(60, 32, Hkv, D, B, 16)
        cache.table.copy_(torch.randperm(60, generator=torch.Generator().manual_seed(5))[:48].view(3, 16))
        old = torch.randn((B, 400, 2 * Hkv, D), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
        dtree.kv_append(cache, old[:, :, :Hkv], old[:, :, Hkv:], count=lens)
        cache.len.copy_(lens)
        s = dict(cache=cache, new=torch.zeros_like(lens), status=torch.zeros(B, **I32),
                 q=torch.zeros((B, M, Hq, D), dtype=torch.bfloat16, device="cuda"),
                 k=torch.zeros((B, M, Hkv, D), dtype=torch.bfloat16, device="cuda"),
                 out=torch.zeros((B, M, Hq, D), dtype=torch.bfloat16, device="cuda"), ws=dtree.attention_workspace(cache, M, Hq))
        s["grown"] = dtree.PagedCache4(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, s["new"])
        s["kv"] = [torch.zeros((B, M, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        return s

    def layer(s, x):
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        dtree.qk_norm(q, k, w, w, rope=rope, len=s["cache"].len, n_nodes=count, q_out=s["q"], k_out=s["k"], status=s["status"])
        dtree.tree_attention(s["cache"], s["q"], s["k"], v, n_nodes=count, out=s["out"], workspace=s["ws"], status=s["status"])
        dtree.kv_append(s["cache"], s["k"], v, count=count, len_out=s["new"], status=s["status"])
        dtree.kv_read(s["grown"], start=s["cache"].len, count=count, k=s["kv"][0], v=s["kv"][1], status=s["status"])

    def outcome(s):
        return [t.clone() for t in (s["q"], s["k"], s["out"], s["new"], *s["kv"], s["cache"].k, s["cache"].v,
                                    s["cache"].k_scale, s["cache"].v_scale)]

    xs = [torch.randn((B, M, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    a, b, buf = fresh(), fresh(), torch.zeros_like(xs[0])
    layer(a, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(a, buf)
    for x in xs:
        buf.copy_(x)
        graph.replay()
        layer(b, x)
        for y, z in zip(outcome(a), outcome(b)):
            assert torch.equal(y, z)
    assert not a["status"].any() and not b["status"].any()
    for i, n in enumerate(count.tolist()):  # what was appended is what the norms gave
        assert torch.equal(b["kv"][0][i, :n].double(), ref4.values4(*ref4.quantised(b["k"][i, :n].double())))


def test_calls_on_two_streams():
    """The same calls on streams of their own, many times over, change nothing of each other's results."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((8, 50, 12, 128), generator=g).to(torch.bfloat16).cuda()
    caches = [dtree.PagedCache4.empty(80, 16, 2, 128, 8, 10) for _ in range(2)]
    for c in caches:
        c.table.copy_(torch.arange(80).view(8, 10))
    k, v = x[:, :, 8:10], x[:, :, 10:]
    want = dtree.qk_norm(x[:, :, :8], k)
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for c, s in zip(caches, streams):
        with torch.cuda.stream(s):
            for _ in range(20):
                q1, k1 = dtree.qk_norm(x[:, :, :8], k)
                dtree.kv_append(c, k1, v)
                c2 = dtree.PagedCache4(c.k, c.v, c.k_scale, c.v_scale, c.table, torch.full_like(c.len, 50))
                kv = dtree.kv_read(c2, N=50)
            got.append((q1, k1, *kv))
    torch.cuda.synchronize()
    for q1, k1, kr, vr in got:
        assert torch.equal(q1, want[0]) and torch.equal(k1, want[1])
        for y, z in ((kr, k1), (vr, v)):
            assert torch.equal(y.double(), ref4.values4(*ref4.quantised(z.double())))


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another device."""

    def get_device(self):
        return 1 + super().get_device()


def test_tensors_on_another_device_are_refused():
    B, M, H, D = 1, 2, 2, 64
    x = torch.zeros((B, M, H, D), dtype=torch.bfloat16, device="cuda")
    one, mask = torch.ones(B, **I32), torch.zeros((B, M, 1), **I32)
    pos, w = torch.zeros((B, M), **I32), torch.ones(D, device="cuda")
    away = lambda t: t.as_subclass(Elsewhere)  # noqa: E731
    for kind in (dtree.PagedCache, dtree.PagedCache4):
        cache = kind.empty(2, 16, H, D, B, 2)
        ws, n = dtree.attention_workspace(cache, M, H)
        calls = [(dtree.kv_append, (cache, x, x), dict(rows=pos, count=one, len_out=one.clone(), status=one)),
                 (dtree.kv_read, (cache,), dict(rows=pos, count=one, status=one)),
                 (dtree.kv_read, (cache, 2), dict(start=one)),
                 (dtree.tree_attention, (cache, x, x, x), dict(mask=mask, pos=pos, n_nodes=one, out=x.clone(),
                                                               workspace=(ws, n), status=one)),
                 (dtree.qk_norm, (x, x), dict(q_weight=w, k_weight=w, len=one, pos=pos, n_nodes=one, status=one))]
        for call, args, kw in calls:
            for name, t in kw.items():
                t = (away(ws), n) if name == "workspace" else away(t)
                with pytest.raises(ValueError):
                    call(*args, **{**kw, name: t})
        f = dict(k=cache.k, v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale, table=cache.table, len=cache.len)
        for name, t in f.items():
            with pytest.raises(ValueError):
                kind(**{**f, name: away(t)})
