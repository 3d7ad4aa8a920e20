"""The target-side operators of one speculative round, as cases that can be timed and compared.

Three operators work together around the tree walk:

  attend    attention of the tree's rows over a paged e4m3 cache (a scale per page and head)
            and over the tree's own keys, under the ancestor mask;
  append    rotation, quantisation and storing of the accepted rows' keys and values;
  logprobs  log-probability, rank, entropy and top alternatives of given tokens.

`run` computes them with elementary torch operations in 32 bits when `own` is false, and with
the library's entry points when it is true.  `exact` is the same result in 64 bits.
"""
import math

import torch

own = False

LOG2_MIN = -48  # smallest exponent of a block scale
E4M3_MAX = 448.0
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attend(name, batch, nodes, Hq, Hkv, D, page, lo, hi, tree, rot=None, interleaved=False, fused=True):
    c = dict(op="attend", batch=batch, nodes=nodes, Hq=Hq, Hkv=Hkv, D=D, page=page, ctx_lo=lo, ctx_hi=hi, tree=tree,
             rot=D if rot is None else rot, interleaved=interleaved, fused=fused)
    return dict(c, name=name) if name else c


def _append(name, batch, nodes, count, Hkv, D, page, lo, hi, path, dtype="bf16", rot=None, interleaved=False):
    c = dict(op="append", batch=batch, nodes=nodes, count=count, Hkv=Hkv, D=D, page=page, ctx_lo=lo, ctx_hi=hi,
             path=path, dtype=dtype, rot=D if rot is None else rot, interleaved=interleaved)
    return dict(c, name=name) if name else c


def _logprobs(name, batch, nodes, count, V, top, path, dtype="bf16"):
    c = dict(op="logprobs", batch=batch, nodes=nodes, count=count, V=V, top=top, path=path, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request, one new token (a round whose tree is the root alone): latency
        _attend("attend_step_b1", 1, 1, 32, 8, 128, 64, 1000, 1000, False),
        # a full serving batch of single tokens over ragged contexts: bandwidth of the cache
        _attend("attend_step_b64", 64, 1, 32, 8, 128, 64, 1001, 16384, False),
        # one request's tree of 256 nodes over a long context
        _attend("attend_tree_b1_n257", 1, 257, 32, 8, 128, 64, 8000, 8000, True),
        # many requests with small trees, seven query heads to a key head, short pages
        _attend("attend_tree_b64_n61", 64, 61, 28, 4, 128, 16, 200, 4000, True, rot=64),
        # one key head per query head, narrow heads, interleaved rotation
        _attend("attend_tree_b8_n513_d64", 8, 513, 16, 16, 64, 32, 500, 2500, True, interleaved=True),
        # the stochastic batch: sixteen trees of 256 nodes over long contexts
        _attend("attend_tree_b16_n257", 16, 257, 64, 8, 128, 128, 5000, 16384, True),
        # the accepted path of four requests, fp32 activations
        _append("append_path_b4_f32", 4, 257, 17, 8, 128, 64, 700, 3000, True, dtype="f32"),
        # the accepted paths of a serving batch into short pages
        _append("append_path_b64", 64, 61, 17, 4, 128, 16, 200, 4000, True, rot=64, interleaved=True),
        # eight prompts of some thousand tokens that begin in the middle of a page
        _append("append_prompt_b8", 8, 4000, 4000, 8, 128, 64, 10, 600, False),
        # what one request emitted in a round
        _logprobs("logprobs_path_b1", 1, 257, 17, 151936, 5, True),
        # a batch's paths, fp32 logits of an odd vocabulary
        _logprobs("logprobs_path_b16_f32", 16, 65, 17, 50257, 20, True, dtype="f32"),
        # every position of a long prompt
        _logprobs("logprobs_prompt_4000", 1, 4000, 4000, 151936, 1, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "logprobs", "logprobs"])
    if op == "attend":
        while True:
            Hkv = rng.choice([1, 2, 4, 8, 16])
            G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            D = rng.choice([64, 128, 128])
            tree = rng.random() < 0.6
            nodes = _log_int(rng, 2, 1025) if tree else rng.choice([1, 1, _log_int(rng, 1, 600)])
            batch = _log_int(rng, 1, 64)
            hi = _log_int(rng, 1, 65536)
            lo = rng.randint(0, hi)
            rot = rng.choice([0, D // 2, D, D])
            c = _attend(None, batch, nodes, G * Hkv, Hkv, D, rng.choice([16, 32, 64, 128]), lo, hi, tree, rot,
                        rng.random() < 0.3, rng.random() < 0.5)
            if batch * Hkv * G * nodes * (hi + nodes) <= 2.5e9 and batch * hi * Hkv * D <= 7e8:
                return c
    if op == "append":
        while True:
            path = rng.random() < 0.5
            D = rng.choice([64, 128])
            nodes = _log_int(rng, 1, 1025 if path else 8000)
            count = min(nodes, rng.randint(1, 33)) if path else nodes
            hi = _log_int(rng, 1, 8000)
            c = _append(None, _log_int(rng, 1, 64), nodes, count, rng.choice([1, 2, 3, 4, 8, 16]), D,
                        rng.choice([16, 32, 64, 128]), rng.randint(0, hi), hi, path, rng.choice(["bf16", "bf16", "f32"]),
                        rng.choice([0, D // 2, D]), rng.random() < 0.3)
            if c["batch"] * c["nodes"] * c["Hkv"] * D <= 3.2e7 and c["batch"] * (hi + nodes) * c["Hkv"] * D <= 6e7:
                return c
    while True:
        path = rng.random() < 0.5
        nodes = _log_int(rng, 1, 300 if path else 4000)
        c = _logprobs(None, _log_int(rng, 1, 16), nodes, min(nodes, rng.randint(1, 17)) if path else nodes,
                      _log_int(rng, 1000, 151936), rng.randint(0, 20), path, rng.choice(["bf16", "bf16", "f32"]))
        if c["batch"] * nodes * c["V"] * (4 if c["dtype"] == "f32" else 2) <= 1.2e9:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(batch, lo, hi, salt):
    """`batch` whole numbers spread over [lo, hi], out of order; the last is hi.  They belong to the
    case, not to the seed, so that work() knows them."""
    if batch == 1:
        return [hi]
    at = [lo + (hi - lo) * i // (batch - 1) for i in range(batch)]
    step = next(s for s in (7, 5, 3, 11, 13, 1) if math.gcd(s, batch) == 1)
    return [at[(i * step + salt) % batch] for i in range(batch)][:batch]


def _lens(c):
    return _spread(c["batch"], c["ctx_lo"], c["ctx_hi"], 1)


def _sizes(c):
    """Rows in use per request: all of them for one request, from half on for a batch."""
    return _spread(c["batch"], (c["nodes"] + 1) // 2, c["nodes"], 3)


def _counts(c):
    return _spread(c["batch"], 1 if c["path"] else (c["count"] + 1) // 2, c["count"], 2)


def _gen(seed, salt=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale


def _rope(c, positions):
    """cos and sin tables [positions, rot / 2], or None."""
    if not c["rot"]:
        return None
    inv = 1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def _block_exponent(amax):
    """The smallest e >= LOG2_MIN with amax <= 448 * 2^e."""
    f, x = torch.frexp(amax)
    e = x.to(torch.int32) - torch.where(f <= 0.875, 9, 8)
    return torch.where(amax > 0, e, LOG2_MIN).clamp(min=LOG2_MIN)


def _pow2(e):
    """2^e in fp32, for -126 <= e <= 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _pool(c, n_pages, g):
    """Codes [n_pages, Hkv, page, D] (e4m3 bytes) and scales [n_pages, Hkv] of a filled cache:
    keys have a few strong channels, as trained models do."""
    Hkv, page, D = c["Hkv"], c["page"], c["D"]
    strong = 1.0 + 3.0 * (torch.rand((Hkv, 1, D), generator=g, device=DEV) < 0.05)
    out = []
    for width in (strong, torch.ones_like(strong)):
        codes = torch.empty((n_pages, Hkv, page, D), dtype=torch.uint8, device=DEV)
        scales = torch.empty((n_pages, Hkv), dtype=torch.float32, device=DEV)
        step = max(1, (1 << 27) // (Hkv * page * D))
        for i in range(0, n_pages, step):
            x = _randn((min(step, n_pages - i), Hkv, page, D), g) * width
            s = _pow2(_block_exponent(x.abs().amax((2, 3))))
            codes[i:i + step] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scales[i:i + step] = s
        out += [codes, scales]
    return out[0], out[2], out[1], out[3]


def _table(batch, max_pages, g):
    """Page tables in no order, and pages that no table names."""
    n = batch * max_pages + 3
    return torch.randperm(n, generator=g, device=DEV)[:batch * max_pages].to(torch.int32).view(batch, max_pages), n


def _trees(batch, nodes, sizes, seed):
    """Ancestor masks [batch, nodes, ceil(nodes / 32)] (bits) and depths [batch, nodes] of random
    trees of at most 16 levels whose parents come first."""
    g = torch.Generator()
    g.manual_seed(int(seed) + 17)
    level = torch.zeros((batch, nodes), dtype=torch.int64)
    anc = torch.zeros((batch, nodes, nodes), dtype=torch.bool)
    u = torch.rand((batch, nodes), generator=g)
    every = torch.arange(batch)
    anc[:, 0, 0] = True
    for i in range(1, nodes):
        up = (u[:, i].square() * i).long().clamp(max=i - 1)
        up = torch.where(level[every, up] >= 16, torch.zeros_like(up), up)
        level[:, i] = level[every, up] + 1
        anc[:, i] = anc[every, up]
        anc[:, i, i] = True
    words = (nodes + 31) // 32
    bits = torch.zeros((batch, nodes, words * 32), dtype=torch.int32, device=DEV)
    bits[:, :, :nodes] = anc.to(DEV)
    packed = (bits.view(batch, nodes, words, 32) << torch.arange(32, dtype=torch.int32, device=DEV)).sum(-1)
    packed = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
    return packed, level.to(torch.int32).to(DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "logprobs":
        x = torch.empty((c["batch"], c["nodes"], c["V"]), device=DEV,
                        dtype=torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
        flat = x.view(-1, c["V"])
        step = max(1, (1 << 27) // c["V"])
        for i in range(0, flat.shape[0], step):
            y = _randn((min(step, flat.shape[0] - i), c["V"]), g, 3.0)
            sure = torch.rand(y.shape[0], generator=g, device=DEV) < 0.7
            at = torch.randint(0, c["V"], (y.shape[0],), generator=g, device=DEV)
            y[torch.arange(y.shape[0], device=DEV), at] += 8.0 * sure
            y[:, -1] = -math.inf  # a token that the sampler has ruled out
            flat[i:i + step] = y
        s["logits"] = x
        counts = torch.tensor(_counts(c), device=DEV)
        used = torch.arange(c["count"], device=DEV)[None] < counts[:, None]
        if c["path"]:
            rows = torch.rand((c["batch"], c["nodes"]), generator=g, device=DEV).argsort(1)[:, :c["count"]].sort(1).values
            s["rows"] = torch.where(used, rows, -1).to(torch.int32)
        tok = torch.randint(0, c["V"], (c["batch"], c["count"]), generator=g, device=DEV)
        best = x.float().argmax(-1) if x.numel() < 1 << 28 else None
        if best is not None and c["path"]:  # most emitted tokens are likely ones
            likely = best.gather(1, s["rows"].clamp(min=0).long())
            tok = torch.where(torch.rand(tok.shape, generator=g, device=DEV) < 0.7, likely, tok)
        s["tokens"] = torch.where(used, tok, -1).to(torch.int32).contiguous()
        if own:
            from speculative_decoding_draft_bf16_gb300 import dtree
            s["out"] = dtree.alloc_logprobs(c["batch"], c["count"], c["top"])
        return s

    lens = _lens(c)
    grow = c["count"] if c["op"] == "append" else 0
    max_pages = max(1, -(-(c["ctx_hi"] + grow) // c["page"]))
    s["table"], n_pages = _table(c["batch"], max_pages, g)
    s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"] = _pool(c, n_pages, g)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rope = _rope(c, c["ctx_hi"] + c["nodes"] + 1)
    if rope:
        s["cos"], s["sin"] = rope
    B, M, Hkv, D = c["batch"], c["nodes"], c["Hkv"], c["D"]
    if c["op"] == "append":
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        kv = _randn((B, M, 2 * Hkv, D), g, 1.5).to(dt)
        s["k"], s["v"] = kv[:, :, :Hkv], kv[:, :, Hkv:]
        s["count"] = torch.tensor(_counts(c), dtype=torch.int32, device=DEV)
        if c["path"]:
            rows = torch.rand((B, M), generator=g, device=DEV).argsort(1)[:, :c["count"]].sort(1).values
            used = torch.arange(c["count"], device=DEV)[None] < s["count"][:, None]
            s["rows"] = torch.where(used, rows, -1).to(torch.int32).contiguous()
        s["len_out"] = torch.zeros_like(s["len"])
    else:
        Hq = c["Hq"]
        qkv = _randn((B, M, Hq + 2 * Hkv, D), g).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        if not c["fused"]:
            s["q"], s["k"], s["v"] = s["q"].contiguous(), s["k"].contiguous(), s["v"].contiguous()
        s["n_nodes"] = torch.tensor(_sizes(c), dtype=torch.int32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(D)
        if c["tree"]:
            s["mask"], s["pos"] = _trees(B, M, _sizes(c), seed)
    if own:
        from speculative_decoding_draft_bf16_gb300 import dtree
        s["cache"] = dtree.PagedCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"], s["len"])
        s["rope"] = dtree.Rope(s["cos"], s["sin"], c["interleaved"]) if rope else None
        s["status"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
        if c["op"] == "attend":
            s["out"] = torch.empty((B, M, c["Hq"], D), dtype=torch.bfloat16, device=DEV)
            s["workspace"] = dtree.attention_workspace(s["cache"], M, c["Hq"])
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _turn(x, c, cos, sin):
    """The rotation of x [..., D]; cos, sin broadcast over its rows."""
    r = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return y if r == x.shape[-1] else torch.cat((y, x[..., r:]), -1)


def _plain_attend(s):
    c = s["case"]
    B, M, Hq, Hkv, D = c["batch"], c["nodes"], c["Hq"], c["Hkv"], c["D"]
    G, S = Hq // Hkv, s["table"].shape[1] * c["page"]
    t = s["table"].long()

    def held(codes, scale):  # [B, Hkv, S, D]
        x = codes[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, S, D)

    node = torch.arange(M, device=DEV)
    depth = s["pos"] if c["tree"] else node[None].expand(B, M)
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["rot"]:
        at = (s["len"][:, None] + depth).long().clamp(max=s["cos"].shape[0] - 1)
        cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
        q, k = _turn(q, c, cos, sin), _turn(k, c, cos, sin)
    q = q.view(B, M, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * M, D) * s["scale"]
    k, v = k.transpose(1, 2), v.transpose(1, 2)
    live = node[None] < s["n_nodes"][:, None]
    if c["tree"]:
        sees = ((s["mask"][:, :, node // 32] >> (node % 32)) & 1).bool()
    else:
        sees = (node[None, :] <= node[:, None])[None].expand(B, M, M)
    sees = sees & live[:, None, :]
    old = torch.matmul(q, held(s["k_codes"], s["k_scale"]).transpose(2, 3))
    old.masked_fill_((torch.arange(S, device=DEV)[None] >= s["len"][:, None])[:, None, None], -math.inf)
    new = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, M, M).masked_fill(~sees[:, None, None], -math.inf)
    new = new.view(B, Hkv, G * M, M)
    top = torch.maximum(old.amax(-1), new.amax(-1))[..., None]
    top = torch.where(top == -math.inf, 0.0, top)
    old, new = old.sub_(top).exp_(), new.sub_(top).exp_()
    total = old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True)
    out = torch.matmul(old, held(s["v_codes"], s["v_scale"])) + torch.matmul(new, v)
    out = torch.where(total > 0, out / total, 0.0)
    out = out.view(B, Hkv, G, M, D).permute(0, 3, 1, 2, 4).reshape(B, M, Hq, D)
    return (out * live[:, :, None, None]).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    B, Hkv, D, page, N = c["batch"], c["Hkv"], c["D"], c["page"], c["count"]
    j = torch.arange(N, device=DEV)[None]
    start, count = s["len"].long()[:, None], s["count"].long()[:, None]
    used = j < count
    rows = s["rows"].long().clamp(min=0) if c["path"] else j.expand(B, N)
    k = s["k"].gather(1, rows[:, :, None, None].expand(B, N, Hkv, D)).float()
    v = s["v"].gather(1, rows[:, :, None, None].expand(B, N, Hkv, D)).float()
    if c["rot"]:
        at = (start + j).clamp(max=s["cos"].shape[0] - 1)
        k = _turn(k, c, s["cos"][at][:, :, None], s["sin"][at][:, :, None])
    # the pages from the first one written on, as slots: what they hold, then the new rows
    P = -(-(N + page - 1) // page) if N > 1 else 1
    first = start // page
    pages = first + torch.arange(P, device=DEV)[None]                    # [B, P] logical pages
    touched = pages * page < start + count
    ids = s["table"].gather(1, pages.clamp(max=s["table"].shape[1] - 1)).long()
    slot = pages[:, :, None] * page + torch.arange(page, device=DEV)     # [B, P, page] positions
    fresh = (slot >= start[:, :, None]) & (slot < (start + count)[:, :, None])
    kept = slot < start[:, :, None]
    src = (slot - start[:, :, None]).clamp(0, N - 1).view(B, P * page)
    for x, codes, scales in ((k, s["k_codes"], s["k_scale"]), (v, s["v_codes"], s["v_scale"])):
        y = x.gather(1, src[:, :, None, None].expand(B, P * page, Hkv, D))
        y = y.view(B, P, page, Hkv, D).transpose(2, 3) * fresh[:, :, None, :, None]
        e = _block_exponent(y.abs().amax((3, 4)))                        # [B, P, Hkv]
        had = torch.frexp(scales[ids])[1].to(torch.int32) - 1
        e = torch.where(kept.any(2)[:, :, None], torch.maximum(e, had), e)
        old = codes[ids].view(torch.float8_e4m3fn).float() * _pow2(had - e)[..., None, None]
        z = torch.where(fresh[:, :, None, :, None], y / _pow2(e)[..., None, None], old).to(torch.float8_e4m3fn)
        # slots past the new rows keep their bytes
        z = torch.where((fresh | kept)[:, :, None, :, None], z.view(torch.uint8), codes[ids])
        codes[ids[touched]] = z[touched]
        scales[ids[touched]] = _pow2(e)[touched]
    s["len_out"].copy_(s["len"] + s["count"])
    return _append_out(s)


def _append_out(s):
    return {"k": s["k_codes"].view(torch.float8_e4m3fn), "v": s["v_codes"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"], "len": s["len_out"]}


def _plain_logprobs(s):
    c = s["case"]
    x, tok = s["logits"], s["tokens"].long()
    used = s["rows"] >= 0 if c["path"] else torch.ones_like(tok, dtype=torch.bool)
    if c["path"]:
        x = x.gather(1, s["rows"].long().clamp(min=0)[:, :, None].expand(-1, -1, c["V"]))
    x = x.float()
    top = x.amax(-1, keepdim=True)
    y = x - top
    e = y.exp()
    z = e.sum(-1)
    lse = top[..., 0] + z.log()
    entropy = z.log() - torch.where(e > 0, y * e, 0.0).sum(-1) / z
    named = used & (tok >= 0)
    at = x.gather(-1, tok.clamp(min=0)[..., None])
    ids = torch.arange(c["V"], device=DEV)
    rank = ((x > at) | ((x == at) & (ids < tok[..., None]))).sum(-1)
    out = {"logprob": torch.where(named, at[..., 0] - lse, 0.0), "entropy": torch.where(used, entropy, 0.0),
           "rank": torch.where(named, rank, -1).to(torch.int32)}
    if c["top"]:
        best, order = torch.sort(x, dim=-1, descending=True, stable=True)
        best, order = best[..., :c["top"]], order[..., :c["top"]]
        out["top_id"] = torch.where(used[..., None], order, -1).to(torch.int32)
        out["top_logprob"] = torch.where(used[..., None], best - lse[..., None], 0.0)
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "logprobs": _plain_logprobs}[c["op"]](s)
    from speculative_decoding_draft_bf16_gb300 import dtree
    if c["op"] == "attend":
        return dtree.tree_attention(s["cache"], s["q"], s["k"], s["v"], mask=s.get("mask"), pos=s.get("pos"),
                                    n_nodes=s["n_nodes"], rope=s["rope"], scale=s["scale"], out=s["out"],
                                    workspace=s["workspace"], status=s["status"])
    if c["op"] == "append":
        dtree.kv_append(s["cache"], s["k"], s["v"], rope=s["rope"], rows=s.get("rows"), count=s["count"],
                        len_out=s["len_out"], status=s["status"])
        return _append_out(s)
    o = dtree.token_logprobs(s["logits"], s["tokens"], top=c["top"], rows=s.get("rows"), out=s["out"])
    got = {"logprob": o.logprob, "entropy": o.entropy, "rank": o.rank}
    if c["top"]:
        got |= {"top_id": o.top_id, "top_logprob": o.top_logprob}
    return got


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "logprobs":
        n = sum(_counts(c)) if c["path"] else c["batch"] * c["count"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * (c["V"] * size + 16 + 8 * c["top"]), "flops": 6 * n * c["V"]}
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] == "append":
        n, size = sum(_counts(c)), 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * Hkv * D * 2 * (size + 1) + n * c["rot"] * 4, "flops": n * Hkv * (3 * c["rot"] + 4 * D)}
    Hq, lens, sizes = c["Hq"], _lens(c), _sizes(c)
    seen = sum(n * min(n, 8) if c["tree"] else n * (n + 1) // 2 for n in sizes)
    pairs = sum(n * m for n, m in zip(sizes, lens)) + seen
    bytes_ = sum(m * Hkv * D * 2 + -(-m // c["page"]) * Hkv * 8 for m in lens)
    bytes_ += sum(n * (2 * Hq + 2 * Hkv) * D * 2 + n * c["rot"] * 4 for n in sizes)
    if c["tree"]:
        bytes_ += sum(n * ((c["nodes"] + 31) // 32) * 4 for n in sizes)
    return {"bytes": bytes_, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one request at a time
# ---------------------------------------------------------------------------

def _e4m3_value(b):
    """Values of e4m3 bytes: sign, four exponent bits (bias 7), three of the fraction."""
    b = b.to(torch.int64)
    e, f = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).double()))
    return torch.where(b >= 128, -mag, mag)


def _e4m3_round(x):
    """The e4m3 value nearest to x (|x| <= 448), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _turn_exact(x, c, s, at):
    """Rotation of x [n, H, D] to the positions `at`: each pair as a complex number."""
    r = c["rot"]
    if not r:
        return x
    turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
    first, second = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_attend(c, s):
    out = torch.zeros((c["batch"], c["nodes"], c["Hq"], c["D"]), dtype=torch.float64, device=DEV)
    G = c["Hq"] // c["Hkv"]
    for b in range(c["batch"]):
        n, m = int(s["n_nodes"][b]), int(s["len"][b])
        depth = s["pos"][b, :n].long() if c["tree"] else torch.arange(n, device=DEV)
        q = _turn_exact(s["q"][b, :n].double(), c, s, m + depth)
        k = _turn_exact(s["k"][b, :n].double(), c, s, m + depth)
        v = s["v"][b, :n].double()
        ids = s["table"][b, :-(-m // c["page"])].long()
        sees = torch.ones((n, m + n), dtype=torch.bool, device=DEV)
        col = torch.arange(n, device=DEV)
        if c["tree"]:
            sees[:, m:] = ((s["mask"][b, :n].long()[:, col // 32] >> (col % 32)) & 1).bool()
        else:
            sees[:, m:] = col[None, :] <= col[:, None]
        for h in range(c["Hkv"]):
            kc = (_e4m3_value(s["k_codes"][ids, h]) * s["k_scale"][ids, h].double()[:, None, None]).view(-1, c["D"])[:m]
            vc = (_e4m3_value(s["v_codes"][ids, h]) * s["v_scale"][ids, h].double()[:, None, None]).view(-1, c["D"])[:m]
            kh, vh = torch.cat((kc, k[:, h])), torch.cat((vc, v[:, h]))
            for i in range(h * G, h * G + G):
                z = (q[:, i] @ kh.T * s["scale"]).masked_fill(~sees, -math.inf)
                p = torch.softmax(z, -1)
                out[b, :n, i] = torch.where(sees.any(-1, keepdim=True), p, 0.0) @ vh
    return out


def _exact_append(c, s):
    names = (("k_codes", "k_scale"), ("v_codes", "v_scale"))
    got = {n: (_e4m3_value(s[n]) if i == 0 else s[n].double()) for pair in names for i, n in enumerate(pair)}
    page = c["page"]
    for b in range(c["batch"]):
        m, n = int(s["len"][b]), int(s["count"][b])
        rows = s["rows"][b, :n].long() if c["path"] else torch.arange(n, device=DEV)
        k = _turn_exact(s["k"][b][rows].double(), c, s, m + torch.arange(n, device=DEV))
        v = s["v"][b][rows].double()
        for p in range(m // page, (m + n - 1) // page + 1):
            at = int(s["table"][b, p])
            lo, hi = max(m, p * page), min(m + n, (p + 1) * page)
            for x, (codes, scale) in zip((k, v), names):
                y = x[lo - m:hi - m].transpose(0, 1)                     # [Hkv, rows, D]
                top = y.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / E4M3_MAX))
                e = (e - (top <= E4M3_MAX * torch.exp2(e - 1)).double()).clamp(min=LOG2_MIN)  # log2 may round up
                f = got[scale][at]
                if m > p * page:
                    e = torch.maximum(e, torch.log2(f))
                    got[codes][at, :, :lo - p * page] = _e4m3_round(
                        got[codes][at, :, :lo - p * page] * (f / torch.exp2(e))[:, None, None])
                got[codes][at, :, lo - p * page:hi - p * page] = _e4m3_round(y / torch.exp2(e)[:, None, None])
                got[scale][at] = torch.exp2(e)
    return {"k": got["k_codes"], "v": got["v_codes"], "k_scale": got["k_scale"], "v_scale": got["v_scale"], "len": None}


def _exact_logprobs(c, s):
    B, N, top = c["batch"], c["count"], c["top"]
    zero = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
    out = {"logprob": zero(B, N), "entropy": zero(B, N), "rank": None}
    if top:
        out |= {"top_id": None, "top_logprob": zero(B, N, top)}
    for b in range(B):
        for i in range(0, N, 256):
            r = s["rows"][b, i:i + 256].long() if c["path"] else torch.arange(i, min(N, i + 256), device=DEV)
            ok = r >= 0
            t = s["tokens"][b, i:i + 256].long()
            lp = torch.log_softmax(s["logits"][b][r.clamp(min=0)].double(), -1)
            p = lp.exp()
            out["logprob"][b, i:i + 256] = torch.where(t >= 0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
            out["entropy"][b, i:i + 256] = torch.where(ok, -torch.where(p > 0, p * lp, 0.0).sum(-1), 0.0)
            if top:
                out["top_logprob"][b, i:i + 256] = torch.where(ok[:, None], lp.topk(top).values, 0.0)
    return out


def exact(case, seed):
    c = case
    if c["op"] == "attend" and c["batch"] * c["Hq"] * c["nodes"] * (c["ctx_hi"] + c["nodes"]) * c["D"] > 1e12:
        return None
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "logprobs": _exact_logprobs}[c["op"]](c, s)
