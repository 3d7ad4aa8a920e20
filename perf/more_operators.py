"""The operators of a target model with normalised heads and a 4-bit cache, as cases that can be
timed and compared.

Four operators follow one another in each of the model's layers:

  norm     root-mean-square norms of every query and key head, with the position rotation;
  attend   attention of the tree's rows over a paged cache in 4 bits (e2m1 codes, a scale for each
           16 elements) and over the tree's own keys, under the ancestor mask;
  append   rotation, quantisation to 4 bits and storing of accepted rows, which a drafter that
           works on the target's keys and values then reads back;
  read     reading back a cache, in 4 bits or in 8: ranges of tokens, or picked ones.

`run` computes them with elementary torch operations in 32 bits when `own` is false, and with
the library's entry points when it is true.  `exact` is the same result in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP_SCALE = 226     # byte of the largest scale, 10240: six times it is in fp16's range
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, batch, nodes, Hq, Hkv, D, lo, hi, tree, dtype="bf16", rot=None, interleaved=False, heads=False):
    c = dict(op="norm", batch=batch, nodes=nodes, Hq=Hq, Hkv=Hkv, D=D, ctx_lo=lo, ctx_hi=hi, tree=tree, dtype=dtype,
             rot=D if rot is None else rot, interleaved=interleaved, heads=heads)
    return dict(c, name=name) if name else c


def _attend(name, batch, nodes, Hq, Hkv, D, page, lo, hi, tree, fused=True):
    c = dict(op="attend", batch=batch, nodes=nodes, Hq=Hq, Hkv=Hkv, D=D, page=page, ctx_lo=lo, ctx_hi=hi, tree=tree,
             fused=fused)
    return dict(c, name=name) if name else c


def _append(name, batch, nodes, count, Hkv, D, page, lo, hi, path, dtype="bf16", rot=None, interleaved=False):
    c = dict(op="append", batch=batch, nodes=nodes, count=count, Hkv=Hkv, D=D, page=page, ctx_lo=lo, ctx_hi=hi,
             path=path, dtype=dtype, rot=D if rot is None else rot, interleaved=interleaved)
    return dict(c, name=name) if name else c


def _read(name, batch, count, Hkv, D, page, lo, hi, picked, bits=4, dtype="bf16"):
    c = dict(op="read", batch=batch, count=count, Hkv=Hkv, D=D, page=page, ctx_lo=lo, ctx_hi=hi, picked=picked,
             bits=bits, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # every request of a serving batch with one new token: latency
        _norm("norm_step_b64", 64, 1, 32, 8, 128, 1001, 16384, False),
        # sixteen trees of 256 nodes, fp32 activations, half of a head rotated, weights of each head
        _norm("norm_tree_b16_n257_f32", 16, 257, 28, 4, 128, 5000, 16384, True, dtype="f32", rot=64, heads=True),
        # eight prompts of some thousand tokens
        _norm("norm_prompt_b8", 8, 4000, 32, 8, 128, 0, 600, False),
        # one request, one new token: latency
        _attend("attend_step_b1", 1, 1, 32, 8, 128, 64, 1000, 1000, False),
        # a full serving batch of single tokens over ragged contexts: bandwidth of the cache
        _attend("attend_step_b64", 64, 1, 32, 8, 128, 64, 1001, 16384, False),
        # many requests with small trees, seven query heads to a key head, short pages
        _attend("attend_tree_b64_n61", 64, 61, 28, 4, 128, 16, 200, 4000, True),
        # one key head per query head, narrow heads
        _attend("attend_tree_b8_n513_d64", 8, 513, 16, 16, 64, 32, 500, 2500, True, fused=False),
        # the stochastic batch: sixteen trees of 256 nodes over long contexts
        _attend("attend_tree_b16_n257", 16, 257, 64, 8, 128, 128, 5000, 16384, True),
        # the accepted paths of a serving batch into short pages, back for the drafter
        _append("append_path_b64", 64, 61, 17, 4, 128, 16, 200, 4000, True, rot=64, interleaved=True),
        # eight prompts that begin in the middle of a page
        _append("append_prompt_b8", 8, 4000, 4000, 8, 128, 64, 10, 600, False),
        # the tokens that a drafter with a short memory keeps, fp32, from a cache in 8 bits
        _read("read_picked_b16_e4m3_f32", 16, 129, 8, 64, 32, 500, 9000, True, bits=8, dtype="f32"),
        # whole contexts that move to another server
        _read("read_context_b8", 8, 8000, 8, 128, 64, 500, 8000, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "attend", "attend", "append", "read"])
    while True:
        c = _drawn(rng, op)
        w = work(c)
        if w["bytes"] <= 6.4e8 and w["flops"] <= 1.1e12:
            return c


def _drawn(rng, op):
    D, page, batch = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), _log_int(rng, 1, 64)
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    dtype, rot, interleaved = rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, D // 2, D, D]), rng.random() < 0.3
    if op == "norm":
        tree = rng.random() < 0.6
        hi = _log_int(rng, 1, 65536)
        return _norm(None, batch, _log_int(rng, 2, 1025) if tree else _log_int(rng, 1, 8000), G * Hkv, Hkv, D,
                     rng.randint(0, hi), hi, tree, dtype, rot, interleaved, rng.random() < 0.3)
    if op == "attend":
        while True:
            tree = rng.random() < 0.6
            nodes = _log_int(rng, 2, 1025) if tree else rng.choice([1, 1, _log_int(rng, 1, 600)])
            hi = _log_int(rng, 1, 65536)
            if batch * Hkv * G * nodes * (hi + nodes) <= 2.5e9 and batch * hi * Hkv * D <= 7e8:
                return _attend(None, batch, nodes, G * Hkv, Hkv, D, page, rng.randint(0, hi), hi, tree,
                               rng.random() < 0.5)
    if op == "append":
        path = rng.random() < 0.5
        nodes = _log_int(rng, 1, 1025 if path else 8000)
        hi = _log_int(rng, 1, 8000)
        return _append(None, batch, nodes, min(nodes, rng.randint(1, 33)) if path else nodes, Hkv, D, page,
                       rng.randint(0, hi), hi, path, dtype, rot, interleaved)
    picked = rng.random() < 0.5
    hi = _log_int(rng, 1, 16384)
    return _read(None, batch, _log_int(rng, 1, 600) if picked else hi, Hkv, D, page, rng.randint(1, hi), hi, picked,
                 rng.choice([4, 4, 8]), dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(batch, lo, hi, salt):
    """`batch` whole numbers spread over [lo, hi], out of order; one alone is hi.  They belong to the
    case, not to the seed, so that work() knows them."""
    if batch == 1:
        return [hi]
    at = [lo + (hi - lo) * i // (batch - 1) for i in range(batch)]
    step = next(s for s in (7, 5, 3, 11, 13, 1) if math.gcd(s, batch) == 1)
    return [at[(i * step + salt) % batch] for i in range(batch)]


def _lens(c):
    return _spread(c["batch"], c["ctx_lo"], c["ctx_hi"], 1)


def _sizes(c):
    """Rows in use per request: all of them for one request, from half on for a batch."""
    return _spread(c["batch"], (c["nodes"] + 1) // 2, c["nodes"], 3)


def _counts(c):
    """Rows appended, or read."""
    if c["op"] == "read":
        return _spread(c["batch"], (c["count"] + 1) // 2, c["count"], 2) if c["picked"] else _lens(c)
    return _spread(c["batch"], 1 if c["path"] else (c["count"] + 1) // 2, c["count"], 2)


def _gen(seed, salt=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rope(c, positions):
    """cos and sin tables [positions, rot / 2], or None."""
    if not c["rot"]:
        return None
    inv = 1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def _scales():
    """The scales that bytes 1 to TOP_SCALE stand for: the upper halves of fp16 numbers."""
    return (torch.arange(1, TOP_SCALE + 1, device=DEV, dtype=torch.int32) << 7).to(torch.int16).view(torch.float16).float()


def _to4(x):
    """Codes [..., D / 2] and scale bytes [..., D / 16] of x [..., D]: of each 16 elements the smallest
    scale with the largest magnitude within 6 of it, elements over the scale to the nearest of e2m1."""
    y = x.unflatten(-1, (-1, 16))
    table = _scales()
    at = torch.searchsorted(table * 6.0, y.abs().amax(-1).contiguous()).clamp(max=TOP_SCALE - 1)
    a = y / table[at][..., None]
    n = torch.signbit(a).to(torch.uint8) * 8
    a = a.abs()
    for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        n += (a >= edge) if up else (a > edge)
    n = n.flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), (at + 1).to(torch.uint8)


def _from4(codes, scales):
    """Values [..., D] of codes [..., D / 2] and scale bytes [..., D / 16], fp32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    s = (scales.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()
    return (lut[n.int()].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _block_exponent(amax):
    """The smallest e >= -48 with amax <= 448 * 2^e."""
    f, x = torch.frexp(amax)
    e = x.to(torch.int32) - torch.where(f <= 0.875, 9, 8)
    return torch.where(amax > 0, e, -48).clamp(min=-48)


def _pool(c, n_pages, g):
    """A filled cache: codes and scales of keys, of values.  Keys have a few strong channels, as
    trained models do."""
    Hkv, page, D, eight = c["Hkv"], c["page"], c["D"], c.get("bits") == 8
    strong = 1.0 + 3.0 * (torch.rand((Hkv, 1, D), generator=g, device=DEV) < 0.05)
    out = []
    for width in (strong, torch.ones_like(strong)):
        codes = torch.empty((n_pages, Hkv, page, D if eight else D // 2), dtype=torch.uint8, device=DEV)
        scales = torch.empty((n_pages, Hkv), device=DEV) if eight else \
            torch.empty((n_pages, Hkv, page, D // 16), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 27) // (Hkv * page * D))
        for i in range(0, n_pages, step):
            x = _randn((min(step, n_pages - i), Hkv, page, D), g) * width
            if eight:
                s = torch.exp2(_block_exponent(x.abs().amax((2, 3))).float())
                codes[i:i + step] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                scales[i:i + step] = s
            else:
                codes[i:i + step], scales[i:i + step] = _to4(x)
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


def _depths(batch, nodes, g):
    """Positions of a tree's nodes below its root, as a norm needs them."""
    d = torch.randint(1, 17, (batch, nodes), generator=g, device=DEV, dtype=torch.int32)
    d[:, 0] = 0
    return d


def _picked(batch, count, counts, among, g):
    """Distinct numbers below among[b] in rising order, counts[b] of them, -1 behind.  Where there are
    too few, some come again."""
    rows = torch.full((batch, count), -1, dtype=torch.int32, device=DEV)
    for b, (n, m) in enumerate(zip(counts, among)):
        at = torch.randperm(m, generator=g, device=DEV)
        rows[b, :n] = at[torch.arange(n, device=DEV) % m].sort().values.to(torch.int32)
    return rows


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    B, Hkv, D = c["batch"], c["Hkv"], c["D"]
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    s["len"] = _ints(_lens(c))
    if c.get("rot"):
        s["cos"], s["sin"] = _rope(c, c["ctx_hi"] + c["nodes"] + 17)
    if c["op"] == "norm":
        M, Hq = c["nodes"], c["Hq"]
        qkv = _randn((B, M, Hq + 2 * Hkv, D), g, 2.0).to(dt)
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        s["eps"] = 1e-6
        s["q_weight"] = 1.0 + _randn((Hq, D) if c["heads"] else (D,), g, 0.2)
        s["k_weight"] = 1.0 + _randn((Hkv, D) if c["heads"] else (D,), g, 0.2)
        s["pos"] = _depths(B, M, g) if c["tree"] else None
        s["q_out"] = torch.zeros((B, M, Hq, D), dtype=dt, device=DEV)
        s["k_out"] = torch.zeros((B, M, Hkv, D), dtype=dt, device=DEV)
        s["n_nodes"] = _ints(_sizes(c))
    else:
        grow = c["count"] if c["op"] == "append" else 0
        s["table"], n_pages = _table(B, max(1, -(-(c["ctx_hi"] + grow) // c["page"])), g)
        s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"] = _pool(c, n_pages, g)
    if c["op"] == "append":
        kv = _randn((B, c["nodes"], 2 * Hkv, D), g, 1.5).to(dt)
        s["k"], s["v"] = kv[:, :, :Hkv], kv[:, :, Hkv:]
        s["count"] = _ints(_counts(c))
        if c["path"]:
            s["rows"] = _picked(B, c["count"], _counts(c), [c["nodes"]] * B, g)
        s["len_out"] = torch.zeros_like(s["len"])
    if c["op"] == "read":
        s["count"] = _ints(_counts(c))
        if c["picked"]:
            s["rows"] = _picked(B, c["count"], _counts(c), _lens(c), g)
    if c["op"] in ("append", "read"):
        out = torch.bfloat16 if c["op"] == "append" else dt
        s["k_out"] = torch.zeros((B, c["count"], Hkv, D), dtype=out, device=DEV)
        s["v_out"] = torch.zeros((B, c["count"], Hkv, D), dtype=out, device=DEV)
    if c["op"] == "attend":
        M, Hq = c["nodes"], c["Hq"]
        qkv = _randn((B, M, Hq + 2 * Hkv, D), g).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        if not c["fused"]:
            s["q"], s["k"], s["v"] = s["q"].contiguous(), s["k"].contiguous(), s["v"].contiguous()
        s["n_nodes"] = _ints(_sizes(c))
        s["scale"] = 1.0 / math.sqrt(D)
        if c["tree"]:
            s["mask"], s["pos"] = _trees(B, M, _sizes(c), seed)
    if own:
        from speculative_decoding_draft_bf16_gb300 import dtree
        s["rope"] = dtree.Rope(s["cos"], s["sin"], c["interleaved"]) if c.get("rot") else None
        s["status"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
        if c["op"] != "norm":
            form = dtree.PagedCache if c.get("bits") == 8 else dtree.PagedCache4
            held = (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"])
            s["cache"] = form(*held, s["len"])
            if c["op"] == "append":
                s["grown"] = form(*held, s["len_out"])
        if c["op"] == "attend":
            s["out"] = torch.empty((B, c["nodes"], c["Hq"], D), dtype=torch.bfloat16, device=DEV)
            s["workspace"] = dtree.attention_workspace(s["cache"], c["nodes"], c["Hq"])
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


def _plain_norm(s):
    c = s["case"]
    node = torch.arange(c["nodes"], device=DEV)
    at = (s["len"][:, None] + (s["pos"] if c["tree"] else node[None])).long()
    live = (node[None] < s["n_nodes"][:, None])[:, :, None, None]
    for x, w, out in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        y = x.float()
        y = y * ((y * y).sum(-1, keepdim=True) / c["D"] + s["eps"]).rsqrt() * w
        if c["rot"]:
            y = _turn(y, c, s["cos"][at][:, :, None], s["sin"][at][:, :, None])
        out.copy_(torch.where(live, y, out.float()))  # rows behind the last node stay
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_attend(s):
    c = s["case"]
    B, M, Hq, Hkv, D = c["batch"], c["nodes"], c["Hq"], c["Hkv"], c["D"]
    G, S = Hq // Hkv, s["table"].shape[1] * c["page"]
    t = s["table"].long()

    def held(codes, scale):  # [B, Hkv, S, D]
        return _from4(codes[t], scale[t]).transpose(1, 2).reshape(B, Hkv, S, D)

    node = torch.arange(M, device=DEV)
    q, k, v = s["q"].float(), s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    q = q.view(B, M, Hkv, G, D) if q.is_contiguous() else q.unflatten(2, (Hkv, G))
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * M, D) * s["scale"]
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


def _slots(s, at):
    """Physical page and slot of the tokens `at` [B, N]."""
    page = s["case"]["page"]
    ids = s["table"].gather(1, (at // page).clamp(max=s["table"].shape[1] - 1)).long()
    return ids, at % page


def _plain_read_rows(s, at, used):
    """The tokens `at` [B, N] into k_out and v_out, where `used`."""
    ids, slot = _slots(s, at)
    for codes, scale, out in ((s["k_codes"], s["k_scale"], s["k_out"]), (s["v_codes"], s["v_scale"], s["v_out"])):
        x = codes[ids, :, slot]                                                # [B, N, Hkv, D or D / 2]
        if s["case"].get("bits") == 8:
            y = x.view(torch.float8_e4m3fn).float() * scale[ids][..., None]
        else:
            y = _from4(x, scale[ids, :, slot])
        out.copy_(torch.where(used[:, :, None, None], y, out.float()))


def _plain_append(s):
    c = s["case"]
    B, Hkv, D, N = c["batch"], c["Hkv"], c["D"], c["count"]
    j = torch.arange(N, device=DEV)[None]
    used = j < s["count"][:, None]
    at = s["len"].long()[:, None] + j
    rows = s["rows"].long().clamp(min=0) if c["path"] else j.expand(B, N)
    k, v = (s[n].gather(1, rows[:, :, None, None].expand(B, N, Hkv, D)).float() for n in ("k", "v"))
    if c["rot"]:
        k = _turn(k, c, s["cos"][at][:, :, None], s["sin"][at][:, :, None])
    ids, slot = _slots(s, at)
    for x, codes, scale in ((k, s["k_codes"], s["k_scale"]), (v, s["v_codes"], s["v_scale"])):
        n, f = _to4(x)
        codes[ids[used], :, slot[used]] = n[used]
        scale[ids[used], :, slot[used]] = f[used]
    s["len_out"].copy_(s["len"] + s["count"])
    _plain_read_rows(s, at, used)
    return _append_out(s)


def _append_out(s):
    """What the new rows stand for, and the whole cache's bytes, the other rows' among them."""
    return {"k": s["k_out"], "v": s["v_out"], "len": s["len_out"], "k_codes": s["k_codes"], "v_codes": s["v_codes"],
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_read(s):
    c = s["case"]
    j = torch.arange(c["count"], device=DEV)[None]
    used = j < s["count"][:, None]
    at = s["rows"].long().clamp(min=0) if c["picked"] else j.expand(c["batch"], -1)
    _plain_read_rows(s, at, used)
    return {"k": s["k_out"], "v": s["v_out"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "attend": _plain_attend, "append": _plain_append, "read": _plain_read}[c["op"]](s)
    from speculative_decoding_draft_bf16_gb300 import dtree
    if c["op"] == "norm":
        dtree.qk_norm(s["q"], s["k"], s["q_weight"], s["k_weight"], eps=s["eps"], rope=s["rope"], len=s["len"],
                      pos=s["pos"], n_nodes=s["n_nodes"], q_out=s["q_out"], k_out=s["k_out"], status=s["status"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "attend":
        return dtree.tree_attention(s["cache"], s["q"], s["k"], s["v"], mask=s.get("mask"), n_nodes=s["n_nodes"],
                                    scale=s["scale"], out=s["out"], workspace=s["workspace"], status=s["status"])
    if c["op"] == "append":
        dtree.kv_append(s["cache"], s["k"], s["v"], rope=s["rope"], rows=s.get("rows"), count=s["count"],
                        len_out=s["len_out"], status=s["status"])
        dtree.kv_read(s["grown"], start=s["len"], count=s["count"], k=s["k_out"], v=s["v_out"], status=s["status"])
        return _append_out(s)
    dtree.kv_read(s["cache"], rows=s.get("rows"), count=s["count"], k=s["k_out"], v=s["v_out"], status=s["status"])
    return {"k": s["k_out"], "v": s["v_out"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    Hkv, D = c["Hkv"], c["D"]
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "norm":
        n, heads = sum(_sizes(c)), c["Hq"] + Hkv
        return {"bytes": n * heads * D * size * 2 + n * c["rot"] * 4, "flops": n * heads * (4 * D + 3 * c["rot"])}
    held = D if c.get("bits") == 8 else D // 2 + D // 16   # bytes of a token's keys in a head
    if c["op"] == "read":
        n = sum(_counts(c))
        return {"bytes": n * Hkv * 2 * (held + D * size), "flops": n * Hkv * 2 * D}
    if c["op"] == "append":
        n = sum(_counts(c))
        return {"bytes": n * Hkv * 2 * (D * size + held + D * 2) + n * c["rot"] * 4,
                "flops": n * Hkv * (3 * c["rot"] + 8 * D)}
    Hq, lens, sizes = c["Hq"], _lens(c), _sizes(c)
    seen = sum(n * min(n, 8) if c["tree"] else n * (n + 1) // 2 for n in sizes)
    pairs = sum(n * m for n, m in zip(sizes, lens)) + seen
    bytes_ = sum(m * Hkv * held * 2 for m in lens) + sum(n * (2 * Hq + 2 * Hkv) * D * 2 for n in sizes)
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


def _e2m1_value(n):
    """Values of e2m1 numbers: sign, two exponent bits (bias 1), one of the fraction."""
    n = n.to(torch.int64)
    e, f = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, f * 0.5, (2 + f) * torch.exp2((e - 2).double()))
    return torch.where(n >= 8, -mag, mag)


def _e5m3_value(b):
    """Values of scale bytes: five exponent bits (bias 15), three of the fraction."""
    b = b.to(torch.int64)
    e, f = b >> 3, (b & 7).double()
    return torch.where(e == 0, f * 2.0 ** -17, (8 + f) * torch.exp2((e - 18).double()))


def _held(c, codes, scale):
    """Values [..., D] of a cache's codes and scales, 64 bits."""
    if c.get("bits") == 8:
        return _e4m3_value(codes) * scale.double()
    x = torch.empty((*codes.shape[:-1], c["D"]), dtype=torch.float64, device=DEV)
    x[..., 0::2], x[..., 1::2] = _e2m1_value(codes & 15), _e2m1_value(codes >> 4)
    return x * _e5m3_value(scale).repeat_interleave(16, -1)


def _round4(x):
    """x [..., D] as a 4-bit cache holds it: steps of 2^-17 to 2^10 from the largest magnitudes."""
    y = x.unflatten(-1, (-1, 16))
    least = y.abs().amax(-1, keepdim=True) / 6.0
    step = torch.exp2(torch.floor(torch.log2(least.clamp(min=2.0 ** -40))).clamp(min=-14) - 3)
    scale = (torch.ceil(least / step) * step).clamp(min=2.0 ** -17, max=10240.0)
    z = (y / scale).clamp(-6.0, 6.0)
    ulp = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -9))).clamp(min=0.0) - 1)
    return (torch.round(z / ulp) * ulp * scale).flatten(-2)


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


def _exact_norm(c, s):
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "k")}
    for b in range(c["batch"]):
        n, m = int(s["n_nodes"][b]), int(s["len"][b])
        at = m + (s["pos"][b, :n].long() if c["tree"] else torch.arange(n, device=DEV))
        for name in ("q", "k"):
            x = s[name][b, :n].double()
            root = torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / c["D"] + s["eps"])
            out[name][b, :n] = _turn_exact(x / root * s[name + "_weight"].double(), c, s, at)
    return out


def _exact_attend(c, s):
    out = torch.zeros((c["batch"], c["nodes"], c["Hq"], c["D"]), dtype=torch.float64, device=DEV)
    G = c["Hq"] // c["Hkv"]
    for b in range(c["batch"]):
        n, m = int(s["n_nodes"][b]), int(s["len"][b])
        q, k, v = (s[x][b, :n].double() for x in ("q", "k", "v"))
        ids = s["table"][b, :-(-m // c["page"])].long()
        sees = torch.ones((n, m + n), dtype=torch.bool, device=DEV)
        col = torch.arange(n, device=DEV)
        if c["tree"]:
            sees[:, m:] = ((s["mask"][b, :n].long()[:, col // 32] >> (col % 32)) & 1).bool()
        else:
            sees[:, m:] = col[None, :] <= col[:, None]
        for h in range(c["Hkv"]):
            kc = _held(c, s["k_codes"][ids, h], s["k_scale"][ids, h]).view(-1, c["D"])[:m]
            vc = _held(c, s["v_codes"][ids, h], s["v_scale"][ids, h]).view(-1, c["D"])[:m]
            kh, vh = torch.cat((kc, k[:, h])), torch.cat((vc, v[:, h]))
            for i in range(h * G, h * G + G):
                z = (q[:, i] @ kh.T * s["scale"]).masked_fill(~sees, -math.inf)
                p = torch.softmax(z, -1)
                out[b, :n, i] = torch.where(sees.any(-1, keepdim=True), p, 0.0) @ vh
    return out


def _exact_append(c, s):
    out = {n: torch.zeros(s[n + "_out"].shape, dtype=torch.float64, device=DEV) for n in ("k", "v")}
    for b in range(c["batch"]):
        m, n = int(s["len"][b]), int(s["count"][b])
        rows = s["rows"][b, :n].long() if c["path"] else torch.arange(n, device=DEV)
        out["k"][b, :n] = _round4(_turn_exact(s["k"][b][rows].double(), c, s, m + torch.arange(n, device=DEV)))
        out["v"][b, :n] = _round4(s["v"][b][rows].double())
    # bytes: compared whole with the plain form's
    return out | dict.fromkeys(("len", "k_codes", "v_codes", "k_scale", "v_scale"))


def _exact_read(c, s):
    out = {n: torch.zeros(s[n + "_out"].shape, dtype=torch.float64, device=DEV) for n in ("k", "v")}
    for b in range(c["batch"]):
        n = int(s["count"][b])
        at = s["rows"][b, :n].long() if c["picked"] else torch.arange(n, device=DEV)
        ids, slot = s["table"][b, at // c["page"]].long(), at % c["page"]
        for name in ("k", "v"):
            codes, scale = s[name + "_codes"][ids, :, slot], s[name + "_scale"]
            out[name][b, :n] = _held(c, codes, scale[ids][..., None] if c["bits"] == 8 else scale[ids, :, slot])
    return out


def exact(case, seed):
    c = case
    if c["op"] == "attend" and c["batch"] * c["Hq"] * c["nodes"] * (c["ctx_hi"] + c["nodes"]) * c["D"] > 1e12:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "attend": _exact_attend, "append": _exact_append, "read": _exact_read}[c["op"]](c, s)
