"""Plain 64-bit references of the target-side calls, one request at a time, with the
error bounds the tests hold the kernels to."""
import math

import torch


def e4m3_values(codes):
    """Values of e4m3 bytes: sign, four exponent bits (bias 7), three fraction bits; 0x7F is NaN."""
    b = codes.to(torch.int64)
    e, f = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).double()))
    mag = torch.where((b & 127) == 127, math.nan, mag)
    return torch.where(b >= 128, -mag, mag)


def rope_tables(positions, rot, device, base=1e4):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return a.cos().float().to(device), a.sin().float().to(device)


def rotate(x, at, rope):
    """x [n, H, D] float64 to the positions `at` [n]; rope = (cos, sin, interleaved) or None."""
    if rope is None:
        return x
    cos, sin, interleaved = rope
    co, si = cos[at].double()[:, None], sin[at].double()[:, None]
    r = 2 * cos.shape[1]
    y = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = x[..., a] * co - x[..., b] * si
    y[..., b] = x[..., b] * co + x[..., a] * si
    return y


def held(codes, scale, table, length, page):
    """Dequantised [length, Hkv, D] of one request."""
    n = -(-length // page)
    ids = table[:n].long()
    x = e4m3_values(codes[ids]) * scale[ids].double()[..., None, None]  # [n, Hkv, page, D]
    return x.transpose(1, 2).reshape(n * page, codes.shape[1], codes.shape[3])[:length]


def attention(cache, b, q, k, v, sees, at, rope, scale):
    """Outputs [n, Hq, D] of one request's n rows and a bound on the kernel's error.

    The kernel rounds q, new k and v, and the probabilities to fp16 (each within 2^-11
    relative, after scaling), accumulates in fp32 (2^-23 per step and element), and rounds
    the result to bf16 (2^-9 relative).  A score error ds moves a probability by a factor
    within e^(2 ds) (numerator and sum)."""
    n, Hq, D = q.shape
    Hkv, m = cache.Hkv, int(cache.len[b])
    G = Hq // Hkv
    q, k, v = rotate(q.double(), at, rope), rotate(k.double(), at, rope), v.double()
    codes = (cache.k, cache.v)
    kc, vc = (held(c, s, cache.table[b], m, cache.page) for c, s in zip(codes, (cache.k_scale, cache.v_scale)))
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    for h in range(Hq):
        K, W = torch.cat((kc[:, h // G], k[:, h // G])), torch.cat((vc[:, h // G], v[:, h // G]))
        see = torch.cat((torch.ones((n, m), dtype=torch.bool, device=q.device), sees), 1)
        W = torch.where(see.any(0)[:, None], W, 0.0)   # what nobody sees does not matter
        K = torch.where(see.any(0)[:, None], K, 0.0)
        s = (q[:, h] @ K.T * scale).masked_fill(~see, -math.inf)
        p = torch.softmax(s, -1).masked_fill(~see, 0.0)
        p = torch.where(see.any(-1, keepdim=True), p, 0.0)
        out[:, h] = p @ W
        size = (q[:, h].abs() @ K.abs().T * scale).masked_fill(~see, 0.0)
        ds = (size.amax(-1, keepdim=True) if size.shape[1] else torch.zeros((n, 1), device=q.device).double())
        ds = ds * (2 * 2.0 ** -11 + D * 2.0 ** -23)
        a = p @ W.abs()
        steps = (m + n) * 2.0 ** -23
        bound[:, h] = 2.0 ** -9 * 1.01 * out[:, h].abs() + a * (2 * ds * 1.05 + 2 * 2.0 ** -11 + steps) + 1e-30
    return out, bound


def path_bits(parents):
    """Ancestor-or-self matrix of a parent list (root first)."""
    n = len(parents)
    anc = torch.zeros((n, n), dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            anc[i] = anc[p]
        anc[i, i] = True
    return anc


def pack(sees, M):
    """Bits [n, n] to int32 words [M, ceil(M / 32)]."""
    words = (M + 31) // 32
    full = torch.zeros((M, words * 32), dtype=torch.int64)
    full[:sees.shape[0], :sees.shape[1]] = sees.to("cpu", torch.int64)
    w = (full.view(M, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
