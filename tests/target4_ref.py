"""Plain 64-bit references of the 4-bit cache's calls and of the head norms, with the error
bounds the tests hold the kernels to."""
import math

import torch

import target_ref as ref

TOP = 226  # byte of the largest scale


def e2m1_values(n):
    """Values of e2m1 numbers 0..15: sign, two exponent bits (bias 1), one of the fraction."""
    n = n.to(torch.int64)
    e, f = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, f * 0.5, (2 + f) * torch.exp2((e - 2).double()))
    return torch.where(n >= 8, -mag, mag)


def scale_values(b):
    """Values of scale bytes: five exponent bits (bias 15), three of the fraction; NaN from 248 on."""
    b = b.to(torch.int64)
    e, f = b >> 3, (b & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -17, (8 + f) * torch.exp2((e - 18).double()))
    return torch.where(b >= 248, math.nan, v)


def values4(codes, scales):
    """Values [..., D] of codes [..., D / 2] and scale bytes [..., D / 16]."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return e2m1_values(n) * scale_values(scales).repeat_interleave(16, -1)


def quantised(x):
    """Codes and scale bytes of x [..., D] (float64), by the definition: the first scale of the list that
    holds the block, and of all codes the nearest, the even one of two."""
    y = x.unflatten(-1, (-1, 16))
    table = scale_values(torch.arange(1, TOP + 1, device=x.device))
    top = y.abs().amax(-1)
    at = torch.searchsorted(table * 6, top.contiguous()).clamp(max=TOP - 1)
    z = (y / table[at][..., None]).clamp(-6, 6)
    mags = e2m1_values(torch.arange(8, device=x.device))
    edges = (mags[1:] + mags[:-1]) / 2
    low = torch.searchsorted(edges, z.abs().contiguous())                # edges below |z|
    up = torch.searchsorted(edges, z.abs().contiguous(), right=True)     # edges below or at |z|
    n = torch.where(low == up, low, torch.where(low % 2 == 0, low, up))  # at an edge: the even code
    n = (n + 8 * torch.signbit(y)).to(torch.uint8)
    at = (at + 1).to(torch.uint8)
    bad = ~torch.isfinite(y).all(-1)
    n, at = torch.where(bad[..., None], 0, n).to(torch.uint8), torch.where(bad, 255, at).to(torch.uint8)
    n = n.flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), at


def rotated32(x, at, rope):
    """x [n, H, D] rotated to `at` [n] in fp32, every step rounded once, as append does it."""
    x = x.float()
    if rope is None:
        return x
    cos, sin, interleaved = rope
    co, si = cos[at][:, None], sin[at][:, None]
    r = 2 * cos.shape[1]
    y = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = x[..., a] * co - x[..., b] * si
    y[..., b] = x[..., b] * co + x[..., a] * si
    return y


def held(codes, scales, table, length, page):
    """Values [length, Hkv, D] that a request's tokens stand for; codes and scales of one cache."""
    n = -(-length // page)
    ids = table[:n].long()
    x = values4(codes[ids], scales[ids]) if scales.dtype == torch.uint8 else \
        ref.e4m3_values(codes[ids]) * scales[ids].double()[..., None, None]
    return x.transpose(1, 2).reshape(n * page, x.shape[1], x.shape[3])[:length]


def attention(cache, b, q, k, v, sees, at, rope, scale):
    """Outputs [n, Hq, D] of one request's n rows and a bound on the kernel's error.

    What the cache stands for is exact in fp16.  The kernel rounds q, new k and v, and the probabilities
    to fp16 (each within 2^-11 relative, after scaling), accumulates in fp32 (2^-23 per step and element)
    and rounds the result to bf16 (2^-8 relative).  A score error ds moves a probability by a factor
    within e^(2 ds) (numerator and sum)."""
    n, Hq, D = q.shape
    m, G = int(cache.len[b]), Hq // cache.Hkv
    q, k, v = ref.rotate(q.double(), at, rope), ref.rotate(k.double(), at, rope), v.double()
    kc, vc = held(cache.k, cache.k_scale, cache.table[b], m, cache.page), held(cache.v, cache.v_scale, cache.table[b], m, cache.page)
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
        ds = size.amax(-1, keepdim=True) if size.shape[1] else torch.zeros((n, 1), device=q.device).double()
        ds = ds * (2 * 2.0 ** -11 + D * 2.0 ** -23)
        a = p @ W.abs()
        bound[:, h] = 2.0 ** -8 * 1.01 * out[:, h].abs() + a * (2 * ds * 1.05 + 2 * 2.0 ** -11 + (m + n) * 2.0 ** -23) + 1e-30
    return out, bound


def normed(x, w, eps, at, rope, dtype):
    """Norms [n, H, D] of x's heads times w ([D], [H, D] or None), rotated to `at`, and a bound on the
    kernel's error.

    u = 2^-24 is half a step of fp32.  A sum of D <= 128 squares is formed in runs of 8, then pairwise in
    at most 4 more additions: within 8 + 4 + 1 steps, 13 u, of the sum of its (positive) terms; the mean,
    eps and the reciprocal root (2 steps of 2 u) and halving for the root make 13 / 2 + 6 u; two products
    (by the root, by w) 2 u more: 15 u of an element's magnitude.  A rotation adds two products and a sum,
    2 u of |a cos| + |b sin| each.  Rounding to the result's type: half a step, relative to the value."""
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    mag = y.abs()
    if rope is not None:
        cos, sin, interleaved = rope
        mag = ref.rotate(mag, at, (cos.abs(), -sin.abs(), interleaved))   # first of a pair: a |cos| + b |sin|
        mag = torch.maximum(mag, ref.rotate(y.abs(), at, (cos.abs(), sin.abs(), interleaved)))
        y = ref.rotate(y, at, rope)
    return y, mag * (18 * 2.0 ** -24) * 1.01 + y.abs() * torch.finfo(dtype).eps / 2 * 1.01 + 1e-37
