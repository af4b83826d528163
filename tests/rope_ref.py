"""64-bit values of the norm, rotation and 4-bit cache tests, with error bounds.

Everything is computed in float64 from the definitions on the inputs' bf16 (and the table's
fp32) values. The bounds count the kernels' roundings (u = 2^-8, half a step of bf16 relative
to the value; fp32 steps are 2^-24, at most half of one an operation, 2 for rsqrt):

  norm      the row's sum of squares d / 2 + 4 steps, rsqrt 4, two products 2: relative
            e_n = (d / 2 + 12) 2^-24
  turned    a c - b s: three roundings more, relative to A = |a c| + |b s|
            y: u |y| + (e_n + 4 2^-24) A
  gradient  g = R^T dy with 4 2^-24 A(dy); dx = r (g w - n mean(g w n)), each product and sum of
            it a rounding, relative to M = r (A w + |n| mean(A w |n|)):
            dx: u |dx| + 2 (e_n + d 2^-24) M
            dw: a lane's sum has at most `total` terms, then 64 + d more:
            (total + 64 + d + 2 d) 2^-24 sum(A |n|)
  4 bits    a value is off by half a scale inside [min, min + 15 scale], else by the
            distance from there, at most the rounding of min, or 15 roundings of scale
  scores    products of q with 128 + code (up to 143), of sum q with min - 128 scale:
            e_s = (d + 8) 2^-24 scale |q| (271 s + |min|)
  O         weights times scales in bf16, |code - 8| <= 8, the rest in fp32:
            u |O| + (u + 2 e_s + 2^-14) P (8 s + |min + 8 s|)
  L         e_s of the row's largest + 2^-20 (1 + |L|)
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
E = 2.0 ** -24


def turn(x, cos, sin, interleaved, back=False):
    """x [T, H, d] (float64) turned, and the magnitudes |a c| + |b s| of its terms."""
    h = cos.shape[1]
    c, s = cos[:, None], (-sin if back else sin)[:, None]
    y, mag = x.clone(), x.abs()
    ia = torch.arange(h, device=x.device) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else h)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return y, mag


def table64(cos_sin, pos):
    rows = cos_sin.double()[pos.long()]
    return rows.chunk(2, dim=1)


def norm_rope64(x, w, cos_sin, pos, eps, interleaved):
    """Values before the last rounding, and the bound without it, of [T, H, d]."""
    x = x.double()
    d = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if cos_sin is None:
        return x, (d / 2 + 16) * E * x.abs()
    y, mag = turn(x, *table64(cos_sin, pos), interleaved)
    return y, (d / 2 + 16) * E * mag


def rounded(y, e):
    """Bound of y in bf16."""
    return U * (y.abs() + e) + e


def norm_rope_backward64(dy, x, w, cos_sin, pos, eps, interleaved):
    """(dx, bound, dw, bound)."""
    x, dy = x.double(), dy.double()
    t, _, d = x.shape
    g, mag = (dy, dy.abs()) if cos_sin is None else turn(
        dy, *table64(cos_sin, pos), interleaved, back=True)
    if w is None:
        return g, U * g.abs() + 8 * E * mag, None, None
    w = w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    m = r * (mag * w.abs() + n.abs() * (mag * w.abs() * n.abs()).mean(-1, keepdim=True))
    e = 2 * (1.5 * d + 16) * E * m
    dw, sm = (g * n).sum((0, 1)), (mag * n.abs()).sum((0, 1))
    return dx, U * dx.abs() + e, dw, (t + 64 + 3 * d) * E * sm


# ------------------------------------------------------------------ the cache in 4 bits
def groups(d):
    return 2 if d > 64 else 1


def places(d):
    """Byte of the block, and shift, of each code [2 (K, V), 16 rows, d], and the byte of each
    pair [2, 16, G], as include/fa.h gives them."""
    G = groups(d)
    code = torch.zeros(2, 16, d, dtype=torch.long)
    shift = torch.zeros(2, 16, d, dtype=torch.long)
    pair = torch.zeros(2, 16, G, dtype=torch.long)
    for r in range(16):
        for c in range(d):
            j, w, e = c // 64, c % 64 // 8, c % 8
            words = (8 * G * r + 2 * G * (w // 2) + 2 * j + w % 2,
                     128 * G + 128 * j + 16 * w + 4 * (r % 8 // 2) + r % 2 + 2 * (r // 8))
            for kv in (0, 1):
                code[kv, r, c] = 4 * words[kv] + e // 2
                shift[kv, r, c] = 4 * (e % 2)
        for j in range(G):
            pair[0, r, j] = 4 * (256 * G + 2 * G * r + j)
            pair[1, r, j] = 4 * (256 * G + 2 * G * r + G + j)
    return code, shift, pair


def unpack(cache, d):
    """cache [pages, H, page / 16, bytes] -> codes [2, pages, H, page, d] (int) and (scale, min)
    [2, pages, H, page, G, 2] (float64)."""
    cache = cache.cpu()
    code, shift, pair = places(d)
    pages, H, blocks, _ = cache.shape
    codes = [(cache[..., code[kv].flatten()].long() >> shift[kv].flatten()) & 15 for kv in (0, 1)]
    codes = torch.stack(codes).reshape(2, pages, H, blocks * 16, d)
    raw = torch.stack([torch.stack([cache[..., pair[kv].flatten() + i] for i in range(4)], -1)
                       for kv in (0, 1)])
    pairs = raw.contiguous().view(torch.bfloat16).double()
    return codes, pairs.reshape(2, pages, H, blocks * 16, groups(d), 2)


def pack(codes, pairs, d, like):
    """The reverse, into a copy of `like`, whose other bits stay."""
    out = like.cpu().clone()
    code, shift, pair = places(d)
    pages, H, blocks, _ = out.shape
    for kv in (0, 1):
        c = codes[kv].reshape(pages, H, blocks, 16 * d).to(torch.uint8)
        s, at = shift[kv].flatten(), code[kv].flatten()
        for half in (0, 4):
            pick = s == half
            mask = 15 << half
            out[..., at[pick]] = (out[..., at[pick]] & (255 - mask)) | (c[..., pick] << half)
        raw = pairs[kv].to(torch.bfloat16).contiguous().view(torch.uint8).reshape(
            pages, H, blocks, -1, 4)
        for i in range(4):
            out[..., pair[kv].flatten() + i] = raw[..., i]
    return out


def values(codes, pairs):
    """min + scale * code, [..., d]."""
    d = codes.shape[-1]
    wide = pairs.repeat_interleave(64, dim=-2)[..., :d, :]
    return wide[..., 1] + wide[..., 0] * codes


def quantize(x):
    """Codes [..., d] and (scale, min) [..., G, 2] of x (fp32 values): the definition, with
    the division in fp32 as its rounding to bf16 follows it."""
    d = x.shape[-1]
    lo, scale = [], []
    for g in x.float().split(64, -1):
        a = g.amin(-1).to(torch.bfloat16)
        lo.append(a)
        scale.append(((g.amax(-1) - a.float()).clamp(min=0) / 15).to(torch.bfloat16))
    pairs = torch.stack([torch.stack(scale, -1), torch.stack(lo, -1)], -1).double()
    wide = pairs.repeat_interleave(64, dim=-2)[..., :d, :]
    s = wide[..., 0]
    q = (x.double() - wide[..., 1]) / torch.where(s > 0, s, torch.ones_like(s))
    codes = torch.where(s > 0, torch.round(q).clamp(0, 15), torch.zeros_like(q)).long()
    return codes, pairs


def decode64(q, codes, pairs, scale):
    """One request, one key/value head: q [g, d], codes and pairs [2, n, ...] of its keys.
    Returns (value, bound) of O [g, d] and L [g]."""
    d = q.shape[-1]
    k, v = values(codes[0], pairs[0]), values(codes[1], pairs[1])
    wide = pairs.repeat_interleave(64, dim=-2)[..., :d, :]
    sk, mk, sv, mv = wide[0, ..., 0], wide[0, ..., 1], wide[1, ..., 0], wide[1, ..., 1]
    s = q @ k.T * scale
    es = (d + 8) * E * scale * (q.abs() @ (271 * sk + mk.abs()).T)
    es = es.amax(-1, keepdim=True)
    L = torch.logsumexp(s, -1)
    p = torch.exp(s - L[:, None])
    o = p @ v
    mag = p @ (8 * sv + (mv + 8 * sv).abs())
    return ((o, U * o.abs() + (U + 2 * es + 2.0 ** -14) * mag),
            (L, es[:, 0] + 2.0 ** -20 * (1 + L.abs())))


def softmax_scale(d):
    return 1.0 / math.sqrt(d)
