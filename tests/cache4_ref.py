"""64-bit values of decode over the cache in 4 bits, with the error bounds of its arithmetic.

The steps (U = 2^-8 half a step of bf16 relative to the value, H = 2^-11 of fp16, E = 2^-24 of
fp32; ex2.approx is 2^-22 off at most):

  scores    q is held in fp16 relative to its row's largest magnitude, 2^-29 of that off at
            most; codes are exact. Products and sums of d terms in fp32, where the tensor
            cores may cut instead of round (2 E):
            e_s = scale ((d + 8) 2 E |q| (s c + |min|) + 2^-29 max|q| sum(s c))
  weights   of each key relative: 2 e_s (its own score, and those in the sum), 8 E |score - max|
            (two roundings of the exponent, and the references that moved on the way), 2^-17
            (ex2 of up to 32 moves)
  sums      at most n / 16 + 64 additions one after another, 2 E each
  codes     P s is rounded to fp16 relative to a unit, per query and group of 64 channels, that
            is at most the largest P s met, or 2^-110 of the largest weight: H, or the half step
            2^-25 of the unit where that is more (but not more than P s itself)
  O         U |O| for the last rounding
"""
from __future__ import annotations

import torch

from tests import rope_ref as ref

U, H, E = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def wide(pairs, d):
    """(scale, min) [..., G, 2] as two of [..., d]."""
    w = pairs.repeat_interleave(64, dim=-2)[..., :d, :]
    return w[..., 0], w[..., 1]


def scores64(q, codes, pairs, scale):
    return q @ ref.values(codes, pairs).T * scale


def decode_bounds(q, codes, pairs, scale):
    """One request, one key/value head: q [g, d] (float64), codes and pairs [2, n, ...] of its
    keys. Returns (value, bound) of O [g, d] and L [g]."""
    d, n = q.shape[-1], codes.shape[1]
    sk, mk = wide(pairs[0], d)
    sv, mv = wide(pairs[1], d)
    s = scores64(q, codes[0], pairs[0], scale)
    es = scale * ((d + 8) * 2 * E * (q.abs() @ (sk * codes[0] + mk.abs()).T)
                  + 2.0 ** -29 * q.abs().amax(-1, keepdim=True) * (sk * codes[0]).sum(-1))
    es = es.amax(-1, keepdim=True)
    L = torch.logsumexp(s, -1)
    p = torch.exp(s - L[:, None])
    o = p @ ref.values(codes[1], pairs[1])
    sums = (n / 16 + 64) * 2 * E
    ep = 2 * es + 2.0 ** -17 + 8 * E * (s.amax(-1, keepdim=True) - s) + sums
    e = (p * ep) @ (sv * codes[1] + mv.abs()) + H * (p @ (sv * codes[1]))
    for j in range(0, d, 64):
        ps = p * sv[:, j]  # one scale a group
        unit = torch.maximum(ps.amax(-1, keepdim=True), 2.0 ** -110 * p.amax(-1, keepdim=True))
        e[:, j:j + 64] += torch.minimum(2.0 ** -25 * unit, ps) @ codes[1][:, j:j + 64].double()
    return ((o, U * (o.abs() + e) + e),
            (L, es[:, 0] + sums + 2.0 ** -20 * (1 + L.abs())))


def telling(q, codes, pairs, place, seed):
    """Queries and (scale, min) for which a part of the keys that is lost, weighted wrongly or taken
    for another moves O by many bounds: scores that differ by about 1 from one 32 keys to the
    next, and values that go along with them and differ by 10, around 0. Returns (q, pairs); q
    [B, Hq, d] is of bf16 values."""
    g = torch.Generator().manual_seed(seed)
    B, Hq, d = q.shape
    Hkv = codes.shape[2]
    base = 0.05 + 0.1 * torch.randn(Hkv, d, generator=g, dtype=torch.float64)
    q = (base.repeat_interleave(Hq // Hkv, 0)
         + 0.02 * torch.randn(B, Hq, d, generator=g, dtype=torch.float64)).to(torch.bfloat16)
    pairs = pairs.clone()
    for pg, r in place:
        n = len(pg)
        if n == 0:
            continue
        by = torch.randn(2, -(-n // 32), Hkv, generator=g, dtype=torch.float64)
        by = by.repeat_interleave(32, 1)[:, :n]
        for h in range(Hkv):
            pairs[0, pg, h, r, :, 1] += (by[0, :, h] * d ** 0.5 / (0.05 * d))[:, None]
            s = scores64(base[h][None], codes[0, pg, h, r], pairs[0, pg, h, r], d ** -0.5)[0]
            add = 10 * by[1, :, h] + 5 * s
            pairs[1, pg, h, r, :, 1] += (add - torch.softmax(s, 0) @ add)[:, None]
    return q, pairs.to(torch.bfloat16).double()
