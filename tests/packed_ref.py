"""64-bit values of the packed, paged and prefix attention tests, with error bounds.

Everything is computed in float64 from the definitions on the inputs' bf16 values. The
bounds count the kernels' roundings (u = 2^-8, half a step of bf16 relative to the value;
fp32 steps are 2^-24):

  scores   products of bf16 values summed in fp32: e_s <= (d + 4) 2^-24 scale (|Q| |K|^T),
           which is also the relative error it gives each exp
  O        every weight P is rounded to bf16 (u), and O is: u |O| + (u + 2 e_s + 2^-14) P|V|
           (2^-14 covers exp2, the fp32 sums and products of two of the terms)
  L        e_s of the row's largest + 2^-20 (1 + |L|)
  dV       u |dV| + (u + 2 e_s + 2^-13) P^T |dO|
  D        the row sum of dO o O with O in bf16: e_D = |dO| . (bound of O)
  dS       e_dS = (u + 3 e_s + 2^-12) P (|dO| |V|^T + |D|) + P e_D
  dQ       u |dQ| + scale e_dS |K|        dK   u |dK| + scale e_dS^T |Q|
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8


def packed_inputs(lens, hq, hkv, d, seed, rest=0, std=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens) + rest
    mk = lambda h, s: (torch.randn(total, h, d, generator=g) * s).to(torch.bfloat16).to(device)  # noqa: E731
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    cu = torch.tensor(at, dtype=torch.int32, device=device)
    return mk(hq, std), mk(hkv, std), mk(hkv, 1.0), mk(hq, 1.0), cu


def attention64(q, k, v, causal, scale, do=None):
    """One sequence, one key/value head: q, do [g, n, d], k, v [m, d] (float64). Returns
    values and bounds of O [g, n, d], L [g, n] and, with do, of dQ, dK, dV (dK, dV summed
    over the g query heads)."""
    d = q.shape[-1]
    s = torch.matmul(q, k.T) * scale
    es = (d + 4) * 2.0 ** -24 * scale * torch.matmul(q.abs(), k.abs().T)
    if causal:
        hidden = torch.ones(s.shape[-2:], dtype=torch.bool, device=s.device).triu(1)
        s = s.masked_fill(hidden, -math.inf)
        es = es.masked_fill(hidden, 0.0)
    es = es.amax(dim=-1, keepdim=True)
    L = torch.logsumexp(s, dim=-1)
    p = torch.exp(s - L[..., None])
    o, pv = torch.matmul(p, v), torch.matmul(p, v.abs())
    out = {"O": (o, U * o.abs() + (U + 2 * es + 2.0 ** -14) * pv),
           "L": (L, es[..., 0] + 2.0 ** -20 * (1 + L.abs()))}
    if do is None:
        return out
    pt = p.transpose(-1, -2)
    dv = torch.matmul(pt, do).sum(0)
    dv_b = U * dv.abs() + torch.matmul(((U + 2 * es + 2.0 ** -13) * p).transpose(-1, -2),
                                       do.abs()).sum(0)
    dp = torch.matmul(do, v.T)
    D = (do * o).sum(-1, keepdim=True)
    e_d = (do.abs() * out["O"][1]).sum(-1, keepdim=True)
    ds = p * (dp - D)
    e_ds = ((U + 3 * es + 2.0 ** -12) * p * (torch.matmul(do.abs(), v.abs().T) + D.abs())
            + p * e_d)
    dq = scale * torch.matmul(ds, k)
    dk = scale * torch.matmul(ds.transpose(-1, -2), q).sum(0)
    out["dQ"] = (dq, U * dq.abs() + scale * torch.matmul(e_ds, k.abs()))
    out["dK"] = (dk, U * dk.abs() + scale * torch.matmul(e_ds.transpose(-1, -2), q.abs()).sum(0))
    out["dV"] = (dv, dv_b)
    return out


def packed64(q, k, v, lens, causal, scale=None, do=None):
    """Values and bounds over the packed layout: O, dQ [total, Hq, d], L [Hq, total],
    dK, dV [total, Hkv, d]; NaN in rows that no sequence covers."""
    total, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64, device=q.device)  # noqa: E731
    shapes = {"O": (total, hq, d), "L": (hq, total)}
    if do is not None:
        shapes.update(dQ=(total, hq, d), dK=(total, hkv, d), dV=(total, hkv, d))
    out = {name: (nan(*s), nan(*s)) for name, s in shapes.items()}
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        for h in range(hkv):
            hs = slice(h * g, (h + 1) * g)
            r = attention64(q[rows, hs].double().transpose(0, 1), k[rows, h].double(),
                            v[rows, h].double(), causal, scale,
                            None if do is None else do[rows, hs].double().transpose(0, 1))
            for i in (0, 1):
                out["O"][i][rows, hs] = r["O"][i].transpose(0, 1)
                out["L"][i][hs, rows] = r["L"][i]
                if do is not None:
                    out["dQ"][i][rows, hs] = r["dQ"][i].transpose(0, 1)
                    out["dK"][i][rows, h] = r["dK"][i]
                    out["dV"][i][rows, h] = r["dV"][i]
    return out


def assert_close(name, got, want, mask=None):
    """Every element within its bound (`want`: value and bound)."""
    ref, bound = want
    got = got.double()
    if mask is not None:
        got, ref, bound = got[mask], ref[mask], bound[mask]
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{name}: {int((~torch.isfinite(got)).sum())} not finite"
    over = (got - ref).abs() / (bound + 1e-30)
    worst = float(over.max())
    assert worst <= 1.0, (f"{name}: an error of {worst:.2f} times its bound "
                          f"({int((over > 1).sum())} of {over.numel()} outside)")
