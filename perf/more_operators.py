"""Cases, plain forms and 64-bit values of the operators between projection and attention, and
of the cache in 4 bits.

The operators, in the layouts of the package's entry points (bf16 in and out):

  qk       queries Q [T, Hq, d] and keys K [T, Hkv, d], slices of one projection. Each head's
           row is divided by its root mean square, times a weight [d] (or not), and its first
           `rot` channels are turned by the angles of the row's position, in pairs (i, i + rot/2)
           or (2i, 2i + 1); cosines and sines come from a table [positions, rot]. Training adds
           the gradients of Q, K and the weights.
  append   the same on the way into a paged cache: K and V rows of several requests (cu_seqlens)
           go to positions starts[i], starts[i] + 1, ... in the pages their block tables name,
           K normed and turned for that position, and Q comes back normed and turned.
  chunk4   a chunk of several prompts: appended like that to a cache in 4 bits, and the requests'
           whole contexts (what the cache held before, and the chunk) read back in bf16, as the
           attention of the chunk needs them.
  decode4  one new token for each of B requests, Q [B, Hq, d], over the first lens[b] positions
           of the request's keys and values in a cache in 4 bits.

A row of the cache in 4 bits has groups of 64 channels (the last one filled up to 64), each with
a scale and a minimum in bf16: value = minimum + scale * code, codes 0 to 15, of a tie the even
one. 16 rows of a head lie together in a block of 1152 bytes per group (see _places).

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true,
with the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # A small ragged batch of an odd head dimension, both directions: latency counts.
        dict(name="qk_train_small", kind="qk", total=333, positions=400, lens_seed=7, hq=6, hkv=2,
             d=96, rot=96, norm=True, inter=False, train=True),
        # Packed training of a model with grouped heads.
        dict(name="qk_train", kind="qk", total=16384, positions=8192, lens_seed=4, hq=32, hkv=8,
             d=128, rot=128, norm=True, inter=False, train=True),
        # Prompts of a model that turns half of each head in neighbouring pairs, without norms.
        dict(name="qk_prompts", kind="qk", total=30001, positions=32768, lens_seed=2, hq=16,
             hkv=16, d=64, rot=32, norm=False, inter=True, train=False),
        # The new tokens of one decode step, one for each request.
        dict(name="append_step", kind="append", total=64, nseq=64, lens_seed=1, start_max=4000,
             hq=32, hkv=8, d=128, rot=128, norm=True, inter=False, page=16),
        # A batch of prompts.
        dict(name="append_prompts", kind="append", total=32768, nseq=24, lens_seed=2,
             start_max=1000, hq=32, hkv=8, d=128, rot=128, norm=True, inter=False, page=64),
        # A few short prompts of a small model, behind short contexts.
        dict(name="chunk4_small", kind="chunk4", total=150, nseq=3, lens_seed=3, start_max=100,
             hq=8, hkv=2, d=64, rot=64, norm=True, inter=False, page=16),
        # The next chunks of long prompts, behind what was taken in before.
        dict(name="chunk4_prompts", kind="chunk4", total=8192, nseq=8, lens_seed=5,
             start_max=16000, hq=32, hkv=8, d=128, rot=128, norm=True, inter=False, page=64),
        # Two requests of a small model: the smallest decode step.
        dict(name="decode4_small", kind="decode4", batch=2, most=300, lens_seed=1, hq=8, hkv=2,
             d=64, page=16),
        # A serving batch of ordinary contexts.
        dict(name="decode4_batch", kind="decode4", batch=32, most=4096, lens_seed=2, hq=32, hkv=8,
             d=128, page=16),
        # Many requests.
        dict(name="decode4_wide", kind="decode4", batch=256, most=8192, lens_seed=3, hq=32, hkv=8,
             d=128, page=64),
        # As many key/value heads as query heads, a head dimension that fills no group.
        dict(name="decode4_mha", kind="decode4", batch=24, most=5000, lens_seed=5, hq=16, hkv=16,
             d=80, page=32),
        # Two very long contexts: work has to be split along the keys.
        dict(name="decode4_long", kind="decode4", batch=2, most=200000, lens_seed=4, hq=16, hkv=2,
             d=128, page=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["qk", "append", "chunk4", "decode4", "decode4"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = min(hkv * rng.choice([1, 2, 3, 4, 7, 8]), 32)
    d = rng.choice([32, 40, 64, 72, 80, 96, 128, 128])
    c = dict(kind=kind, lens_seed=rng.randrange(1 << 20), hq=hq, hkv=hkv, d=d)
    if kind == "decode4":
        batch = _log_int(rng, 1, 200)
        return dict(c, hq=hkv * rng.choice([1, 2, 4, 5, 8, 16]), batch=batch,
                    most=_log_int(rng, 1, min(100000, 800000 // batch)),
                    page=rng.choice([16, 32, 64, 128]))
    c.update(rot=rng.choice([d, d, d - d % 16, d // 16 * 8, 8]), norm=rng.random() < 0.7,
             inter=rng.random() < 0.3)
    if kind == "qk":
        total = _log_int(rng, 1, 16384)
        return dict(c, total=total, positions=_log_int(rng, 100, 100000),
                    train=rng.random() < 0.6)
    total = _log_int(rng, 1, 30000 if kind == "append" else 8000)
    nseq = min(total, _log_int(rng, 1, 200 if kind == "append" else 12))
    return dict(c, total=total, nseq=nseq, page=rng.choice([16, 32, 64, 128]),
                start_max=_log_int(rng, 1, 2000 if kind == "append" else 8000))


def _lengths(total, nseq, seed):
    """nseq lengths >= 1 that sum to total, unequal as real batches are."""
    r = random.Random(seed)
    w = [r.expovariate(1.0) + 0.02 for _ in range(nseq)]
    s = sum(w)
    n = [1 + int((total - nseq) * x / s) for x in w]
    n[0] += total - sum(n)
    return n


def _contexts(case):
    """Keys of each request of a decode step: from 1 to most."""
    r = random.Random(case["lens_seed"])
    return [r.randint(1, case["most"]) for _ in range(case["batch"])]


def _starts(case):
    r = random.Random(case["lens_seed"] + 1)
    return [r.randint(0, case["start_max"]) for _ in range(case["nseq"])]


def _groups(d):
    return -(-d // 64)


def work(case):
    kind, d, hq, hkv = case["kind"], case["d"], case["hq"], case["hkv"]
    if kind == "decode4":
        keys = sum(_contexts(case))
        return {"bytes": keys * hkv * 72 * _groups(d) + case["batch"] * hq * (4 * d + 4),
                "flops": 4 * keys * hq * d}
    t = case["total"]
    qk = 2 * t * (hq + hkv) * d  # bytes of Q and K once
    if kind == "qk":  # read and written; the gradients too
        n = 4 if case["train"] else 2
        return {"bytes": n * qk, "flops": (24 if case["train"] else 9) * t * (hq + hkv) * d}
    kv = 2 * t * hkv * d
    q = qk - kv
    if kind == "append":
        return {"bytes": 2 * (q + 2 * kv), "flops": 9 * t * (hq + hkv) * d}
    ctx = t + sum(_starts(case))
    row = 72 * hkv * _groups(d)
    return {"bytes": 2 * q + 2 * kv + ctx * (row + 4 * hkv * d),
            "flops": t * (9 * (hq + hkv) + 10 * hkv) * d + 4 * ctx * hkv * d}


# ---------------------------------------------------------------- the inputs
def _randn(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(
        torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _bounds(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _table(need, page, spare, gen):
    """A block table [len(need), most] for requests of need[i] tokens, over scattered pages,
    and the number of pages; unused entries are 0."""
    count = [-(-n // page) for n in need]
    total = sum(count)
    order = torch.randperm(total + spare, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(len(need), max(1, max(count)), dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(count):
        table[i, :c] = order[at:at + c]
        at += c
    return table, total + spare


def _angles(positions, rot):
    """The table [positions, rot]: cosines, then sines; the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def _places(ng):
    """[16, 72 ng]: where in a block of 1152 ng bytes the bytes of its row r lie: those of K's
    codes (two channels each, the lower one in the lower four bits), of V's codes, of K's
    and of V's pairs (scale, minimum). Codes lie in words of 8 channels, K's by row, then pair
    of words of every group; V's by group, word, and row in the order that follows."""
    r = torch.arange(16, device=DEV)[:, None]
    b = torch.arange(32 * ng, device=DEV)[None, :]
    j, w = b // 32, b // 4 % 8
    k = 4 * (r * 8 * ng + w // 2 * 2 * ng + 2 * j + w % 2) + b % 4
    v = 4 * (128 * ng + 128 * j + (4 * w + r % 8 // 2) * 4 + r % 2 + 2 * (r // 8)) + b % 4
    p = 4 * (256 * ng + r * 2 * ng) + torch.arange(8 * ng, device=DEV)[None, :]
    return torch.cat([k, v, p], 1)


def _quantize(x):
    """[..., d] in 32 or 64 bits: codes [..., ng, 64] (uint8) and pairs [..., ng, 2] (bf16)."""
    d = x.shape[-1]
    fill = _groups(d) * 64 - d
    lo = torch.stack([g.amin(-1) for g in x.split(64, -1)], -1).to(torch.bfloat16)
    hi = torch.stack([g.amax(-1) for g in x.split(64, -1)], -1)
    scale = ((hi - lo.to(x.dtype)) / 15).clamp(min=0).to(torch.bfloat16)
    g = torch.nn.functional.pad(x, (0, fill)).unflatten(-1, (-1, 64))
    q = (g - lo.to(x.dtype)[..., None]) / scale.to(x.dtype)[..., None]
    code = torch.where(scale[..., None] > 0, torch.round(q), torch.zeros_like(q)).clamp(0, 15)
    return code.to(torch.uint8), torch.stack([scale, lo], -1)


def _row_bytes(k, v):
    """The bytes [..., 72 ng] of rows K and V [..., d], in the order of _places."""
    (kc, kp), (vc, vp) = _quantize(k), _quantize(v)
    pack = lambda c: c.flatten(-2)[..., 0::2] | (c.flatten(-2)[..., 1::2] << 4)  # noqa: E731
    raw = lambda p: p.contiguous().flatten(-2).view(torch.uint8)  # noqa: E731
    return torch.cat([pack(kc), pack(vc), raw(kp), raw(vp)], -1)


def _filled(gen, pages, hkv, page, d):
    """A cache in 4 bits [pages, hkv, page / 16, 1152 ng] of random rows."""
    ng = _groups(d)
    cache = torch.empty(pages, hkv, page // 16, 1152 * ng, dtype=torch.uint8, device=DEV)
    flat, at = cache.view(-1, 1152 * ng), _places(ng).flatten()
    step = (1 << 26) // (16 * d)
    for i in range(0, flat.shape[0], step):
        n = min(step, flat.shape[0] - i)
        rows = _row_bytes(*(torch.randn(n, 16, d, generator=gen, device=DEV) for _ in (0, 1)))
        flat[i:i + n, at] = rows.flatten(1)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, d, hq, hkv = case["kind"], case["d"], case["hq"], case["hkv"]
    s = dict(kind=kind, d=d)
    if kind == "decode4":
        lens, page = _contexts(case), case["page"]
        s["table"], pages = _table(lens, page, 2, gen)
        s.update(q=_randn(gen, case["batch"], hq, d), cache=_filled(gen, pages, hkv, page, d),
                 page=page, lens=_ints(lens))
        if own:
            import exact_io_aware_27_gb300 as fa
            s["ws"] = fa.alloc_cache4_workspace(case["batch"], hq, hkv, d,
                                                s["table"].shape[1] * page, DEV)
        return s
    t, rot = case["total"], case["rot"]
    proj = _randn(gen, t, hq + 2 * hkv, d)  # one projection's output
    s.update(q=proj[:, :hq], k=proj[:, hq:hq + hkv], v=proj[:, hq + hkv:], inter=case["inter"],
             wq=None, wk=None)
    if case["norm"]:
        s["wq"], s["wk"] = (torch.randn(d, generator=gen, device=DEV).mul_(0.3).add_(1.0).to(
            torch.bfloat16) for _ in (0, 1))
    if kind == "qk":
        r = random.Random(case["lens_seed"])
        pos, most = [], case["positions"]
        while len(pos) < t:  # sequences that begin anywhere (chunks of longer ones among them)
            a = r.randrange(most)
            pos += range(a, min(most, a + r.randint(1, most)))
        s.update(pos=_ints(pos[:t]), table=_angles(most, rot), train=case["train"])
        if case["train"]:
            s.update(dq=_randn(gen, t, hq, d), dk=_randn(gen, t, hkv, d))
            if own:
                import exact_io_aware_27_gb300 as fa
                s["ws"] = fa.alloc_qk_norm_rope_workspace(hq, hkv, d, DEV)
        return s
    page, lens, starts = case["page"], _lengths(t, case["nseq"], case["lens_seed"]), _starts(case)
    ends = [a + n for a, n in zip(starts, lens)]
    table, pages = _table(ends, page, 3, gen)
    s.update(cu=_ints(_bounds(lens)), starts=_ints(starts), pages=table, page=page,
             table=_angles(max(ends), rot))
    if kind == "append":
        s.update(kc=_randn(gen, pages, hkv, page, d), vc=_randn(gen, pages, hkv, page, d))
    else:
        s.update(cache=_filled(gen, pages, hkv, page, d), ctx=_ints(_bounds(ends)),
                 zero=_ints([0] * len(ends)), rows=sum(ends))
    return s


# ---------------------------------------------------------------- plain forms, 32 bits
def _turn(x, cos, sin, inter, sign=1.0):
    """x [T, H, d] with its first rot channels turned by the angles [T, rot / 2]."""
    h = cos.shape[1]
    c, s = cos[:, None], sin[:, None] * sign
    y = x.clone()
    if inter:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2] = a * c - b * s
        y[..., 1:2 * h:2] = b * c + a * s
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h] = a * c - b * s
        y[..., h:2 * h] = b * c + a * s
    return y


def _angles_of(s, pos):
    return s["table"][pos.long()].chunk(2, 1)


def _plain_row(x, w, angles, inter):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(x, *angles, inter)


def _plain_back(dy, x, w, angles, inter):
    g = _turn(dy.float(), *angles, inter, -1.0)
    if w is None:
        return g.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    gw = g * w.float()
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (g * n).sum((0, 1))


def _plain_qk(s):
    angles = _angles_of(s, s["pos"])
    out = [_plain_row(s[x], s["w" + x], angles, s["inter"]).to(torch.bfloat16) for x in "qk"]
    if not s["train"]:
        return tuple(out)
    (dq, dwq), (dk, dwk) = (_plain_back(s["d" + x], s[x], s["w" + x], angles, s["inter"])
                            for x in "qk")
    return (*out, dq, dk, dwq, dwk)


def _where(cu, starts, total):
    """Request and position of each of `total` rows."""
    t = torch.arange(total, device=DEV)
    req = (t[:, None] >= cu[None, 1:]).sum(dim=1)
    return req, starts[req] + t - cu[req]


def _plain_append(s):
    req, pos = _where(s["cu"], s["starts"], s["k"].shape[0])
    page = s["pages"][req, pos // s["page"]].long()
    angles = _angles_of(s, pos)
    q, k = (_plain_row(s[x], s["w" + x], angles, s["inter"]) for x in "qk")
    if s["kind"] == "append":
        s["kc"][page, :, pos % s["page"]] = k.to(torch.bfloat16)
        s["vc"][page, :, pos % s["page"]] = s["v"]
        return q.to(torch.bfloat16), s["kc"], s["vc"]
    cache = s["cache"]
    at = _places(_groups(s["d"]))[pos % 16][:, None]                            # [T, 1, bytes]
    block = (page * cache.shape[1] * cache.shape[2] + pos % s["page"] // 16)[:, None]
    block = block + torch.arange(cache.shape[1], device=DEV) * cache.shape[2]   # [T, Hkv]
    cache.view(-1)[block[..., None] * cache.shape[3] + at] = _row_bytes(k, s["v"].float())
    req, pos = _where(s["ctx"], s["zero"], s["rows"])
    kv = _values(cache, s["pages"][req, pos // s["page"]].long(), pos, s["page"], s["d"])
    return (q.to(torch.bfloat16), *(x.to(torch.bfloat16) for x in kv))


def _decoded(rows, d):
    """K and V [..., d] in 32 bits of rows' bytes [..., 72 ng]."""
    ng = _groups(d)
    out = []
    for i in (0, 1):
        c = rows[..., 32 * ng * i:32 * ng * (i + 1)]
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).float().unflatten(-1, (ng, 64))
        p = rows[..., 64 * ng + 4 * ng * i:64 * ng + 4 * ng * (i + 1)].contiguous().view(
            torch.bfloat16).float().unflatten(-1, (ng, 2))
        out.append((p[..., 1:] + p[..., :1] * c).flatten(-2)[..., :d])
    return out


def _values(cache, page, pos, size, d):
    """K and V [T, Hkv, d] of the rows at positions pos of pages page."""
    block = cache[page, :, pos % size // 16]                       # [T, Hkv, bytes of a block]
    at = _places(_groups(d))[pos % 16][:, None].expand(-1, cache.shape[1], -1)
    return _decoded(torch.gather(block, 2, at), d)


def _plain_decode(s):
    q, lens, d = s["q"], s["lens"], s["d"]
    b, hq, _ = q.shape
    cache, ng = s["cache"], _groups(d)
    hkv = cache.shape[1]
    rows = cache[s["table"].long()][..., _places(ng).flatten()].unflatten(-1, (16, 72 * ng))
    rows = rows.transpose(1, 2).flatten(2, 4)                      # [B, Hkv, keys, bytes]
    k, v = _decoded(rows, d)
    qf = q.float().view(b, hkv, hq // hkv, d)
    x = torch.matmul(qf, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    hidden = torch.arange(k.shape[2], device=q.device) >= lens[:, None]
    x = x.masked_fill(hidden[:, None, None], -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / l
    return o.reshape(b, hq, d).to(torch.bfloat16), (m + torch.log(l)).reshape(b, hq)


def run(state):
    s = state
    if not own:
        return {"qk": _plain_qk, "append": _plain_append, "chunk4": _plain_append,
                "decode4": _plain_decode}[s["kind"]](s)
    import exact_io_aware_27_gb300 as fa
    if s["kind"] == "decode4":
        return fa.fa_cache4_decode(s["q"], s["cache"], s["table"], s["lens"], workspace=s["ws"])
    how = dict(cos_sin=s["table"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
               interleaved=s["inter"])
    if s["kind"] == "append":
        q = fa.fa_rope_append(s["q"], s["k"], s["v"], s["cu"], s["starts"], s["pages"], s["kc"],
                              s["vc"], **how)
        return q, s["kc"], s["vc"]
    if s["kind"] == "chunk4":
        q = fa.fa_cache4_append(s["q"], s["k"], s["v"], s["cu"], s["starts"], s["pages"],
                                s["cache"], **how)
        return (q, *fa.fa_cache4_read(s["cache"], s["ctx"], s["zero"], s["pages"], s["rows"],
                                      s["d"]))
    out = fa.fa_qk_norm_rope(s["q"], s["k"], s["pos"], **how)
    if not s["train"]:
        return out
    return (*out, *fa.fa_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"],
                                               workspace=s["ws"], **how))


# ---------------------------------------------------------------- 64 bits
def _exact_row(x, w, table, pos, inter):
    """As complex numbers: a pair of channels times cos + i sin."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    t = table[pos.long()].double()
    h = t.shape[1] // 2
    z = torch.complex(t[:, :h], t[:, h:]).unsqueeze(1)
    if inter:
        y = torch.view_as_complex(x[..., :2 * h].unflatten(-1, (h, 2)).contiguous()) * z
        y = torch.view_as_real(y).flatten(-2)
    else:
        y = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * z
        y = torch.cat([y.real, y.imag], -1)
    return torch.cat([y, x[..., 2 * h:]], -1)


def _exact_qk(s):
    """The gradients by automatic differentiation of the forward pass."""
    out, grads, more = [], [], []
    for x in "qk":
        leaf = s[x].double().requires_grad_(s["train"])
        w = s["w" + x].double().requires_grad_(s["train"]) if s["w" + x] is not None else None
        y = _exact_row(leaf, w, s["table"], s["pos"], s["inter"])
        out.append(y.detach())
        if s["train"]:
            y.backward(s["d" + x].double())
            grads.append(leaf.grad)
            more.append(None if w is None else w.grad)
    return (*out, *grads, *more)


def _exact_group(x):
    """The values that a group of up to 64 channels is held as."""
    lo = x.amin(-1, keepdim=True).to(torch.bfloat16).double()
    step = torch.clamp((x.amax(-1, keepdim=True) - lo) / 15, min=0).to(torch.bfloat16).double()
    code = torch.clamp(torch.round((x - lo) / step), 0, 15)
    return torch.where(step > 0, lo + step * code, lo)


def _exact_head(cache, block, row, h, kv, d):
    """Values of K (kv = 0) or V (1) of head h: rows `row` of blocks `block` of the planes of
    that head, from the layout's definition, a channel at a time."""
    ng = -(-d // 64)
    plane = cache[:, h].reshape(-1, cache.shape[-1])
    out = torch.empty(len(row), d, dtype=torch.float64, device=DEV)
    for c in range(d):
        j, w, e = c // 64, c % 64 // 8, c % 8
        if kv == 0:
            word = row * 8 * ng + (w // 2) * 2 * ng + 2 * j + w % 2
        else:
            word = 128 * ng + 128 * j + 16 * w + (row % 8) // 2 * 4 + row % 2 + (row // 8) * 2
        code = torch.bitwise_and(plane[block, 4 * word + e // 2] >> (4 * (e % 2)), 15).double()
        if c % 64 == 0:
            at = 4 * (256 * ng + row * 2 * ng + kv * ng + j)
            two = torch.stack([plane[block, at + i] for i in range(4)], -1)
            two = two.view(torch.bfloat16).double()
        out[:, c] = two[:, 1] + two[:, 0] * code
    return out


def _exact_decode(s):
    b, hq, d = s["q"].shape
    hkv, page = s["cache"].shape[1], s["page"]
    out = torch.zeros(b, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(b, hq, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    at = torch.cat([torch.arange(n, device=DEV) for n in lens])
    req = torch.repeat_interleave(torch.arange(b, device=DEV), s["lens"].long())
    block = s["table"][req, at // page].long() * (page // 16) + at % page // 16
    ends = torch.cumsum(s["lens"].long(), 0).tolist()
    g = hq // hkv
    for h in range(hkv):
        k, v = (_exact_head(s["cache"], block, at % 16, h, i, d) for i in (0, 1))
        for i in range(b):
            rows = slice(ends[i] - lens[i], ends[i])
            x = s["q"][i, h * g:(h + 1) * g].double() @ k[rows].T / d ** 0.5
            lse[i, h * g:(h + 1) * g] = torch.logsumexp(x, dim=-1)
            out[i, h * g:(h + 1) * g] = torch.softmax(x, dim=-1) @ v[rows]
    return out, lse


def _exact_append(s):
    """Request by request."""
    cu, starts = s["cu"].tolist(), s["starts"].tolist()
    pos = torch.cat([torch.arange(a, a + cu[i + 1] - cu[i], device=DEV)
                     for i, a in enumerate(starts)])
    q, k = (_exact_row(s[x], s["w" + x], s["table"], pos, s["inter"]) for x in "qk")
    v, page = s["v"].double(), s["page"]
    if s["kind"] == "append":
        kc, vc = s["kc"].double(), s["vc"].double()
        for i, a in enumerate(starts):
            p = torch.arange(a, a + cu[i + 1] - cu[i], device=DEV)
            where = s["pages"][i, p // page].long() * page + p % page
            for cache, new in ((kc, k), (vc, v)):
                for h in range(cache.shape[1]):
                    plane = cache[:, h].reshape(-1, s["d"])
                    plane[where] = new[cu[i]:cu[i + 1], h]
                    cache[:, h] = plane.view(-1, page, s["d"])
        return q, kc, vc
    parts = ([], [])
    for i, a in enumerate(starts):
        p = torch.arange(a, device=DEV)
        block = s["pages"][i, p // page].long() * (page // 16) + p % page // 16
        for kv, new in ((0, k), (1, v)):
            old = [_exact_head(s["cache"], block, p % 16, h, kv, s["d"])
                   for h in range(s["cache"].shape[1])]
            rows = new[cu[i]:cu[i + 1]]
            held = torch.cat([_exact_group(g) for g in rows.split(64, -1)], -1)
            parts[kv].append(torch.cat([torch.stack(old, 1), held]))
    return (q, *(torch.cat(x) for x in parts))


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk": _exact_qk, "append": _exact_append, "chunk4": _exact_append,
            "decode4": _exact_decode}[s["kind"]](s)
