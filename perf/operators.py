"""Cases, plain forms and 64-bit values of the packed and paged attention operators.

The operators, in the layouts of the package's entry points (bf16 in and out):

  packed forward    Q [T, Hq, d], K and V [T, Hkv, d] hold sequences one after another,
                    bounded by cu_seqlens [nseq + 1]; query head h reads key/value head
                    h // (Hq / Hkv). Per sequence O = softmax(scale Q K^T) V, causal or not,
                    and L = logsumexp per row, fp32 [Hq, T].
  packed training   the same forward, then dQ, dK, dV for a given dO.
  prefix decode     one new token for each of B requests, Q [B, Hq, d]. Keys and values are
                    in pages of a cache [pages, Hkv, page, d]: a prefix that all requests
                    share (prefix_pages, prefix_len) and each request's own tokens after it
                    (block_table [B, max_pages], lens [B]).
  cache append      new K and V rows [T, Hkv, d] of several requests (cu_seqlens) written to
                    the pages their block tables name, from cache position starts[i] on.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is
true, with the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # A few short prompts that arrive together at a small model: latency counts.
        dict(name="prompts_small", kind="forward", total=212, nseq=4, lens_seed=3, hq=8, hkv=2,
             d=64, causal=True),
        # A serving step's prompts of mixed lengths, grouped heads.
        dict(name="prompts_mixed", kind="forward", total=8192, nseq=16, lens_seed=5, hq=32,
             hkv=8, d=128, causal=True),
        # Long documents, the longest about half of the batch.
        dict(name="prompts_long", kind="forward", total=32768, nseq=5, lens_seed=1, hq=32, hkv=8,
             d=128, causal=True),
        # An odd head dimension and a small ragged batch, both directions.
        dict(name="train_small", kind="train", total=333, nseq=5, lens_seed=7, hq=6, hkv=2, d=96,
             causal=True),
        # Packed pre-training rows with as many key/value heads as query heads.
        dict(name="train_mha", kind="train", total=8192, nseq=23, lens_seed=2, hq=16, hkv=16,
             d=64, causal=True),
        # Packed training of a model with grouped heads.
        dict(name="train_grouped", kind="train", total=16384, nseq=12, lens_seed=4, hq=32, hkv=8,
             d=128, causal=True),
        # Two requests behind a short system prompt: the smallest decode step.
        dict(name="decode_small", kind="decode", batch=2, prefix=100, own_max=24, lens_seed=1,
             hq=8, hkv=2, d=64, page=16),
        # A serving batch behind a common system prompt.
        dict(name="decode_batch", kind="decode", batch=32, prefix=2000, own_max=512, lens_seed=2,
             hq=32, hkv=8, d=128, page=16),
        # Many requests over one long document.
        dict(name="decode_wide", kind="decode", batch=256, prefix=8192, own_max=2048, lens_seed=3,
             hq=32, hkv=8, d=128, page=64),
        # A few samples of one very long context: work has to be split along the keys.
        dict(name="decode_long", kind="decode", batch=4, prefix=100000, own_max=8000, lens_seed=4,
             hq=16, hkv=2, d=128, page=32),
        # The keys and values of one decode step, one token for each request.
        dict(name="append_step", kind="append", total=64, nseq=64, lens_seed=1, start_max=2000,
             hkv=8, d=128, page=16),
        # The keys and values of a batch of prompts.
        dict(name="append_prompts", kind="append", total=32768, nseq=24, lens_seed=2,
             start_max=1000, hkv=8, d=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pair(case):
    """Sum over the sequences of visible (query, key) pairs."""
    lens = _lengths(case["total"], case["nseq"], case["lens_seed"])
    return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)


def _draw_packed(rng, kind):
    most = 2.0e12 if kind == "forward" else 1.0e12
    while True:
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        # Rows of one token have gradients of exactly zero: a training batch is longer.
        total = _log_int(rng, 1 if kind == "forward" else 32, 20000)
        nseq = min(total if kind == "forward" else total // 16, _log_int(rng, 1, 40))
        c = dict(kind=kind, total=total, nseq=nseq, lens_seed=rng.randrange(1 << 20),
                 hq=min(hq, 32), hkv=hkv, d=rng.choice([32, 40, 64, 80, 96, 128, 128]),
                 causal=rng.random() < 0.75)
        if work(c)["flops"] <= most:
            return c


def draw(rng):
    kind = rng.choice(["forward", "train", "decode", "decode", "append"])
    if kind in ("forward", "train"):
        return _draw_packed(rng, kind)
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([32, 64, 72, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if kind == "append":
        total = _log_int(rng, 1, 30000)
        return dict(kind=kind, total=total, nseq=min(total, _log_int(rng, 1, 200)),
                    lens_seed=rng.randrange(1 << 20), start_max=_log_int(rng, 1, 2000), hkv=hkv,
                    d=d, page=page)
    batch = _log_int(rng, 1, 200)
    return dict(kind=kind, batch=batch, prefix=_log_int(rng, 1, 8000),
                own_max=_log_int(rng, 1, min(8000, 200000 // batch)),
                lens_seed=rng.randrange(1 << 20), hq=hkv * rng.choice([1, 2, 4, 5, 8, 16]),
                hkv=hkv, d=d, page=page)


def _lengths(total, nseq, seed):
    """nseq lengths >= 1 that sum to total, unequal as real batches are."""
    r = random.Random(seed)
    w = [r.expovariate(1.0) + 0.02 for _ in range(nseq)]
    s = sum(w)
    n = [1 + int((total - nseq) * x / s) for x in w]
    n[0] += total - sum(n)
    return n


def _own_lengths(case):
    """Tokens of each request after the shared prefix: from 1 to own_max."""
    r = random.Random(case["lens_seed"])
    return [r.randint(1, case["own_max"]) for _ in range(case["batch"])]


def _starts(case):
    r = random.Random(case["lens_seed"] + 1)
    return [r.randint(0, case["start_max"]) for _ in range(case["nseq"])]


def work(case):
    kind, d, hkv = case["kind"], case["d"], case["hkv"]
    if kind == "append":  # each row read once and written once; tables and lengths
        return {"bytes": 2 * 2 * case["total"] * hkv * d * 2 + 12 * case["nseq"], "flops": 0}
    hq = case["hq"]
    if kind == "decode":
        lens = _own_lengths(case)
        keys = case["prefix"] + sum(lens)
        pairs = sum(case["prefix"] + n for n in lens)
        return {"bytes": 2 * keys * hkv * d * 2 + case["batch"] * hq * (4 * d + 4),
                "flops": 4 * pairs * hq * d}
    t, pairs = case["total"], _pair(case)
    qo, kv, lse = t * hq * d * 2, t * hkv * d * 2, t * hq * 4
    if kind == "forward":
        return {"bytes": 2 * qo + 2 * kv + lse, "flops": 4 * pairs * hq * d}
    # reads Q, K, V, dO, writes O, dQ, dK, dV; five products backward for two forward
    return {"bytes": 4 * qo + 4 * kv, "flops": 14 * pairs * hq * d}


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


def _pages(need, page, spare, gen):
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
    return table, order[total:], total + spare


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, d, hkv = case["kind"], case["d"], case["hkv"]
    if kind in ("forward", "train"):
        lens = _lengths(case["total"], case["nseq"], case["lens_seed"])
        t, hq = case["total"], case["hq"]
        s = dict(kind=kind, lens=lens, causal=case["causal"], q=_randn(gen, t, hq, d),
                 k=_randn(gen, t, hkv, d), v=_randn(gen, t, hkv, d), cu=_ints(_bounds(lens)))
        if kind == "train":
            s["do"] = _randn(gen, t, hq, d)
        if own:
            import exact_io_aware_27_gb300 as fa
            # The plan of one batch serves every layer of the model.
            s["plan"] = fa.fa_packed_plan(s["cu"], t, causal=case["causal"])
            if kind == "train":
                s["ws"] = fa.alloc_packed_workspace(s["plan"], hq, d)
        return s
    page = case["page"]
    if kind == "append":
        lens, starts = _lengths(case["total"], case["nseq"], case["lens_seed"]), _starts(case)
        table, _, pages = _pages([a + n for a, n in zip(starts, lens)], page, 3, gen)
        return dict(kind=kind, k=_randn(gen, case["total"], hkv, d),
                    v=_randn(gen, case["total"], hkv, d), cu=_ints(_bounds(lens)),
                    starts=_ints(starts), table=table, page=page,
                    kc=_randn(gen, pages, hkv, page, d), vc=_randn(gen, pages, hkv, page, d))
    lens, b, hq = _own_lengths(case), case["batch"], case["hq"]
    shared = -(-case["prefix"] // page)
    table, rest, pages = _pages(lens, page, shared + 2, gen)
    s = dict(kind=kind, q=_randn(gen, b, hq, d), kc=_randn(gen, pages, hkv, page, d),
             vc=_randn(gen, pages, hkv, page, d), prefix_pages=rest[:shared].contiguous(),
             prefix_len=_ints([case["prefix"]]), table=table, lens=_ints(lens))
    if own:
        import exact_io_aware_27_gb300 as fa
        s["ws"] = fa.alloc_prefix_workspace(b, hq, hkv, d, shared * page, table.shape[1] * page,
                                            s["q"].device)
    return s


# ---------------------------------------------------------------- plain forms, 32 bits
def _head_steps(n, group, hkv):
    """Key/value heads at a time, so that the scores stay within a few GB."""
    return max(1, min(hkv, (1 << 29) // max(1, n * n * group)))


def _plain_scores(q, k, scale, causal):
    """q [h, g, n, d], k [h, n, d]: masked scores [h, g, n, n]."""
    s = torch.matmul(q, k.unsqueeze(1).transpose(-1, -2)) * scale
    if causal:
        i = torch.arange(q.shape[-2], device=q.device)
        s = s.masked_fill(i[None, :] > i[:, None], -math.inf)
    return s


def _plain_packed(s):
    q, k, v = s["q"], s["k"], s["v"]
    t, hq, d = q.shape
    hkv = k.shape[1]
    g, scale = hq // hkv, 1.0 / math.sqrt(d)
    train = s["kind"] == "train"
    out = torch.empty(t, hq, d, dtype=torch.float32, device=q.device)
    lse = torch.empty(hq, t, dtype=torch.float32, device=q.device)
    if train:
        dq = torch.empty_like(out)
        dk = torch.empty(t, hkv, d, dtype=torch.float32, device=q.device)
        dv = torch.empty_like(dk)
    at = 0
    for n in s["lens"]:
        step = _head_steps(n, g, hkv)
        for h in range(0, hkv, step):
            e = min(hkv, h + step)
            rows, heads = slice(at, at + n), slice(h * g, e * g)
            as_q = lambda x: x[rows, heads].float().transpose(0, 1).reshape(e - h, g, n, d)  # noqa: E731
            as_k = lambda x: x[rows, h:e].float().transpose(0, 1)  # noqa: E731
            back = lambda x: x.reshape((e - h) * g, n, d).transpose(0, 1)  # noqa: E731
            qf, kf, vf = as_q(q), as_k(k), as_k(v)
            sc = _plain_scores(qf, kf, scale, s["causal"])
            m = sc.amax(dim=-1, keepdim=True)
            p = torch.exp(sc - m)
            del sc
            l = p.sum(dim=-1, keepdim=True)
            p = p / l
            o = torch.matmul(p, vf.unsqueeze(1))
            out[rows, heads] = back(o)
            lse[heads, rows] = (m + torch.log(l)).reshape((e - h) * g, n)
            if train:
                do = as_q(s["do"])
                delta = (do * o).sum(dim=-1, keepdim=True)
                dv[rows, h:e] = torch.matmul(p.transpose(-1, -2), do).sum(dim=1).transpose(0, 1)
                dp = torch.matmul(do, vf.unsqueeze(1).transpose(-1, -2))
                ds = p * (dp - delta) * scale
                del dp, p
                dq[rows, heads] = back(torch.matmul(ds, kf.unsqueeze(1)))
                dk[rows, h:e] = torch.matmul(ds.transpose(-1, -2), qf).sum(dim=1).transpose(0, 1)
                del ds
        at += n
    if train:
        return tuple(x.to(torch.bfloat16) for x in (out, dq, dk, dv))
    return out.to(torch.bfloat16), lse


def _gather(cache, pages):
    """Rows of the pages in order: [..., pages * page, Hkv, d] in 32 bits."""
    x = cache[pages.long()].float()  # [..., p, Hkv, page, d]
    x = x.transpose(-3, -2)
    return x.reshape(*x.shape[:-4], x.shape[-4] * x.shape[-3], x.shape[-2], x.shape[-1])


def _plain_decode(s):
    q, lens = s["q"], s["lens"]
    b, hq, d = q.shape
    hkv = s["kc"].shape[1]
    g, scale = hq // hkv, 1.0 / math.sqrt(d)
    qf = q.float().view(b, hkv, g, d)
    kp, vp = _gather(s["kc"], s["prefix_pages"]), _gather(s["vc"], s["prefix_pages"])
    ks, vs = _gather(s["kc"], s["table"]), _gather(s["vc"], s["table"])
    np_, ns = kp.shape[0], ks.shape[1]
    # the shared keys once for all requests: [Hkv, b * g, keys]
    rows = qf.transpose(0, 1).reshape(hkv, b * g, d)
    sp = torch.matmul(rows, kp.permute(1, 2, 0)).view(hkv, b, g, np_).transpose(0, 1) * scale
    so = torch.matmul(qf, ks.permute(0, 2, 3, 1)) * scale
    at = torch.arange(max(np_, ns), device=q.device)
    sp = sp.masked_fill(at[:np_] >= s["prefix_len"], -math.inf)
    so = so.masked_fill((at[:ns] >= lens[:, None])[:, None, None, :], -math.inf)
    m = torch.maximum(sp.amax(dim=-1, keepdim=True), so.amax(dim=-1, keepdim=True))
    pp, po = torch.exp(sp - m), torch.exp(so - m)
    l = pp.sum(dim=-1, keepdim=True) + po.sum(dim=-1, keepdim=True)
    o = torch.matmul(pp.transpose(0, 1).reshape(hkv, b * g, np_), vp.transpose(0, 1))
    o = o.view(hkv, b, g, d).transpose(0, 1) + torch.matmul(po, vs.permute(0, 2, 1, 3))
    lse = (m + torch.log(l)).reshape(b, hq)
    return (o / l).reshape(b, hq, d).to(torch.bfloat16), lse


def _plain_append(s):
    t = torch.arange(s["k"].shape[0], device=s["k"].device)
    req = (t[:, None] >= s["cu"][None, 1:]).sum(dim=1)
    pos = s["starts"][req] + t - s["cu"][req]
    page = s["table"][req, pos // s["page"]].long()
    s["kc"][page, :, pos % s["page"]] = s["k"]
    s["vc"][page, :, pos % s["page"]] = s["v"]
    return s["kc"], s["vc"]


def run(state):
    s = state
    if not own:
        return {"forward": _plain_packed, "train": _plain_packed, "decode": _plain_decode,
                "append": _plain_append}[s["kind"]](s)
    import exact_io_aware_27_gb300 as fa
    if s["kind"] == "append":
        fa.fa_cache_append(s["k"], s["v"], s["cu"], s["starts"], s["table"], s["kc"], s["vc"])
        return s["kc"], s["vc"]
    if s["kind"] == "decode":
        return fa.fa_prefix_decode(s["q"], s["kc"], s["vc"], s["prefix_pages"], s["prefix_len"],
                                   s["table"], s["lens"], workspace=s["ws"])
    o, lse = fa.fa_packed_forward(s["q"], s["k"], s["v"], s["plan"])
    if s["kind"] == "forward":
        return o, lse
    return (o, *fa.fa_packed_backward(s["q"], s["k"], s["v"], o, lse, s["do"], s["plan"],
                                      workspace=s["ws"]))


# ---------------------------------------------------------------- 64 bits
def _exact_packed(s):
    """Head by head and sequence by sequence, from the definitions: O = P V with
    P = softmax(scale Q K^T), and the gradients through the softmax's Jacobian."""
    t, hq, d = s["q"].shape
    hkv = s["k"].shape[1]
    o = torch.zeros(t, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(hq, t, dtype=torch.float64, device=DEV)
    train = "do" in s
    if train:
        dq = torch.zeros_like(o)
        dk = torch.zeros(t, hkv, d, dtype=torch.float64, device=DEV)
        dv = torch.zeros_like(dk)
    ends = torch.cumsum(torch.tensor(s["lens"]), 0).tolist()
    for end, n in zip(ends, s["lens"]):
        hidden = torch.triu(torch.ones(n, n, dtype=torch.bool, device=DEV), 1)
        for h in range(hq):
            kh = h * hkv // hq
            part = [s[x][end - n:end, i].double() for x, i in (("q", h), ("k", kh), ("v", kh))]
            x = part[0] @ part[1].T
            x /= d ** 0.5
            if s["causal"]:
                x[hidden] = -math.inf
            lse[h, end - n:end] = torch.logsumexp(x, dim=1)
            x = torch.softmax(x, dim=1)
            o[end - n:end, h] = x @ part[2]
            if train:
                g = s["do"][end - n:end, h].double()
                dv[end - n:end, kh] += x.T @ g
                y = g @ part[2].T
                y -= (x * y).sum(dim=1, keepdim=True)
                y *= x
                y /= d ** 0.5
                dq[end - n:end, h] = y @ part[1]
                dk[end - n:end, kh] += y.T @ part[0]
    return (o, dq, dk, dv) if train else (o, lse)


def _exact_decode(s):
    """Request by request over the keys and values laid end to end."""
    b, hq, d = s["q"].shape
    hkv, page = s["kc"].shape[1], s["kc"].shape[2]
    lens, plen = s["lens"].tolist(), int(s["prefix_len"])
    out = torch.zeros(b, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(b, hq, dtype=torch.float64, device=DEV)

    def rows(cache, pages, n):
        return torch.cat([cache[p].double() for p in pages[:-(-n // page)].tolist()], 1)[:, :n]

    first = [rows(c, s["prefix_pages"], plen) for c in (s["kc"], s["vc"])]
    for i in range(b):
        k, v = (torch.cat([f, rows(c, s["table"][i], lens[i])], 1)
                for f, c in zip(first, (s["kc"], s["vc"])))
        qs = s["q"][i].double().view(hkv, hq // hkv, d)
        x = torch.einsum("hgd,hnd->hgn", qs, k) / d ** 0.5
        lse[i] = torch.logsumexp(x, dim=-1).reshape(hq)
        out[i] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, dim=-1), v).reshape(hq, d)
    return out, lse


def _exact_append(s):
    """Token by token in the order of the requests."""
    kc, vc = s["kc"].double(), s["vc"].double()
    cu, table = s["cu"].tolist(), s["table"].tolist()
    where = [(table[i][p // s["page"]], p % s["page"])
             for i, at in enumerate(s["starts"].tolist())
             for p in range(at, at + cu[i + 1] - cu[i])]
    flat = torch.tensor([a * s["page"] + r for a, r in where], device=DEV)
    for cache, new in ((kc, s["k"]), (vc, s["v"])):
        pages, hkv, page, d = cache.shape
        for h in range(hkv):
            plane = cache[:, h].reshape(pages * page, d)
            plane.index_copy_(0, flat, new[:, h].double())
            cache[:, h] = plane.view(pages, page, d)
    return kc, vc


def exact(case, seed):
    s = prepare(case, seed)
    return {"forward": _exact_packed, "train": _exact_packed, "decode": _exact_decode,
            "append": _exact_append}[s["kind"]](s)
