"""The paged cache and decode attention behind a shared prefix, against 64-bit values with
elementwise bounds (tests/packed_ref.py)."""
import math
import random

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests.packed_ref import assert_close, attention64, packed_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def _batch(prefix, lens, hq, hkv, d, page, seed, spare=3, fill=0.0):
    """Queries, caches whose unused rows hold `fill`, tables over shuffled pages, and the
    keys and values of each request in order."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = -(-prefix // page) + sum(-(-n // page) for n in lens) + spare
    order = torch.randperm(pages, generator=g).tolist()
    kc = torch.full((pages, hkv, page, d), fill, dtype=torch.bfloat16)
    vc = kc.clone()
    rows = {}

    def place(n):
        mine = [order.pop() for _ in range(-(-n // page))]
        k = torch.randn(n, hkv, d, generator=g).to(torch.bfloat16)
        v = torch.randn(n, hkv, d, generator=g).to(torch.bfloat16)
        for i, pg in enumerate(mine):
            part = slice(i * page, min(n, (i + 1) * page))
            m = part.stop - part.start
            kc[pg, :, :m] = k[part].transpose(0, 1)
            vc[pg, :, :m] = v[part].transpose(0, 1)
        return mine, k, v

    shared, pk, pv = place(prefix)
    most = max([1] + [-(-n // page) for n in lens])
    table = torch.full((B, most), -7, dtype=torch.int32)  # entries past a length: never read
    keys = []
    for b, n in enumerate(lens):
        mine, k, v = place(n)
        table[b, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
        keys.append((torch.cat([pk, k]), torch.cat([pv, v])))
    q = torch.randn(B, hq, d, generator=g).to(torch.bfloat16)
    dev = lambda x, t=None: torch.as_tensor(x, dtype=t).cuda()  # noqa: E731
    args = [dev(q), dev(kc), dev(vc), dev(shared, torch.int32), dev([prefix], torch.int32),
            dev(table), dev(lens, torch.int32)]
    return args, keys


def _reference(q, keys, hkv, scale=None):
    """Values and bounds of O [B, Hq, d] and L [B, Hq]. The parts' join adds fp32 roundings
    and one more exp2 per part: covered by the bounds' 2^-14 and 2^-20 terms."""
    B, hq, d = q.shape
    g, scale = hq // hkv, 1.0 / math.sqrt(d) if scale is None else scale
    out = {n: [torch.zeros(*s, dtype=torch.float64, device="cuda") for _ in (0, 1)]
           for n, s in (("O", (B, hq, d)), ("L", (B, hq)))}
    for b, (k, v) in enumerate(keys):
        for h in range(hkv):
            hs = slice(h * g, (h + 1) * g)
            if k.shape[0] == 0:
                out["L"][0][b, hs] = -math.inf
                continue
            r = attention64(q[b, hs].double()[:, None], k[:, h].double().cuda(),
                            v[:, h].double().cuda(), False, scale)
            for i in (0, 1):
                out["O"][i][b, hs] = r["O"][i][:, 0]
                out["L"][i][b, hs] = r["L"][i][:, 0]
    return out


def _wide(args):
    """The same call with a table for long contexts, whose capacity rules the single-kernel
    form for small calls out."""
    table = args[5]
    more = torch.full((table.shape[0], 200000 // args[1].shape[2]), -9, dtype=torch.int32,
                      device="cuda")
    return [*args[:5], torch.cat([table, more], 1), *args[6:]]


def _check(args, keys, hkv, scale=None, **kw):
    """Both forms of the call, where the small one takes it."""
    want = _reference(args[0], keys, hkv, scale)
    some = torch.tensor([k.shape[0] > 0 for k, _ in keys], device="cuda")
    for call in (args, _wide(args)):
        O, L = fa.fa_prefix_decode(*call, scale=scale, **kw)
        assert_close("O", O, want["O"])
        assert_close("L", L, want["L"], mask=some[:, None].expand_as(L))
        assert torch.all(L[~some] == -math.inf) and torch.all(O[~some] == 0)
    return O, L


@pytest.mark.parametrize("prefix", [0, 1, 16, 100, 128, 129, 700])
@pytest.mark.parametrize("lens", [[1], [0, 5, 64], [17, 65, 128, 300, 2]])
def test_decode(prefix, lens):
    args, keys = _batch(prefix, lens, 8, 2, 64, 16, 7 + prefix)
    _check(args, keys, 2)


@pytest.mark.parametrize("hq,hkv,d,page", [
    (1, 1, 8, 16), (4, 4, 40, 32), (7, 1, 72, 64), (16, 1, 128, 128), (20, 1, 96, 256),
    (40, 2, 128, 16), (128, 1, 64, 32), (66, 2, 120, 1024)])
def test_decode_heads_dims_and_pages(hq, hkv, d, page):
    args, keys = _batch(333, [40, 1, 130], hq, hkv, d, page, hq + d)
    _check(args, keys, hkv, scale=0.2)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_many_requests(d):
    """More rows than a tile pair holds, and units that span and share workers."""
    r = random.Random(3)
    lens = [r.choice([0, 1, 15, 16, 17, 63, 64, 65, 200, 513]) for _ in range(150)]
    args, keys = _batch(900, lens, 16, 4, d, 16, 19)
    a = _check(args, keys, 4)
    b = fa.fa_prefix_decode(*_wide(args))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_decode_long_keys_of_few_requests():
    args, keys = _batch(20000, [9000, 3], 8, 1, 128, 64, 23)
    _check(args, keys, 1)


@pytest.mark.parametrize("B,hq,hkv,d,page", [(4, 16, 2, 128, 32), (3, 10, 1, 64, 16),
                                             (2, 64, 8, 40, 16), (1, 8, 8, 128, 64),
                                             (32, 8, 8, 96, 16), (33, 4, 4, 128, 16)])
@pytest.mark.parametrize("prefix", [1, 129, 9000])
def test_decode_few_rows_behind_a_long_prefix(B, hq, hkv, d, page, prefix):
    """Up to 32 rows a key/value head and one more, pieces of one unit and of several."""
    args, keys = _batch(prefix, [(7 * i) % 90 for i in range(B)], hq, hkv, d, page, 27 + B)
    a = _check(args, keys, hkv)
    b = fa.fa_prefix_decode(*_wide(args))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("B,hq,hkv", [(3, 4, 2), (40, 4, 2), (40, 32, 2)])
def test_decode_lengths_of_zero_within_capacities(B, hq, hkv):
    """Pages are listed, but the lengths on the device are 0: the prefix's, everyone's own,
    and both."""
    args, keys = _batch(700, [30 + i for i in range(B)], hq, hkv, 64, 16, 31)
    own = [(k[700:], v[700:]) for k, v in keys]
    shared = [(k[:700], v[:700]) for k, v in keys]
    zero = torch.zeros_like
    _check([*args[:4], zero(args[4]), *args[5:]], own, hkv)
    _check([*args[:6], zero(args[6])], shared, hkv)
    for call in (args, _wide(args)):
        O, L = fa.fa_prefix_decode(*call[:4], zero(args[4]), call[5], zero(args[6]))
        assert torch.all(O == 0) and torch.all(L == -math.inf)


@pytest.mark.parametrize("prefix", [0, 300])
def test_decode_the_largest_batch(prefix):
    B, hq, hkv, d = 8192, 2, 1, 32
    args, keys = _batch(prefix, [i % 3 for i in range(B)], hq, hkv, d, 16, 33)
    some = list(range(0, B, 431)) + [B - 1]
    want = _reference(args[0][some], [keys[i] for i in some], hkv)
    has = torch.tensor([keys[i][0].shape[0] > 0 for i in some], device="cuda")
    for call in (args, _wide(args)):
        O, L = fa.fa_prefix_decode(*call)
        assert_close("O", O[some], want["O"])
        assert_close("L", L[some], want["L"], mask=has[:, None].expand(-1, hq))


def test_decode_without_prefix_or_own():
    args, keys = _batch(0, [30, 0, 200], 4, 2, 64, 16, 29)
    args[3] = args[4] = None
    _check(args, keys, 2)
    args, keys = _batch(50, [0, 0], 4, 2, 64, 16, 31)
    args[5] = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    _check(args, keys, 2)
    # a prefix whose pages are listed but whose length is 0, and no key at all
    args, keys = _batch(20, [0, 3], 4, 2, 64, 16, 37)
    args[4].zero_()
    _check(args, [(k[20:], v[20:]) for k, v in keys], 2)


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_decode_ignores_what_pages_held_before(value):
    args, keys = _batch(70, [5, 33], 4, 2, 128, 64, 41, fill=value)
    _check(args, keys, 2)


@pytest.mark.parametrize("wide", [False, True])
def test_decode_requests_do_not_leak(wide):
    args, keys = _batch(40, [33, 70, 5], 4, 2, 64, 16, 43)
    args = _wide(args) if wide else args
    clean = fa.fa_prefix_decode(*args)
    args[0][1] = math.nan
    page = int(args[5][1, 0])
    args[1][page], args[2][page] = math.nan, math.nan
    O, L = fa.fa_prefix_decode(*args)
    for b in (0, 2):
        assert torch.equal(O[b], clean[0][b]) and torch.equal(L[b], clean[1][b])
    assert torch.isnan(O[1].float()).all()


@pytest.mark.parametrize("wide", [False, True])
def test_decode_reports_bad_indices(wide):
    """A bad page or length is reported, and the other requests keep their results."""
    args, keys = _batch(40, [33, 70, 5], 4, 2, 64, 16, 47)
    args = _wide(args) if wide else args
    clean = fa.fa_prefix_decode(*args)
    for bad in (10 ** 6, -1, args[1].shape[0]):
        table = args[5].clone()
        table[1, 2] = bad
        O, L = fa.fa_prefix_decode(*args[:5], table, args[6])
        assert fa.fa_get_device_status() == -8
        for b in (0, 2):
            assert torch.equal(O[b], clean[0][b]) and torch.equal(L[b], clean[1][b])
    for bad in (-1, 10 ** 6):
        lens = args[6].clone()
        lens[0] = bad
        table = args[5].clone().clamp_(min=0)  # more of the row is read than was filled
        O, L = fa.fa_prefix_decode(*args[:5], table, lens)
        assert fa.fa_get_device_status() == -8
        assert torch.equal(O[2], clean[0][2])
    pages = args[3].clone()
    pages[1] = args[1].shape[0]
    fa.fa_prefix_decode(*args[:3], pages, *args[4:])
    assert fa.fa_get_device_status() == -8
    fa.fa_prefix_decode(*args[:4], args[4] + 1000, *args[5:])
    assert fa.fa_get_device_status() == -8
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("wide", [False, True])
def test_decode_in_a_graph_and_on_another_stream(wide):
    args, keys = _batch(300, [40, 90], 8, 2, 64, 16, 53)
    args = _wide(args) if wide else args
    want = fa.fa_prefix_decode(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.fa_prefix_decode(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = fa.alloc_prefix_workspace(2, 8, 2, 64, 300000, 300000, "cuda")  # more than needed
    ws.fill_(255)
    O, L = torch.empty_like(args[0]), torch.empty(2, 8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_prefix_decode(*args, O=O, L=L, workspace=ws)
    # A replay follows the lengths on the device.
    args[4].fill_(130)
    args[6].copy_(torch.tensor([7, 66], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    keys = [(torch.cat([k[:130], k[300:300 + n]]), torch.cat([v[:130], v[300:300 + n]]))
            for (k, v), n in zip(keys, (7, 66))]
    ref = _reference(args[0], keys, 2)
    assert_close("O", O, ref["O"])
    assert_close("L", L, ref["L"])


def test_decode_with_pages_listed_more_than_once():
    """Requests that share pages, name one twice, and name the prefix's."""
    args, keys = _batch(64, [32, 48], 8, 2, 64, 16, 73)
    pages, table = args[3].tolist(), args[5]
    table[1, :3] = torch.tensor([int(table[0, 1]), int(table[0, 1]), pages[0]], dtype=torch.int32)
    args[3] = torch.tensor([pages[1], pages[1], pages[2], pages[2]], dtype=torch.int32,
                           device="cuda")

    def rows(i, lo, hi):
        return keys[i][0][lo:hi], keys[i][1][lo:hi]

    def cat(*parts):
        return tuple(torch.cat(x) for x in zip(*parts))

    p1, p2 = rows(0, 16, 32), rows(0, 32, 48)
    prefix = [p1, p1, p2, p2]
    own1 = rows(0, 80, 96)  # the second page of request 0
    keys = [cat(*prefix, rows(0, 64, 96)), cat(*prefix, own1, own1, rows(0, 0, 16))]
    _check(args, keys, 2)


def test_decode_calls_on_two_streams_at_once():
    jobs = []
    for i, (prefix, lens) in enumerate([(3000, [70] * 40), (100, [9000, 40])]):
        args, _ = _batch(prefix, lens, 8, 2, 128, 16, 79 + i)
        B = len(lens)
        ws = fa.alloc_prefix_workspace(B, 8, 2, 128, 16 * args[3].numel(),
                                       16 * args[5].shape[1], "cuda")
        outs = [(torch.empty_like(args[0]), torch.empty(B, 8, device="cuda")) for _ in range(8)]
        jobs.append((torch.cuda.Stream(), args, ws, fa.fa_prefix_decode(*args), outs))
    torch.cuda.synchronize()
    for r in range(8):
        for s, args, ws, want, outs in jobs:
            fa.fa_prefix_decode(*args, O=outs[r][0], L=outs[r][1], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for s, args, ws, want, outs in jobs:
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


def test_cache_beyond_32_bits():
    """Pages whose values lie more than 2^31 into the cache."""
    hq, hkv, d, page, pages = 16, 8, 128, 1024, 2060
    assert (pages - 8) * hkv * page * d > 2 ** 31
    g = torch.Generator().manual_seed(83)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    mk = lambda n, h: torch.randn(n, h, d, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    kc = torch.empty(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    shared, table = i32([pages - 1]), i32([[pages - 2, pages - 5], [pages - 3, 0]])
    pk, pv, k, v = mk(900, hkv), mk(900, hkv), mk(1500 + 70, hkv), mk(1500 + 70, hkv)
    fa.fa_cache_append(pk, pv, i32([0, 900]), i32([0]), shared[None], kc, vc)
    fa.fa_cache_append(k, v, i32([0, 1500, 1570]), i32([0, 0]), table, kc, vc)
    keys = [(torch.cat([pk, k[a:b]]).cpu(), torch.cat([pv, v[a:b]]).cpu())
            for a, b in ((0, 1500), (1500, 1570))]
    _check([mk(2, hq), kc, vc, shared, i32([900]), table, i32([1500, 70])], keys, hkv)


@pytest.mark.parametrize("hkv,d,page", [(1, 8, 16), (2, 64, 32), (3, 72, 16), (8, 128, 64)])
@pytest.mark.parametrize("lens,starts", [([1], [0]), ([3, 0, 40, 1], [15, 9, 16, 100]),
                                         ([1] * 33, list(range(33)))])
def test_append(hkv, d, page, lens, starts):
    _, k, v, _, cu = packed_inputs(lens, 1, hkv, d, 61, rest=4)
    need = [a + n for a, n in zip(starts, lens)]
    count = [-(-n // page) for n in need]
    pages = sum(count) + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).tolist()
    table = torch.full((len(lens), max(1, max(count))), -1, dtype=torch.int32)
    kc = torch.full((pages, hkv, page, d), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 4.0)
    want_k, want_v = kc.clone(), vc.clone()
    at = 0
    for i, n in enumerate(lens):
        for j in range(count[i]):
            table[i, j] = order.pop()
        for t in range(n):
            pos = starts[i] + t
            pg = int(table[i, pos // page])
            want_k[pg, :, pos % page] = k[at + t]
            want_v[pg, :, pos % page] = v[at + t]
        at += n
    fa.fa_cache_append(k, v, cu, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       table.cuda(), kc, vc)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_append_reports_places_out_of_range():
    lens, starts = [2, 2, 2, 2], [0, 31, -1, 0]
    _, k, v, _, cu = packed_inputs(lens, 1, 2, 64, 67)
    table = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device="cuda")
    table[3] = 8  # the cache has 8 pages: 8 is out of range
    kc = torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    fa.fa_cache_append(k, v, cu, torch.tensor(starts, dtype=torch.int32, device="cuda"), table, kc,
                       vc)
    assert fa.fa_get_device_status() == -8
    want = torch.zeros_like(kc)
    want[0, :, 0], want[0, :, 1], want[3, :, 15] = k[0], k[1], k[2]
    assert torch.equal(kc, want)


def test_prompt_cache_and_decode_together():
    """A serving run: the shared prompt and the requests' own prompts fill the cache, and
    decode steps append and attend; each step's output is that of the packed forward pass
    over the whole sequence, to the 64-bit bounds."""
    hq, hkv, d, page, prefix = 8, 2, 64, 16, 90
    own = [20, 1, 47]
    steps, B = 3, len(own)
    g = torch.Generator().manual_seed(71)
    mk = lambda n, h: torch.randn(n, h, d, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kc = torch.full((40, hkv, page, d), math.nan, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    wide = mk(prefix, hq + 2 * hkv)  # one projection: the slices go in as they are
    qp, kp, vp = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:]
    ppages = i32([3, 9, 1, 0, 7, 22])
    fa.fa_cache_append(kp, vp, i32([0, prefix]), i32([0]), ppages[None], kc, vc)
    plan = fa.fa_packed_plan(i32([0, prefix]), prefix)
    O, _ = fa.fa_packed_forward(qp, kp, vp, plan)
    ref = attention64(qp[:, :4].double().transpose(0, 1), kp[:, 0].double(), vp[:, 0].double(),
                      True, d ** -0.5)
    assert_close("prompt", O[:, :4], tuple(x.transpose(0, 1) for x in ref["O"]))
    table = i32([[10, 11, 12, 13], [14, 15, 16, 17], [18, 19, 20, 21]])
    k, v = mk(sum(own), hkv), mk(sum(own), hkv)
    bounds = [0, 20, 21, 68]
    fa.fa_cache_append(k, v, i32(bounds), i32([0, 0, 0]), table, kc, vc)
    keys = [(torch.cat([kp, k[a:b]]), torch.cat([vp, v[a:b]])) for a, b in zip(bounds, bounds[1:])]
    lens, each = i32(own), i32(list(range(B + 1)))
    ws = fa.alloc_prefix_workspace(B, hq, hkv, d, 96, 64, "cuda")
    for _ in range(steps):
        q, k, v = mk(B, hq), mk(B, hkv), mk(B, hkv)
        fa.fa_cache_append(k, v, each, lens, table, kc, vc)
        lens = lens + 1
        keys = [(torch.cat([a, k[i:i + 1]]), torch.cat([b, v[i:i + 1]]))
                for i, (a, b) in enumerate(keys)]
        O, L = fa.fa_prefix_decode(q, kc, vc, ppages, i32([prefix]), table, lens, workspace=ws)
        want = _reference(q, keys, hkv)
        assert_close("O", O, want["O"])
        assert_close("L", L, want["L"])
