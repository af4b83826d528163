"""The paged cache in 4 bits: append, read and decode attention, against 64-bit values with
elementwise bounds (tests/rope_ref.py)."""
import math

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests import rope_ref as ref
from tests.test_rope_gpu import CASES, _bf16, _inputs, _near, _requests, _rows_of
from tests.packed_ref import attention64

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append and read
@pytest.mark.parametrize("lens,starts,hq,hkv,d,rot,inter,page,rest", CASES)
def test_append_and_read(lens, starts, hq, hkv, d, rot, inter, page, rest):
    total, n = sum(lens) + rest, sum(lens)
    q, k, _, table, wq, wk, _, _ = _inputs(total, hq, hkv, d, rot, 50 + d)
    v = _bf16(torch.Generator().manual_seed(51), total, hkv, d)
    cu, st, bt, pages = _requests(lens, starts, page, 52)
    cache = fa.alloc_cache4(pages, hkv, page, d, "cuda")
    cache.copy_(torch.randint(0, 256, cache.shape, generator=torch.Generator().manual_seed(53)))
    before = cache.clone()
    Qo = fa.fa_cache4_append(q, k, v, cu, st, bt, cache, table, wq, wk, EPS, inter)
    req, pos = _rows_of(lens, starts)
    y, e = ref.norm_rope64(q[:n], wq, table, pos, EPS, inter)
    _near("Qo", Qo[:n], y, ref.rounded(y, e))
    assert not bool(Qo[n:].any())

    codes, pairs = ref.unpack(cache, d)
    pg, r = bt[req, pos // page].long().cpu(), (pos % page).cpu()
    # V's values are bf16, so that the definition gives every bit
    want_c, want_p = ref.quantize(v[:n].cpu())
    assert torch.equal(pairs[1, pg, :, r], want_p)
    assert torch.equal(codes[1, pg, :, r], want_c)
    # K's come from the norm and the rotation
    y, e = (x.cpu() for x in ref.norm_rope64(k[:n], wk, table, pos, EPS, inter))
    got, two = ref.values(codes[0], pairs[0])[pg, :, r], pairs[0, pg, :, r]
    G = ref.groups(d)
    for j in range(G):
        g, ge = y[..., 64 * j:64 * j + 64], e[..., 64 * j:64 * j + 64].amax(-1)
        scale, lo = two[..., j, 0], two[..., j, 1]
        assert ((lo - g.amin(-1)).abs() <= ref.U * lo.abs() + 2 * ge).all()
        span = (g.amax(-1) - lo).clamp(min=0) / 15
        assert ((scale - span).abs() <= ref.U * span + 2 * ge).all()
        room = torch.maximum(torch.maximum(scale / 2, ref.U * g.abs().amax(-1)),
                             15 * ref.U * scale) + 4 * ge
        assert ((got[..., 64 * j:64 * j + 64] - g).abs() <= room[..., None]).all()

    # nothing else is touched: put the old rows' bits back
    old_c, old_p = ref.unpack(before, d)
    codes[:, pg, :, r], pairs[:, pg, :, r] = old_c[:, pg, :, r], old_p[:, pg, :, r]
    raw = lambda c, p: ref.pack(c, torch.nan_to_num(p, 1.5, 2.5, 3.5), d, before)  # noqa: E731
    assert torch.equal(raw(codes, pairs), raw(old_c, old_p))

    # rows back
    held = ref.unpack(cache, d)
    K, V = fa.fa_cache4_read(cache, cu, st, bt, total, d)
    for kv, got in ((0, K), (1, V)):
        want = ref.values(held[0][kv], held[1][kv])[pg, :, r].cuda()
        _near("KV"[kv], got[:n], want, ref.U * want.abs() + 2 * ref.E * 16 * want.abs().amax())
        assert not bool(got[n:].any())
    K2, V2 = torch.full_like(K, 5.0), torch.full_like(V, 5.0)
    fa.fa_cache4_read(cache, cu, st, bt, total, d, K=K2, V=V2)
    assert torch.equal(K2[:n], K[:n]) and torch.equal(V2[:n], V[:n])
    assert bool((K2[n:] == 5.0).all()) and bool((V2[n:] == 5.0).all())


def test_values_that_are_hard_to_hold():
    """Constant groups, tiny and huge ranges, ties, an offset far above the range, infinities
    and NaN."""
    d, page = 128, 16
    x = torch.randn(12, 1, d, generator=torch.Generator().manual_seed(60))
    x[0] = 0.0
    x[1] = -3.25
    x[2] *= 1e-38
    x[3] *= 1e37
    x[4] = torch.arange(d).remainder(31).float()[None] / 2    # halves of the scale 1: ties
    x[5] = 1000 + x[5]
    x[6, 0, 3] = math.inf
    x[7, 0, 100] = math.nan
    x[8, 0, 70] = -math.inf
    x[9] = 3e38 * torch.sign(x[9])
    x[10, 0, :64] = -0.0
    v = x.to(torch.bfloat16).cuda()
    cache = fa.alloc_cache4(1, 1, page, d, "cuda")
    args = (_i32([0, 12]), _i32([2]), _i32([[0]]))
    fa.fa_cache4_append(None, v, v, *args, cache)
    codes, pairs = ref.unpack(cache, d)
    want_c, want_p = ref.quantize(v.cpu())
    broken = {(6, 0), (7, 1), (8, 1), (9, 0), (9, 1)}
    for t in range(12):
        for j in range(2):
            for kv in (0, 1):
                two = pairs[kv, 0, 0, 2 + t, j]
                if (t, j) in broken:
                    assert two.isnan().all(), (t, j, two)
                    continue
                cols = slice(64 * j, 64 * j + 64)
                assert torch.equal(two, want_p[t, 0, j]), (t, j, two, want_p[t, 0, j])
                assert torch.equal(codes[kv, 0, 0, 2 + t, cols], want_c[t, 0, cols]), (t, j)
    K, V = fa.fa_cache4_read(cache, *args, 12, d)
    for got in (K, V):
        nan = got.isnan().reshape(12, 2, 64)
        for t in range(12):
            for j in range(2):
                assert bool(nan[t, j].all()) == bool(nan[t, j].any()) == ((t, j) in broken)


def test_read_reports_bad_places_and_leaves_or_clears_the_rows():
    d, page = 64, 16
    q, k, _, _, _, _, _, _ = _inputs(9, 2, 2, d, d, 61)
    cu, st, bt, pages = _requests([3, 3, 3], [0, 20, 4], page, 62)
    cache = fa.alloc_cache4(pages, 2, page, d, "cuda")
    fa.fa_cache4_append(None, k, k, cu, st, bt, cache)
    K, _ = fa.fa_cache4_read(cache, cu, st, bt, 9, d)
    assert bool(K.any(-1).all())
    for bad in ("page", "start", "bounds"):
        t, s, c = bt.clone(), st.clone(), cu.clone()
        if bad == "page":
            t[1, 1] = pages
        elif bad == "start":
            s[1] = 31
        else:
            c[1] = 8
        K2, V2 = fa.fa_cache4_read(cache, c, s, t, 9, d)
        assert fa.fa_get_device_status() == -8
        assert torch.isfinite(K2).all() and torch.isfinite(V2).all()
        if bad == "page":
            assert not bool(K2[3:6].any()) and torch.equal(K2[:3], K[:3])
            assert torch.equal(K2[6:], K[6:])
        K3 = torch.full_like(K, 5.0)
        fa.fa_cache4_read(cache, c, s, t, 9, d, K=K3, V=torch.empty_like(K))
        assert fa.fa_get_device_status() == -8
        if bad == "page":
            assert bool((K3[3:6] == 5.0).all())


# ------------------------------------------------------------------ decode
def _decode_inputs(lens, hq, hkv, d, page, seed, std=1.0):
    """Q, cache (bits that no request has are ones: NaN), table, lens and each row's place."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need))), -7, dtype=torch.int32)
    codes = torch.randint(0, 16, (2, pages, hkv, page, d), generator=g)
    scale = 0.05 + 0.3 * torch.rand(2, pages, hkv, page, ref.groups(d), generator=g)
    lo = -7.5 * scale + 0.2 * torch.randn(scale.shape, generator=g)
    pairs = torch.stack([scale, lo], -1).to(torch.bfloat16).double()
    place = []
    ours = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        mine = [order.pop() for _ in range(need[b])]
        table[b, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
        p = torch.arange(n)
        pg = torch.tensor(mine, dtype=torch.long)[p // page] if n else p
        ours[pg, p % page] = True
        place.append((pg, p % page))
    hidden = ~ours[None, :, None, :]
    codes = torch.where(hidden[..., None], 15, codes)
    pairs = torch.where(hidden[..., None, None], math.nan, pairs)
    like = torch.full((pages, hkv, page // 16, 1152 * ref.groups(d)), 255, dtype=torch.uint8)
    cache = ref.pack(codes, pairs, d, like)
    q = (torch.randn(len(lens), hq, d, generator=g) * std).to(torch.bfloat16).cuda()
    return q, cache.cuda(), table.cuda(), _i32(lens), codes, pairs, place


def _check_decode(q, cache, table, lens, codes, pairs, place, scale=None, O=None, L=None, **kw):
    d, hkv = q.shape[2], cache.shape[1]
    g = q.shape[1] // hkv
    if O is None:
        O, L = fa.fa_cache4_decode(q, cache, table, lens, scale, **kw)
    s = 1 / math.sqrt(d) if scale is None else scale
    for b, (pg, r) in enumerate(place):
        if len(pg) == 0:
            assert not bool(O[b].any()) and bool((L[b] == -math.inf).all())
            continue
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            o, l = ref.decode64(q[b, rows].double().cpu(), codes[:, pg, h, r], pairs[:, pg, h, r], s)
            _near("O", O[b, rows].cpu(), *o)
            _near("L", L[b, rows].cpu(), *l)
    return O, L


@pytest.mark.parametrize("lens,hq,hkv,d,page", [
    ([1], 1, 1, 8, 16), ([1, 0, 2], 2, 1, 64, 16), ([0], 4, 2, 128, 16), ([0, 0, 0], 4, 4, 64, 32),
    ([15, 16, 17, 1, 31, 32, 33], 8, 2, 64, 16), ([63, 64, 65, 127, 128, 129], 4, 1, 128, 32),
    ([300, 5], 7, 1, 72, 64), ([200, 70, 0, 1000], 8, 1, 96, 128), ([500, 3], 18, 2, 64, 16),
    ([130, 64], 16, 1, 128, 16), ([77, 400], 20, 1, 128, 64), ([90], 128, 1, 64, 16),
    ([257, 0, 31], 40, 2, 120, 16), ([70, 33], 24, 1, 128, 16), ([200], 32, 1, 64, 16),
    ([150, 20], 48, 1, 128, 16), ([5000], 32, 8, 128, 64), ([1, 9000], 3, 3, 40, 1024),
    ([i % 37 for i in range(300)], 4, 2, 64, 16), ([40000], 16, 2, 128, 32)])
@pytest.mark.parametrize("capacity", ["as needed", "wide"])
def test_decode(lens, hq, hkv, d, page, capacity):
    """Short tables take a block for each key/value head and request, others even pieces."""
    args = _decode_inputs(lens, hq, hkv, d, page, sum(lens) + d)
    if capacity == "wide":
        more = torch.full((len(lens), 4096 // page), -9, dtype=torch.int32, device="cuda")
        args = (*args[:2], torch.cat([args[2], more], 1), *args[3:])
    _check_decode(*args)


@pytest.mark.parametrize("others,hq,hkv,d", [(330, 1, 1, 128), (330, 7, 1, 64), (45, 16, 8, 128),
                                             (100, 64, 4, 72), (41, 32, 8, 64)])
@pytest.mark.parametrize("long", [0, 20])
def test_decode_one_long_request_among_many(others, hq, hkv, d, long):
    """More than 320 units: single warps take even pieces of them, and the long request's rows are
    joined from well over 32 pieces each."""
    lens = [(11 * i) % 40 for i in range(others)]
    lens.insert(long, 6000)
    _check_decode(*_decode_inputs(lens, hq, hkv, d, 16, others + hq + d))


@pytest.mark.parametrize("std,scale", [(4.0, None), (0.0, None), (1.0, 1e-6), (1.0, 3.0),
                                       (1e-20, None)])
def test_decode_scores(std, scale):
    """Peaked, uniform and all but constant weights."""
    _check_decode(*_decode_inputs([333, 64, 2000], 8, 2, 128, 16, 71, std=std), scale=scale)


@pytest.mark.parametrize("scale", [1e-18, 1e-25, 1e-38])
@pytest.mark.parametrize("others", [0, 330])
def test_decode_scales_that_leave_nothing_of_a_score(scale, others):
    """All weights alike, also of queries that are zero, and pieces and warps without a key."""
    q, cache, table, lens, codes, pairs, place = _decode_inputs(
        [2000, 33, 130] + [7] * others, 4, 1, 64, 16, 85)
    q[:, 1] = 0
    q[:, 2] *= 1e-30
    _check_decode(q, cache, table, lens, codes, pairs, place, scale=scale)


def test_decode_growing_scores():
    """The reference maximum moves many times in both directions of the keys."""
    q, cache, table, lens, codes, pairs, place = _decode_inputs([1000], 4, 1, 64, 16, 72)
    pg, r = place[0]
    for reverse in (False, True):
        ramp = torch.linspace(0.01, 4.0, 1000, dtype=torch.float64)
        if reverse:
            ramp = ramp.flip(0)
        p = pairs.clone()
        p[0, pg, 0, r, 0, 0] = ramp
        p[0, pg, 0, r, 0, 1] = -7.5 * ramp
        p = p.to(torch.bfloat16).double()
        c = ref.pack(codes, p, 64, cache).cuda()
        _check_decode(q, c, table, lens, codes, p, place)


@pytest.mark.parametrize("at", [0, 77, 199])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_a_large_value_of_small_weight(at, d):
    """The other keys' values keep their bits beside a value 2^20 times as large whose weight is
    e^-40, and so do values that grow, or shrink, by 2^40 along the keys."""
    q, cache, table, lens, codes, pairs, place = _decode_inputs([200], 4, 1, d, 16, 84)
    q.fill_(0.5)
    pg, r = place[0]
    p = pairs.clone()
    p[0, pg[at], 0, r[at], :, 0] = 0.0
    p[0, pg[at], 0, r[at], :, 1] = -10.0 * math.sqrt(64 / d)
    p[1, pg[at], 0, r[at]] *= 2.0 ** 20
    _check_decode(q, ref.pack(codes, p, d, cache).cuda(), table, lens, codes, p, place)
    for sign in (1, -1):
        p = pairs.clone()
        p[1, pg, 0, r] *= (2.0 ** (sign * torch.linspace(-20, 20, 200, dtype=torch.float64)))[
            :, None, None]
        p = p.to(torch.bfloat16).double()
        _check_decode(q, ref.pack(codes, p, d, cache).cuda(), table, lens, codes, p, place)


def test_decode_a_key_that_is_not_a_number_reaches_its_head_only():
    q, cache, table, lens, codes, pairs, place = _decode_inputs([100, 100], 8, 2, 128, 16, 73)
    want = fa.fa_cache4_decode(q, cache, table, lens)
    pairs[0, place[1][0][37], 1, place[1][1][37], 0, 0] = math.nan
    O, L = fa.fa_cache4_decode(q, ref.pack(codes, pairs, 128, cache).cuda(), table, lens)
    assert bool(O[1, 4:].isnan().all()) and bool(L[1, 4:].isnan().all())
    O[1, 4:], L[1, 4:] = want[0][1, 4:], want[1][1, 4:]
    assert torch.equal(O, want[0]) and torch.equal(L, want[1])


def test_decode_queries_that_are_not_finite_stay_in_their_row():
    q, cache, table, lens, *_ = _decode_inputs([200, 70], 8, 2, 64, 16, 74)
    want = fa.fa_cache4_decode(q, cache, table, lens)
    q[0, 3, 5], q[1, 6, 0] = math.nan, math.inf
    O, L = fa.fa_cache4_decode(q, cache, table, lens)
    assert bool(O[0, 3].isnan().all()) and bool(O[1, 6].isnan().all())
    for b, h in ((0, 3), (1, 6)):
        O[b, h], L[b, h] = want[0][b, h], want[1][b, h]
    assert torch.equal(O, want[0]) and torch.equal(L, want[1])


def test_decode_does_not_depend_on_the_run_or_the_workspace():
    args = _decode_inputs([3000, 10, 700], 8, 2, 128, 16, 75)
    q, cache, table, lens = args[:4]
    O, L = fa.fa_cache4_decode(q, cache, table, lens)
    ws = fa.alloc_cache4_workspace(3, 8, 2, 128, table.shape[1] * 16, "cuda")
    for fill in (0, 255, 127):
        ws.fill_(fill)
        o, l = torch.full_like(O, 3.0), torch.full_like(L, 3.0)
        got = fa.fa_cache4_decode(q, cache, table, lens, O=o, L=l, workspace=ws)
        assert got[0].data_ptr() == o.data_ptr()
        assert torch.equal(o, O) and torch.equal(l, L)
    with pytest.raises(fa.FAError):
        fa.fa_cache4_decode(q, cache, table, lens, workspace=ws[:-256])


def test_decode_a_wide_table_and_more_capacity_than_keys():
    q, cache, table, lens, codes, pairs, place = _decode_inputs([100, 1, 257], 8, 2, 64, 16, 76)
    wide = torch.full((3, 20000), -9, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    _check_decode(q, cache, wide, lens, codes, pairs, place)


@pytest.mark.parametrize("B", [1, 40, 700])
def test_decode_without_any_page(B):
    cache = fa.alloc_cache4(1, 2, 16, 64, "cuda")
    q = torch.ones(B, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    O, L = fa.fa_cache4_decode(q, cache, table, _i32([0] * B))
    assert not bool(O.any()) and bool((L == -math.inf).all())
    O, L = fa.fa_cache4_decode(q, cache, table, _i32([0] * (B - 1) + [1]))
    assert fa.fa_get_device_status() == -8
    assert not bool(O.any()) and bool((L == -math.inf).all())


def test_decode_the_largest_batch():
    """8192 requests: the lengths' sums take shared memory of the blocks'."""
    lens = [(7 * i) % 50 for i in range(8192)]
    q, cache, table, n, codes, pairs, place = _decode_inputs(lens, 2, 1, 8, 16, 83)
    wide = torch.full((8192, 4096), -9, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    for t in (table, wide):
        O, L = fa.fa_cache4_decode(q, cache, t, n)
        for b in (0, 1, 2, 31, 32, 33, 4000, 4001, 8190, 8191):
            pick = slice(b, b + 1)
            _check_decode(q[pick], cache, t, n, codes, pairs, place[pick], O=O[pick], L=L[pick])
        near = O if t is table else near
    assert bool(((O.float() - near.float()).abs() <= 2 * ref.U * 4).all())


def test_decode_reports_bad_lengths_and_pages():
    q, cache, table, lens, *_ = _decode_inputs([40, 40], 4, 2, 64, 16, 77)
    want = fa.fa_cache4_decode(q, cache, table, lens)
    for bad in (-1, 49, 2 ** 31 - 1):
        n = lens.clone()
        n[0] = bad
        O, L = fa.fa_cache4_decode(q, cache, table, n)
        assert fa.fa_get_device_status() == -8
        assert torch.equal(O[1], want[0][1]) and torch.equal(L[1], want[1][1])
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad
        O, L = fa.fa_cache4_decode(q, cache, t, lens)
        assert fa.fa_get_device_status() == -8
        assert torch.equal(O[1], want[0][1]) and torch.equal(L[1], want[1][1])


def test_decode_in_graphs_that_share_a_workspace():
    """Lengths are read on the device, so that a replay follows them."""
    a = _decode_inputs([100, 0, 900], 8, 2, 128, 16, 78)
    b = _decode_inputs([5, 640, 33], 8, 2, 128, 16, 79)
    b = (b[0], b[1], torch.cat([b[2], torch.full((3, a[2].shape[1]), -1, dtype=torch.int32,
                                                 device="cuda")], 1)[:, :a[2].shape[1]].contiguous(),
         *b[3:])
    want = [fa.fa_cache4_decode(*x[:4]) for x in (a, b)]
    ws = fa.alloc_cache4_workspace(3, 8, 2, 128, a[2].shape[1] * 16, "cuda")
    graphs, got = [], []
    torch.cuda.synchronize()
    for x in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(fa.fa_cache4_decode(*x[:4], workspace=ws))
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    for w, o in zip(want, got):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
    a[3].copy_(_i32([64, 0, 7]))
    graphs[0].replay()
    place = [(pg[:n], r[:n]) for (pg, r), n in zip(a[6], (64, 0, 7))]
    _check_decode(*a[:6], place, O=got[0][0], L=got[0][1])


def test_decode_on_another_stream():
    args = _decode_inputs([3000, 10, 700], 8, 2, 64, 16, 80)
    want = fa.fa_cache4_decode(*args[:4])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    O, L = fa.fa_cache4_decode(*args[:4], stream=side)
    side.synchronize()
    assert torch.equal(O, want[0]) and torch.equal(L, want[1])


def test_far_into_a_large_cache():
    """Offsets beyond 2^32 bytes in append, read and decode."""
    pages, hkv, page, d = 3900, 8, 1024, 128  # 4.6 GB
    cache = torch.zeros(pages, hkv, page // 16, 2304, dtype=torch.uint8, device="cuda")
    q, k, _, _, _, _, _, _ = _inputs(40, 16, hkv, d, d, 81)
    table = _i32([[3899, 3700]])
    args = (_i32([0, 40]), _i32([1000]), table)
    fa.fa_cache4_append(None, k, k, *args, cache)
    K, V = fa.fa_cache4_read(cache, *args, 40, d)
    codes, pairs = ref.quantize(k.cpu())
    want = ref.values(codes, pairs).cuda()
    for got in (K, V):
        _near("KV", got, want, ref.U * want.abs() + 32 * ref.E * want.abs().amax())
    zero = (torch.zeros(2, 1040, hkv, d, dtype=torch.long),
            torch.zeros(2, 1040, hkv, 2, 2, dtype=torch.float64))
    zero[0][:, 1000:], zero[1][:, 1000:] = codes, pairs
    O, L = fa.fa_cache4_decode(q[:1], cache, table, _i32([1040]))
    for h in range(hkv):
        o, l = ref.decode64(q[0, 2 * h:2 * h + 2].double().cpu(), zero[0][:, :, h], zero[1][:, :, h],
                            1 / math.sqrt(d))
        _near("O", O[0, 2 * h:2 * h + 2].cpu(), *o)
        _near("L", L[0, 2 * h:2 * h + 2].cpu(), *l)
    cache[3899], cache[3700] = 0, 0
    assert not bool(cache.any())


def test_a_serving_run():
    """Prompts in two chunks, the second one attending to what the cache holds, then single
    tokens: each part against 64 bits on the values that the cache stands for."""
    hq, hkv, d, page = 8, 2, 128, 16
    chunks = ([30, 100, 1], [17, 0, 64], [1, 1, 1], [1, 1, 1])
    ends = [sum(c[i] for c in chunks) for i in range(3)]
    _, _, bt, pages = _requests(ends, [0, 0, 0], page, 82)
    cache = fa.alloc_cache4(pages, hkv, page, d, "cuda")
    cache.fill_(255)
    table = fa.rope_table(300, d)
    have = [0, 0, 0]
    for step, new in enumerate(chunks):
        total = sum(new)
        at = [0]
        for n in new:
            at.append(at[-1] + n)
        q, k, _, _, wq, wk, _, _ = _inputs(total, hq, hkv, d, d, 90 + step)
        Qo = fa.fa_cache4_append(q, k, k, _i32(at), _i32(have), bt, cache, table, wq, wk)
        have = [a + n for a, n in zip(have, new)]
        codes, pairs = ref.unpack(cache, d)
        if step < 2:
            ctx = [0]
            for n in have:
                ctx.append(ctx[-1] + n)
            K, V = fa.fa_cache4_read(cache, _i32(ctx), _i32([0] * 3), bt, ctx[-1], d)
            # queries of the whole context, the chunk's at its end
            wide = torch.zeros(ctx[-1], hq, d, dtype=torch.bfloat16, device="cuda")
            for i in range(3):
                wide[ctx[i + 1] - new[i]:ctx[i + 1]] = Qo[at[i]:at[i + 1]]
            plan = fa.fa_packed_plan(_i32(ctx), ctx[-1])
            O, _ = fa.fa_packed_forward(wide, K, V, plan)
            for i in range(3):
                rows = slice(ctx[i], ctx[i + 1])
                for h in range(hkv):
                    if have[i]:
                        r = attention64(wide[rows, 4 * h:4 * h + 4].double().transpose(0, 1),
                                        K[rows, h].double(), V[rows, h].double(), True,
                                        1 / math.sqrt(d))
                        _near("O", O[rows, 4 * h:4 * h + 4].transpose(0, 1), *r["O"])
        else:
            place = [(bt[b, torch.arange(n) // page].long().cpu(), torch.arange(n) % page)
                     for b, n in enumerate(have)]
            _check_decode(Qo, cache, bt, _i32(have), codes, pairs, place)
