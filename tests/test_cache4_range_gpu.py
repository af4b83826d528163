"""Decode over the cache in 4 bits at the ends of its number ranges, against 64-bit values with
the bounds of its arithmetic (tests/cache4_ref.py)."""
import math
import os
import subprocess
import sys

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests import cache4_ref, rope_ref as ref
from tests.test_cache4_gpu import _decode_inputs
from tests.test_rope_gpu import _near

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def _check(q, cache, table, lens, codes, pairs, place, scale=None, **kw):
    """Decodes with the cache's pairs replaced by `pairs`, and compares."""
    d, hkv = q.shape[2], cache.shape[1]
    g = q.shape[1] // hkv
    q = q.cuda()
    O, L = fa.fa_cache4_decode(q, ref.pack(codes, pairs, d, cache).cuda(), table, lens, scale, **kw)
    s = 1 / math.sqrt(d) if scale is None else scale
    for b, (pg, r) in enumerate(place):
        for h in range(hkv if len(pg) else 0):
            rows = slice(h * g, (h + 1) * g)
            o, l = cache4_ref.decode_bounds(q[b, rows].double().cpu(), codes[:, pg, h, r],
                                            pairs[:, pg, h, r], s)
            _near("O", O[b, rows].cpu(), *o)
            _near("L", L[b, rows].cpu(), *l)
    return O, L


def _scaled(pairs, which, by):
    """Both numbers of the pairs of K (0) or V (1) times `by`, in bf16 again."""
    p = pairs.clone()
    p[which] *= by
    return p.to(torch.bfloat16).double()


def _growing(args, rises, reverse=False):
    """Scores of each request that grow along its keys by `rises` in all."""
    q, cache, table, lens, codes, pairs, place = args
    q, p = torch.ones_like(q), pairs.clone()
    for pg, r in place:
        n = len(pg)
        if n == 0:
            continue
        ramp = torch.linspace(0.0, rises, n, dtype=torch.float64)
        if reverse:
            ramp = ramp.flip(0)
        p[0, pg, :, r, :, 0] = 2.0 ** -6
        p[0, pg, :, r, :, 1] = (ramp / math.sqrt(q.shape[2]))[:, None, None]
    return q, cache, table, lens, codes, p.to(torch.bfloat16).double(), place


@pytest.mark.parametrize("exponent", [-60, -86, -90, -100, -110, -118])
@pytest.mark.parametrize("lens,hq,hkv,d,reverse", [
    ([1000], 4, 1, 64, False), ([1000], 4, 1, 64, True), ([300, 40], 8, 2, 128, False),
    ([90], 16, 1, 72, False), ([70] * 330, 1, 1, 64, False),
    ([70] * 500, 1, 1, 64, False)])
def test_small_values_and_growing_scores(exponent, lens, hq, hkv, d, reverse):
    """What earlier keys added shrinks with each reference that later scores set, whatever the
    values' size."""
    args = _growing(_decode_inputs(lens, hq, hkv, d, 16, 90 + d), 200.0, reverse)
    q, cache, table, lens, codes, pairs, place = args
    _check(q, cache, table, lens, codes, _scaled(pairs, 1, 2.0 ** exponent), place)


@pytest.mark.parametrize("apart", [12, 18, 24, 40, 100])
@pytest.mark.parametrize("large", [0, 1])
@pytest.mark.parametrize("lens,hq,hkv,d", [([200, 33], 4, 1, 128), ([500], 16, 1, 72),
                                           ([40] * 330, 2, 1, 128), ([3000], 8, 2, 104)])
def test_groups_of_values_far_apart(apart, large, lens, hq, hkv, d):
    """Each group of 64 channels keeps its bits beside one whose values are 2^apart times as
    large."""
    q, cache, table, lens, codes, pairs, place = _decode_inputs(lens, hq, hkv, d, 16, 91 + d)
    p = pairs.clone()
    p[1, ..., large, :] *= 2.0 ** (apart - apart // 2)
    p[1, ..., 1 - large, :] *= 2.0 ** -(apart // 2)
    _check(q, cache, table, lens, codes, p.to(torch.bfloat16).double(), place)


@pytest.mark.parametrize("size", [100, 112, 115, 124])
@pytest.mark.parametrize("small", ["scale", "keys"])
@pytest.mark.parametrize("hq,d", [(4, 64), (4, 128), (16, 128)])
def test_large_queries_of_ordinary_scores(size, small, hq, d):
    """Queries of 2^size whose scores are small by the scale or by the keys, beside ordinary
    ones."""
    q, cache, table, lens, codes, pairs, place = _decode_inputs([300, 17], hq, 1, d, 16, 92 + d)
    q[:, 1::2] = q[:, 1::2].clamp(-4, 4).mul(2.0 ** min(size, 100)).mul(2.0 ** (size - min(size, 100)))
    if small == "scale":
        _check(q, cache, table, lens, codes, pairs, place, scale=2.0 ** -size / math.sqrt(d))
    else:
        _check(q, cache, table, lens, codes, _scaled(pairs, 0, 2.0 ** -size), place)


@pytest.mark.parametrize("size", [100, 116, 121, 125])
@pytest.mark.parametrize("hq,d", [(4, 64), (16, 128)])
def test_small_queries_of_ordinary_scores(size, hq, d):
    """Queries of 2^-size whose scores are ordinary by the keys."""
    q, cache, table, lens, codes, pairs, place = _decode_inputs([300, 17], hq, 1, d, 16, 98 + d)
    by = min(size, 120)
    q = (q.double() * 2.0 ** -size).to(torch.bfloat16)
    _check(q, cache, table, lens, codes, _scaled(pairs, 0, 2.0 ** by), place,
           scale=2.0 ** (size - by + 1) / math.sqrt(d))


@pytest.mark.parametrize("size", [10, 20, 27, 31, 33, 40, 80, 100, 112])
@pytest.mark.parametrize("lens", [[300], [2000, 5], [40] * 330, [40] * 500])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(size, lens, sign):
    """Scores of 2^size: all alike (O is the mean of V), then one key above the rest by a part
    in 32 (O is its value)."""
    d = 64
    q, cache, table, n, codes, pairs, place = _decode_inputs(lens, 4, 1, d, 16, 93)
    q = torch.full_like(q, sign * 2.0 ** (size // 2) * 1.375)
    codes = codes.clone()
    codes[0] = 0
    p = pairs.clone()
    p[0, ..., 0] = 1.0
    p[0, ..., 1] = 2.0 ** (size - size // 2 - 3) * 1.2109375
    score = sign * 2.0 ** size * 1.375 * 1.2109375  # 64 / sqrt(64) / 8 = 1
    O, L = fa.fa_cache4_decode(q, ref.pack(codes, p, d, cache).cuda(), table, n)
    for b, (pg, r) in enumerate(place):
        one = ref.values(codes[1, pg, 0, r], p[1, pg, 0, r])
        s, m = cache4_ref.wide(p[1, pg, 0, r], d)
        # as in decode_bounds, with equal weights
        e = (cache4_ref.H + 2.0 ** -16) * (s * codes[1, pg, 0, r]).mean(0)
        e = e + (len(pg) / 16 + 64) * 2.0 ** -22 * (s * codes[1, pg, 0, r] + m.abs()).mean(0)
        want = one.mean(0)
        # Where a unit may be cut, parts are joined by the fp32 logarithms of their sums, m c and
        # m c + lg2(sum) rounded to 2^-24 of themselves: weights are off by 2^-22 |L| relative to
        # each other, and O by that part, twice, of what the values differ by.
        if lens in ([2000, 5], [40] * 500):
            off = min(1.0, 2 * math.expm1(min(1.0, 2.0 ** -22 * (abs(score) + 10))))
            e = e + off * (one.amax(0) - one.amin(0))
        _near("O", O[b].cpu(), want.expand(4, d), (ref.U * (want.abs() + e) + e).expand(4, d))
        L64 = torch.full((4,), score + math.log(len(pg)), dtype=torch.float64)
        _near("L", L[b].cpu(), L64, 2.0 ** -20 * (1 + L64.abs()))
    if size < 20:
        return  # a part in 32 would leave the others some weight
    for at in (0, 0.4, 1.0):
        p2 = p.clone()
        for pg, r in place:
            i = int(at * (len(pg) - 1))
            p2[0, pg[i], 0, r[i], :, 1] *= 1 + sign / 32
        p2 = p2.to(torch.bfloat16).double()
        O, L = fa.fa_cache4_decode(q, ref.pack(codes, p2, d, cache).cuda(), table, n)
        for b, (pg, r) in enumerate(place):
            i = int(at * (len(pg) - 1))
            want = ref.values(codes[1, pg[i], 0, r[i]], p2[1, pg[i], 0, r[i]])
            s, m = cache4_ref.wide(p2[1, pg[i], 0, r[i]], d)
            e = (cache4_ref.H + 2.0 ** -16) * (s * codes[1, pg[i], 0, r[i]] + m.abs())
            _near("O", O[b].cpu(), want.expand(4, d), (ref.U * (want.abs() + e) + e).expand(4, d))
            L64 = score * float(p2[0, pg[i], 0, r[i], 0, 1] / p[0, pg[i], 0, r[i], 0, 1])
            _near("L", L[b].cpu(), torch.full((4,), L64, dtype=torch.float64),
                  torch.full((4,), 2.0 ** -20 * (1 + abs(L64)), dtype=torch.float64))


@pytest.mark.parametrize("d,B", [(128, 3039), (128, 3040), (128, 3071), (128, 3100), (64, 7647),
                                 (64, 7648), (64, 7679), (64, 7700)])
def test_batches_at_the_end_of_the_default_shared_memory(d, B):
    """In a process of its own: a larger batch before it would raise the kernel's limit."""
    code = f"""
import torch
import exact_io_aware_27_gb300 as fa
cache = fa.alloc_cache4(2, 1, 16, {d}, "cuda")
x = torch.randn(20, 1, {d}, device="cuda", dtype=torch.bfloat16)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
fa.fa_cache4_append(None, x, x, i32([0, 20]), i32([0]), i32([[0, 1]]), cache)
table = i32([[0, 1]]).repeat({B}, 1)
q = torch.randn(1, 2, {d}, device="cuda", dtype=torch.bfloat16)
lens = torch.arange({B}, device="cuda", dtype=torch.int32) % 21
O, L = fa.fa_cache4_decode(q.repeat({B}, 1, 1), cache, table, lens)
for n in range(21):
    o, l = fa.fa_cache4_decode(q, cache, table[:1], i32([n]))
    # two orders of the same sums
    assert ((O[n::21].float() - o.float()).abs() <= 2.0 ** -6 * o.float().abs() + 2.0 ** -9).all()
    assert ((L[n::21] - l).abs() <= 1e-4).all() or n == 0
assert fa.fa_get_device_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("exponent", [60, 90, 100])
@pytest.mark.parametrize("reverse", [False, True])
def test_large_values(exponent, reverse):
    """The largest values that the sums have room for."""
    args = _growing(_decode_inputs([300, 40], 8, 2, 128, 16, 94), 60.0, reverse)
    q, cache, table, lens, codes, pairs, place = args
    _check(q, cache, table, lens, codes, _scaled(pairs, 1, 2.0 ** exponent), place)


@pytest.mark.parametrize("lens,hq,hkv,d,page", [
    ([1], 1, 1, 8, 16), ([2, 3, 0, 20], 4, 1, 64, 16), ([129], 7, 1, 72, 64), ([5000], 32, 8, 128, 64),
    ([1, 9000], 3, 3, 40, 1024), ([40000], 16, 2, 128, 32), ([300, 5], 20, 1, 96, 16),
    ([6000] + [(11 * i) % 40 for i in range(330)], 1, 1, 128, 16),
    ([700] * 330, 2, 1, 64, 16), ([2000, 0, 900], 128, 1, 64, 16)])
def test_every_key_counts(lens, hq, hkv, d, page):
    """Values for which each part of the keys, and each weight, moves O by many bounds."""
    q, cache, table, n, codes, pairs, place = _decode_inputs(lens, hq, hkv, d, page, sum(lens) + d)
    q, pairs = cache4_ref.telling(q, codes, pairs, place, 95)
    _check(q, cache, table, n, codes, pairs, place)


@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([300, 40], 8, 2, 128), ([5000, 1, 700], 16, 2, 128), ([700, 0, 33] * 170, 4, 1, 64),
    ([6000] + [40] * 400, 3, 1, 128)])
def test_the_same_bits_each_time(lens, hq, hkv, d):
    """One launch, pieces by blocks and by warps, and rows joined by blocks."""
    q, cache, table, n, *_ = _decode_inputs(lens, hq, hkv, d, 16, 97)
    O, L = fa.fa_cache4_decode(q, cache, table, n)
    for _ in range(5):
        o, l = fa.fa_cache4_decode(q, cache, table, n)
        assert torch.equal(o, O) and torch.equal(l, L)
