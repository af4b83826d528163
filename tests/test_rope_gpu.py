"""Norms of queries and keys with the rotation, their gradients, and the append to the bf16
cache with them, against 64-bit values with elementwise bounds (tests/rope_ref.py)."""
import math

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests import rope_ref as ref
from tests.packed_ref import attention64

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def _bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def _inputs(total, hq, hkv, d, rot, seed, norm=True, std=1.0, positions=4000, sliced=True):
    """Q, K (slices of one projection), positions, table, weights, gradients."""
    g = torch.Generator().manual_seed(seed)
    proj = _bf16(g, total, hq + 2 * hkv, d, std=std)
    q, k = proj[:, :hq], proj[:, hq:hq + hkv]
    if not sliced:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, positions, (total,), generator=g).to(torch.int32).cuda()
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() if norm else None
         for _ in (0, 1)]
    table = fa.rope_table(positions, rot) if rot else None
    return q, k, pos, table, *w, _bf16(g, total, hq, d), _bf16(g, total, hkv, d)


def _near(name, got, want, bound):
    """Within the bound, or the same infinity, or both NaN."""
    got = got.double()
    good = ((got - want).abs() <= bound) | (got == want) | (got.isnan() & want.isnan())
    bad = ~good
    assert not bool(bad.any()), (name, int(bad.sum()), float((got - want).abs().max()))


def _check(q, k, pos, table, wq, wk, dq, dk, inter, eps=EPS):
    out = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk, eps, inter)
    back = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk, eps, inter)
    for i, (x, w, dy) in enumerate(((q, wq, dq), (k, wk, dk))):
        y, e = ref.norm_rope64(x, w, table, pos, eps, inter)
        _near("y%d" % i, out[i], y, ref.rounded(y, e))
        dx, bx, dw, bw = ref.norm_rope_backward64(dy, x, w, table, pos, eps, inter)
        _near("dx%d" % i, back[i], dx, bx)
        if w is None:
            assert back[2 + i] is None
        else:
            _near("dw%d" % i, back[2 + i], dw, bw)


@pytest.mark.parametrize("total,hq,hkv,d,rot,inter", [
    (1, 1, 1, 8, 8, False), (1, 1, 1, 8, 8, True), (2, 3, 1, 16, 8, False), (5, 2, 2, 24, 24, False),
    (7, 4, 1, 32, 16, True), (33, 6, 2, 40, 40, False), (33, 9, 3, 40, 24, True),
    (64, 8, 8, 56, 48, False), (100, 32, 8, 64, 64, False), (100, 17, 17, 64, 32, True),
    (50, 7, 1, 72, 72, False), (333, 6, 2, 96, 96, False), (333, 6, 2, 96, 40, True),
    (200, 5, 5, 120, 120, False), (257, 32, 8, 128, 128, False), (257, 9, 3, 128, 64, True),
    (3000, 32, 8, 128, 128, False), (20000, 3, 1, 64, 64, False)])
def test_against_64_bits(total, hq, hkv, d, rot, inter):
    _check(*_inputs(total, hq, hkv, d, rot, total + d), inter)


@pytest.mark.parametrize("what", ["no norm", "no rotation", "neither", "queries' norm only",
                                  "keys' norm only"])
@pytest.mark.parametrize("d", [40, 128])
def test_parts(what, d):
    q, k, pos, table, wq, wk, dq, dk = _inputs(90, 6, 2, d, d, 3)
    if what in ("no norm", "neither"):
        wq = wk = None
    if what in ("no rotation", "neither"):
        table = pos = None
    if what == "queries' norm only":
        wk = None
    if what == "keys' norm only":
        wq = None
    _check(q, k, pos, table, wq, wk, dq, dk, False)


@pytest.mark.parametrize("std,eps", [(1e-3, 1e-6), (1e4, 1e-6), (1e-12, 1e-6), (0.0, 1e-6)])
def test_magnitudes(std, eps):
    """Large rows, rows that eps outweighs, and rows of zeros."""
    _check(*_inputs(40, 4, 2, 64, 64, 5, std=std), False, eps=eps)


def test_dense_inputs_and_far_positions():
    q, k, _, _, wq, wk, dq, dk = _inputs(70, 4, 2, 64, 64, 6, sliced=False)
    table = fa.rope_table(1 << 20, 64)
    pos = torch.arange(70, dtype=torch.int32, device="cuda") + ((1 << 20) - 70)
    _check(q, k, pos, table, wq, wk, dq, dk, False)


def test_in_place_and_slices_as_outputs():
    q, k, pos, table, wq, wk, dq, dk = _inputs(77, 8, 2, 64, 64, 7)
    want = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk)
    buf = torch.full((77, 12, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    Qo, Ko = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk, Qo=buf[:, :8], Ko=buf[:, 10:])
    assert Qo.data_ptr() == buf.data_ptr()
    assert torch.equal(buf[:, :8], want[0]) and torch.equal(buf[:, 10:], want[1])
    assert bool((buf[:, 8:10] == 9.0).all())
    grads = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk)
    got = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk, dQ=buf[:, :8],
                                      dK=buf[:, 8:10])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    fa.fa_qk_norm_rope(q, k, pos, table, wq, wk, Qo=q, Ko=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    with pytest.raises(fa.FAError):
        fa.fa_qk_norm_rope(q, k, pos, table, wq, wk, Qo=q, Ko=q[:, :2])


def test_gradients_do_not_depend_on_the_run():
    args = _inputs(5000, 12, 4, 128, 128, 8)
    q, k, pos, table, wq, wk, dq, dk = args
    first = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk)
    ws = fa.alloc_qk_norm_rope_workspace(12, 4, 128, "cuda")
    ws.fill_(255)
    for _ in range(3):
        again = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_a_bad_position_is_reported_and_its_row_left():
    for bad in (-1, 4000, 2 ** 31 - 1, -2 ** 31):
        q, k, pos, table, wq, wk, dq, dk = _inputs(20, 4, 2, 64, 64, 9)
        clean = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk)
        want = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk)
        pos[13] = bad
        Qo, Ko = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        fa.fa_qk_norm_rope(q, k, pos, table, wq, wk, Qo=Qo, Ko=Ko)
        assert fa.fa_get_device_status() == -8
        for got, w in ((Qo, want[0]), (Ko, want[1])):
            assert bool((got[13] == 7.0).all())
            assert torch.equal(got[:13], w[:13]) and torch.equal(got[14:], w[14:])
        dQ, dK = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk, dQ=dQ, dK=dK)
        assert fa.fa_get_device_status() == -8
        assert bool((dQ[13] == 7.0).all()) and torch.equal(dQ[:13], clean[0][:13])
        assert torch.equal(dK[14:], clean[1][14:])


def test_not_a_number_stays_in_its_row():
    q, k, pos, table, wq, wk, dq, dk = _inputs(30, 4, 2, 72, 40, 10)
    want = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk)
    q[11, 2, 5] = math.nan
    k[3, 1, 71] = math.inf
    got = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk)
    assert bool(got[0][11, 2].isnan().all())
    assert not bool(got[1][3, 1].isfinite().all())
    keep = torch.ones(30, 4, dtype=torch.bool)
    keep[11, 2] = False
    assert torch.equal(got[0][keep.cuda()], want[0][keep.cuda()])
    keep = torch.ones(30, 2, dtype=torch.bool)
    keep[3, 1] = False
    assert torch.equal(got[1][keep.cuda()], want[1][keep.cuda()])


def test_another_stream_and_a_graph():
    q, k, pos, table, wq, wk, dq, dk = _inputs(300, 8, 2, 128, 128, 11)
    want = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk)
    grads = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk, stream=side)
    back = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *back), (*want, *grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.fa_qk_norm_rope(q, k, pos, table, wq, wk)
        back = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk)
    q.copy_(torch.randn_like(q))
    pos.add_(5).clamp_(max=3999)
    graph.replay()
    want = (*fa.fa_qk_norm_rope(q, k, pos, table, wq, wk),
            *fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((*got, *back), want))


def test_autograd():
    q, k, pos, table, wq, wk, dq, dk = _inputs(120, 8, 2, 96, 96, 12)
    proj = torch.cat([q, k], 1).requires_grad_()
    wq, wk = wq.clone().requires_grad_(), wk.clone().requires_grad_()
    Qo, Ko = fa.qk_norm_rope(proj[:, :8], proj[:, 8:], pos, table, wq, wk)
    want = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq.detach(), wk.detach())
    torch.autograd.backward((Qo, Ko), (dq, dk))
    assert torch.equal(proj.grad, torch.cat(want[:2], 1))
    assert torch.equal(wq.grad, want[2].to(torch.bfloat16))
    assert torch.equal(wk.grad, want[3].to(torch.bfloat16))
    # an unused output, an expanded gradient, keys that need none
    proj.grad = None
    Qo, Ko = fa.qk_norm_rope(proj[:, :8], k, pos, table, wq, wk)
    Qo.sum().backward()
    want = fa.fa_qk_norm_rope_backward(torch.ones_like(dq), torch.zeros_like(dk), q, k, pos, table,
                                       wq.detach(), wk.detach())
    assert torch.equal(proj.grad[:, :8], want[0])
    # once only
    x = q.clone().requires_grad_()
    Qo, _ = fa.qk_norm_rope(x, k, pos, table, wq, wk)
    (gx,) = torch.autograd.grad(Qo.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.float().sum().backward()


def test_training_step_through_attention():
    """Projection, norm and rotation, packed attention: gradients of the projection and the
    weights against 64 bits. Queries and keys are rounded to bf16 between the two, which the
    reference does as well, so that each part's bounds apply to the part's own inputs."""
    lens, hq, hkv, d = [37, 0, 130, 3], 4, 2, 64
    total = sum(lens)
    q, k, _, _, wq, wk, do, _ = _inputs(total, hq, hkv, d, d, 13)
    g = torch.Generator().manual_seed(14)
    v = _bf16(g, total, hkv, d)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    table = fa.rope_table(200, d)
    cu = torch.tensor([0, 37, 37, 167, 170], dtype=torch.int32, device="cuda")
    plan = fa.fa_packed_plan(cu, total)
    leaves = [x.clone().contiguous().requires_grad_() for x in (q, k, v, wq, wk)]
    Qo, Ko = fa.qk_norm_rope(leaves[0], leaves[1], pos, table, leaves[3], leaves[4])
    Qo.retain_grad()
    Ko.retain_grad()
    O = fa.flash_attention_packed(Qo, Ko, leaves[2], plan)
    O.backward(do)
    at = 0
    for n in lens:
        for h in range(hkv):
            if n == 0:
                continue
            rows, hs = slice(at, at + n), slice(2 * h, 2 * h + 2)
            r = attention64(Qo[rows, hs].double().transpose(0, 1), Ko[rows, h].double(),
                            v[rows, h].double(), True, 1 / math.sqrt(d),
                            do[rows, hs].double().transpose(0, 1))
            _near("O", O[rows, hs].transpose(0, 1), *r["O"])
            _near("dQ", Qo.grad[rows, hs].transpose(0, 1), *r["dQ"])
            _near("dK", Ko.grad[rows, h], *r["dK"])
            _near("dV", leaves[2].grad[rows, h], *r["dV"])
        at += n
    for x, w, y in ((0, 3, Qo), (1, 4, Ko)):
        dx, bx, dw, bw = ref.norm_rope_backward64(y.grad, leaves[x].detach(), leaves[w].detach(),
                                                  table, pos, 1e-6, False)
        _near("dx", leaves[x].grad, dx, bx)
        _near("dw", leaves[w].grad, dw, bw + ref.U * (dw.abs() + bw))


# ------------------------------------------------------------------ append
def _requests(lens, starts, page, seed, rest=0, spare=2):
    """cu, starts, table over shuffled pages (unused entries are -7), pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(a + n) // page) for a, n in zip(starts, lens)]
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need))), -7, dtype=torch.int32)
    for i, n in enumerate(need):
        for j in range(n):
            table[i, j] = order.pop()
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(at), i32(starts), table.cuda(), sum(need) + spare


def _rows_of(lens, starts):
    req = [i for i, n in enumerate(lens) for _ in range(n)]
    pos = [a + j for a, n in zip(starts, lens) for j in range(n)]
    return (torch.tensor(req, device="cuda", dtype=torch.long),
            torch.tensor(pos, device="cuda", dtype=torch.long))


CASES = [  # lens, starts, hq, hkv, d, rot, interleaved, page, rest
    ([1], [0], 1, 1, 8, 8, False, 16, 0),
    ([1, 1, 1], [15, 16, 17], 4, 1, 64, 64, False, 16, 0),
    ([0, 5, 0, 0, 17, 3, 0], [3, 0, 9, 1, 30, 14, 2], 6, 2, 40, 24, True, 16, 4),
    ([1] * 70, list(range(70)), 8, 2, 64, 64, False, 16, 0),
    ([1] * 1100, [i % 50 for i in range(1100)], 2, 1, 32, 32, False, 16, 0),
    ([33, 128, 250], [7, 0, 100], 32, 8, 128, 128, False, 64, 1),
    ([100], [1000], 9, 3, 96, 96, False, 1024, 0),
    ([13, 29], [3, 50], 5, 5, 120, 56, True, 32, 0),
]


@pytest.mark.parametrize("lens,starts,hq,hkv,d,rot,inter,page,rest", CASES)
def test_append(lens, starts, hq, hkv, d, rot, inter, page, rest):
    total = sum(lens) + rest
    q, k, _, table, wq, wk, _, _ = _inputs(total, hq, hkv, d, rot, 20 + d)
    g = torch.Generator().manual_seed(21)
    v = _bf16(g, total, hkv, d)
    cu, st, bt, pages = _requests(lens, starts, page, 22)
    kc, vc = _bf16(g, pages, hkv, page, d), _bf16(g, pages, hkv, page, d)
    before = kc.clone(), vc.clone()
    Qo = fa.fa_rope_append(q, k, v, cu, st, bt, kc, vc, table, wq, wk, EPS, inter)
    req, pos = _rows_of(lens, starts)
    n = sum(lens)
    y, e = ref.norm_rope64(q[:n], wq, table, pos, EPS, inter)
    _near("Qo", Qo[:n], y, ref.rounded(y, e))
    assert not bool(Qo[n:].any())
    y, e = ref.norm_rope64(k[:n], wk, table, pos, EPS, inter)
    pg, r = bt[req, pos // page].long(), pos % page
    _near("K", kc[pg, :, r], y, ref.rounded(y, e))
    assert torch.equal(vc[pg, :, r], v[:n])
    kc[pg, :, r] = before[0][pg, :, r]
    vc[pg, :, r] = before[1][pg, :, r]
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])  # nothing else is touched
    # without norm and rotation it is fa_cache_append
    a, b = [x.clone() for x in before], [x.clone() for x in before]
    assert fa.fa_rope_append(None, k, v, cu, st, bt, *a) is None
    fa.fa_cache_append(k, v, cu, st, bt, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_append_gives_what_the_separate_calls_give():
    lens, starts, page = [20, 1, 44], [0, 63, 5], 16
    q, k, _, table, wq, wk, _, _ = _inputs(65, 8, 2, 128, 128, 23)
    cu, st, bt, pages = _requests(lens, starts, page, 24)
    _, pos = _rows_of(lens, starts)
    caches = [torch.zeros(pages, 2, page, 128, dtype=torch.bfloat16, device="cuda")
              for _ in range(4)]
    Qo = fa.fa_rope_append(q, k, k, cu, st, bt, *caches[:2], table, wq, wk)
    Qs, Ks = fa.fa_qk_norm_rope(q, k, pos.to(torch.int32), table, wq, wk)
    fa.fa_cache_append(Ks, k, cu, st, bt, *caches[2:])
    assert torch.equal(Qo, Qs)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("bounds", [[0, 5, 3, 10], [1, 5, 10], [0, 5, 11], [0, -2, 10],
                                    [0, 2 ** 31 - 1, 10], [0, 10, 4]])
@pytest.mark.parametrize("four", [False, True])
def test_append_reports_bad_bounds(bounds, four):
    q, k, _, table, wq, wk, _, _ = _inputs(10, 2, 2, 64, 64, 25)
    n = len(bounds) - 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (q, k, k, i32(bounds), i32([0] * n), i32([[i] for i in range(n)]))
    if four:
        cache = fa.alloc_cache4(n, 2, 16, 64, "cuda")
        fa.fa_cache4_append(*args, cache, table, wq, wk)
        held, pairs = ref.unpack(cache, 64)
        rows = pairs[1, :, 0, :, 0].abs().sum(-1) > 0  # scale and minimum of V
    else:
        kc = torch.zeros(n, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        fa.fa_rope_append(*args, kc, vc, table, wq, wk)
        rows = vc.float().abs().sum((1, 3)) > 0
        for i, r in rows.nonzero().tolist():  # a row goes only to a request that owns it
            t = bounds[i] + r
            assert 0 <= t < 10 and t < bounds[i + 1] and torch.equal(vc[i, :, r], k[t])
    assert fa.fa_get_device_status() == -8
    assert int(rows.sum()) <= 10


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("what", ["page", "negative page", "position", "start", "angles",
                                  "far start", "far start, nothing turned"])
def test_append_reports_bad_places(what, four):
    """The row concerned is not written, the others are."""
    total, page, d = 6, 16, 64
    q, k, _, table, wq, wk, _, _ = _inputs(total, 2, 2, d, d, 26)
    cu, st, bt, pages = _requests([2, 2, 2], [3, 14, 3], page, 27)
    ok = 4
    if what == "page":
        bt[1, 0] = pages
    elif what == "negative page":
        bt[1, 0] = -1
    elif what == "position":
        bt = bt[:, :1].contiguous()
        st[1] = 15
        ok = 5
    elif what == "start":
        st[1] = -1
    elif what == "angles":
        table = table[:15].contiguous()
        ok = 5
    else:
        st[1] = 2 ** 31 - 1
        if "nothing" in what:
            table = None
    if four:
        cache = fa.alloc_cache4(pages, 2, page, d, "cuda")
        Qo = fa.fa_cache4_append(q, k, k, cu, st, bt, cache, table, wq, wk)
        _, pairs = ref.unpack(cache, d)
        written = int((pairs[0].abs().sum((-1, -2)) > 0).sum()) // 2
    else:
        kc = torch.zeros(pages, 2, page, d, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        Qo = fa.fa_rope_append(q, k, k, cu, st, bt, kc, vc, table, wq, wk)
        written = int((kc.float().abs().sum((1, 3)) > 0).sum())
        assert written == int((vc.float().abs().sum((1, 3)) > 0).sum())
    assert fa.fa_get_device_status() == -8
    # (14, 15 of the second request lie in one page, so that a bad one loses both)
    assert written == ok, (what, written)
    assert torch.isfinite(Qo).all()


def test_a_decode_step_on_the_bf16_cache():
    """Prompts, then two single tokens a request: rotation on the way into the cache, and decode
    attention to it, against 64 bits on the rows that the cache holds."""
    lens, page, hq, hkv, d = [40, 1, 77], 16, 8, 2, 64
    cu, st, bt, pages = _requests([n + 2 for n in lens], [0, 0, 0], page, 28)
    kc = torch.full((pages, hkv, page, d), math.nan, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = fa.rope_table(200, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    have = [0, 0, 0]
    for step, new in enumerate((lens, [1] * 3, [1] * 3)):
        total = sum(new)
        q, k, _, _, wq, wk, _, _ = _inputs(total, hq, hkv, d, d, 30 + step)
        v = _bf16(torch.Generator().manual_seed(40 + step), total, hkv, d)
        at = [0]
        for n in new:
            at.append(at[-1] + n)
        Qo = fa.fa_rope_append(q, k, v, i32(at), i32(have), bt, kc, vc, table, wq, wk)
        have = [a + n for a, n in zip(have, new)]
    O, L = fa.fa_prefix_decode(Qo, kc, vc, None, None, bt, i32(have))
    for b, n in enumerate(have):
        p = torch.arange(n, device="cuda")
        rows = bt[b, p // page].long()
        for h in range(hkv):
            r = attention64(Qo[b, 4 * h:4 * h + 4].double()[:, None],
                            kc[rows, h, p % page].double(), vc[rows, h, p % page].double(), False,
                            1 / math.sqrt(d))
            _near("O", O[b, 4 * h:4 * h + 4], r["O"][0][:, 0], r["O"][1][:, 0])
            _near("L", L[b, 4 * h:4 * h + 4], r["L"][0][:, 0], r["L"][1][:, 0])


def test_append_far_into_a_large_cache():
    """Offsets beyond 2^32 bytes."""
    pages, hkv, page, d = 2300, 8, 1024, 128  # 4.8 GB each
    kc = torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, _, _, wq, wk, _, _ = _inputs(3, 16, hkv, d, d, 31)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = fa.rope_table(2000, d)
    args = (i32([0, 3]), i32([1022]), i32([[2299, 2100]]))
    fa.fa_rope_append(q, k, k, *args, kc, vc, table, wq, wk)
    pos = torch.arange(1022, 1025, device="cuda")
    pg = torch.tensor([2299, 2299, 2100], device="cuda")
    y, e = ref.norm_rope64(k, wk, table, pos, 1e-6, False)
    _near("K", kc[pg, :, pos % page], y, ref.rounded(y, e))
    assert torch.equal(vc[pg, :, pos % page], k)
    vc[pg, :, pos % page] = 0
    assert not bool(vc.any())
