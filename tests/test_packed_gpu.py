"""Attention over packed sequences with grouped heads, against 64-bit values with
elementwise bounds (tests/packed_ref.py)."""
import math

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests.packed_ref import assert_close, packed64, packed_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


LENS = {
    "one_token": [1],
    "one_tile": [128],
    "tile_and_one": [129, 257],
    "empty_between": [0, 5, 0, 0, 300, 1, 0],
    "half_steps": [63, 64, 65, 191, 192, 193],
    "long_and_short": [700, 3, 2, 1, 90],
    "many": [(7 * i) % 41 for i in range(150)],
}


def _check(q, k, v, cu, lens, causal, scale=None):
    plan = fa.fa_packed_plan(cu, q.shape[0], causal)
    O, L = fa.fa_packed_forward(q, k, v, plan, scale)
    want = packed64(q, k, v, lens, causal, scale)
    n = sum(lens)
    assert_close("O", O[:n], tuple(x[:n] for x in want["O"]))
    assert_close("L", L[:, :n], tuple(x[:, :n] for x in want["L"]))
    assert torch.all(O[n:] == 0) and torch.all(L[:, n:] == -math.inf)
    return O, L


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (3, 3, 128)])
def test_forward(name, causal, hq, hkv, d):
    lens = LENS[name]
    q, k, v, _, cu = packed_inputs(lens, hq, hkv, d, 11 + len(lens))
    _check(q, k, v, cu, lens, causal)


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 8), (8, 1, 40), (6, 3, 96), (14, 2, 72), (5, 1, 120)])
def test_forward_heads_and_dims(hq, hkv, d):
    lens = [70, 0, 301, 33]
    q, k, v, _, cu = packed_inputs(lens, hq, hkv, d, 5, rest=9)
    _check(q, k, v, cu, lens, True, scale=0.3)


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 64), (16, 2, 128)])
def test_forward_many_items_per_cta(hq, hkv, d):
    lens = [(37 * i) % 400 + 1 for i in range(90)]
    q, k, v, _, cu = packed_inputs(lens, hq, hkv, d, 77)
    _check(q, k, v, cu, lens, True)


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (2, 1, 64), (1, 1, 128), (16, 8, 40)])
@pytest.mark.parametrize("causal", [True, False])
def test_forward_long_sequences_of_few_heads(hq, hkv, d, causal):
    """Fewer row tiles than SMs."""
    lens = [1500, 1, 63, 700]
    q, k, v, _, cu = packed_inputs(lens, hq, hkv, d, 83, rest=3)
    _check(q, k, v, cu, lens, causal)


def test_forward_matches_dense():
    """Sequences of one length are a dense batch: the same kernel, the same bits."""
    B, n, h, d = 3, 384, 4, 128
    q, k, v, _, cu = packed_inputs([n] * B, h, h, d, 21)
    O, L = fa.fa_packed_forward(q, k, v, fa.fa_packed_plan(cu, B * n))
    dense = [x.view(B, n, h, d).transpose(1, 2).contiguous() for x in (q, k, v)]
    Od, Ld = fa.fa_forward(*dense, causal=True)
    assert torch.equal(O.view(B, n, h, d).transpose(1, 2), Od)
    assert torch.equal(L.view(h, B, n).transpose(0, 1), Ld)


def test_forward_projection_slices():
    """Q, K, V as column slices of one projection."""
    lens, hq, hkv, d = [50, 210, 7], 6, 2, 64
    q, k, v, _, cu = packed_inputs(lens, hq, hkv, d, 31)
    wide = torch.cat([x.flatten(1) for x in (q, k, v)], 1)
    qs = wide[:, :hq * d].unflatten(1, (hq, d))
    ks = wide[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    vs = wide[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    plan = fa.fa_packed_plan(cu, q.shape[0])
    a, b = fa.fa_packed_forward(q, k, v, plan), fa.fa_packed_forward(qs, ks, vs, plan)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
def test_forward_sequences_do_not_leak(d):
    """NaN and infinities in one sequence, and in rows of no sequence, stay there."""
    lens = [100, 60, 130, 1]
    q, k, v, _, cu = packed_inputs(lens, 4, 2, d, 41, rest=70)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    clean = fa.fa_packed_forward(q, k, v, plan)
    for t, value in ((q, math.nan), (k, math.nan), (v, math.nan)):
        t[100:160] = value
        t[291:] = math.inf
    O, L = fa.fa_packed_forward(q, k, v, plan)
    keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    keep[100:160] = False
    assert torch.equal(O[keep], clean[0][keep]) and torch.equal(L[:, keep], clean[1][:, keep])
    assert torch.isnan(O[100:160].float()).all()


def test_forward_leaves_the_rest():
    """Outputs that are passed in keep their rows behind the last sequence."""
    lens = [33, 100]
    q, k, v, _, cu = packed_inputs(lens, 2, 1, 64, 51, rest=40)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    O = torch.full_like(q, 7.0)
    L = torch.full((2, q.shape[0]), 5.0, device="cuda")
    fa.fa_packed_forward(q, k, v, plan, O=O, L=L)
    assert torch.all(O[133:] == 7.0) and torch.all(L[:, 133:] == 5.0)
    want = packed64(q, k, v, lens, True)
    assert_close("O", O[:133], tuple(x[:133] for x in want["O"]))


def test_all_sequences_empty():
    q, k, v, _, cu = packed_inputs([0, 0, 0], 2, 2, 64, 3, rest=5)
    O, L = fa.fa_packed_forward(q, k, v, fa.fa_packed_plan(cu, 5))
    assert torch.all(O == 0) and torch.all(L == -math.inf)


@pytest.mark.parametrize("bounds", [[0, 5, 3, 10], [1, 5, 10], [0, 5, 11], [0, -2, 10],
                                    [0, 2 ** 31 - 1, 10]])
def test_bad_bounds_are_reported(bounds):
    q, k, v, _, _ = packed_inputs([10], 2, 2, 64, 3)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    plan = fa.fa_packed_plan(cu, 10)
    O = torch.full_like(q, 3.0)
    L = torch.full((2, 10), 3.0, device="cuda")
    fa.fa_packed_forward(q, k, v, plan, O=O, L=L)
    assert fa.fa_get_device_status() == -8
    assert torch.all(O == 3.0) and torch.all(L == 3.0)
    assert fa.fa_get_device_status() == 0


def test_forward_in_a_graph_and_on_another_stream():
    lens = [40, 260, 3]
    q, k, v, _, cu = packed_inputs(lens, 4, 2, 64, 61)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    want = fa.fa_packed_forward(q, k, v, plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = fa.fa_packed_forward(q, k, v, plan, stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # The plan and the pass captured together: a replay follows new bounds.
    graph = torch.cuda.CUDAGraph()
    O, L = torch.empty_like(q), torch.empty(4, q.shape[0], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fa.fa_packed_plan(cu, q.shape[0], plan=plan)
        fa.fa_packed_forward(q, k, v, plan, O=O, L=L)
    lens = [100, 3, 200]
    cu.copy_(torch.tensor([0, 100, 103, 303], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ref = packed64(q, k, v, lens, True)
    assert_close("O", O, ref["O"])
    assert_close("L", L, ref["L"])


def _grads(q, k, v, do, cu, lens, causal, scale=None, **kw):
    plan = fa.fa_packed_plan(cu, q.shape[0], causal)
    O, L = fa.fa_packed_forward(q, k, v, plan, scale)
    got = fa.fa_packed_backward(q, k, v, O, L, do, plan, scale, **kw)
    want = packed64(q, k, v, lens, causal, scale, do)
    n = sum(lens)
    for name, t in zip(("dQ", "dK", "dV"), got):
        assert_close(name, t[:n], tuple(x[:n] for x in want[name]))
        if not kw:
            assert torch.all(t[n:] == 0), f"{name}: rows of no sequence"
    return got


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (3, 3, 128)])
def test_backward(name, causal, hq, hkv, d):
    lens = LENS[name]
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 111 + len(lens))
    _grads(q, k, v, do, cu, lens, causal)


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 8), (8, 1, 40), (6, 3, 96), (14, 2, 72), (5, 1, 120)])
def test_backward_heads_and_dims(hq, hkv, d):
    lens = [70, 0, 301, 33]
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 105, rest=9)
    _grads(q, k, v, do, cu, lens, True, scale=0.3)


@pytest.mark.parametrize("d", [64, 128])
def test_backward_many_items_per_cta(d):
    lens = [(37 * i) % 400 + 1 for i in range(90)]
    q, k, v, do, cu = packed_inputs(lens, 16, 4, d, 177)
    first = _grads(q, k, v, do, cu, lens, True)
    again = _grads(q, k, v, do, cu, lens, True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))  # no order of atomics


@pytest.mark.parametrize("lens,hq,hkv,d", [([1500, 1, 63, 700], 8, 1, 128), ([2100], 4, 2, 64),
                                           ([700, 30, 1, 900], 6, 2, 40), ([3000], 2, 1, 96)])
@pytest.mark.parametrize("causal", [True, False])
def test_backward_long_sequences_of_few_heads(lens, hq, hkv, d, causal):
    """Few key blocks with many queries each, whose sums come from several SMs."""
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 183, rest=5)
    first = _grads(q, k, v, do, cu, lens, causal)
    again = _grads(q, k, v, do, cu, lens, causal)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 2, 64)])
def test_long_sequences_of_few_heads_do_not_leak(hq, hkv, d):
    lens = [610, 1, 1300]
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 185, rest=30)
    plan = fa.fa_packed_plan(cu, q.shape[0])

    def run():
        O, L = fa.fa_packed_forward(q, k, v, plan)
        return [O, L.T, *fa.fa_packed_backward(q, k, v, O, L, do, plan)]

    clean = run()
    for t in (q, k, v, do):
        t[:610] = math.nan
        t[1911:] = math.inf
    for a, b in zip(run(), clean):
        assert torch.equal(a[610:1911], b[610:1911])


def test_calls_on_two_streams_at_once():
    """Different batches, each with its plan and workspace, interleaved on two streams."""
    jobs = []
    for i, (lens, hq, hkv, d) in enumerate([([1400, 300], 8, 1, 128), ([90] * 20, 8, 4, 64)]):
        q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 191 + i)
        plan = fa.fa_packed_plan(cu, q.shape[0])
        O, L = fa.fa_packed_forward(q, k, v, plan)
        want = fa.fa_packed_backward(q, k, v, O, L, do, plan)
        ws = fa.alloc_packed_workspace(plan, hq, d)
        grads = [[torch.empty_like(x) for x in (q, k, v)] for _ in range(4)]
        outs = [(torch.empty_like(O), torch.empty_like(L)) for _ in range(4)]
        jobs.append((torch.cuda.Stream(), q, k, v, do, plan, O, L, want, ws, grads, outs))
    torch.cuda.synchronize()
    for r in range(4):
        for s, q, k, v, do, plan, O, L, want, ws, grads, outs in jobs:
            fa.fa_packed_forward(q, k, v, plan, O=outs[r][0], L=outs[r][1], stream=s)
            fa.fa_packed_backward(q, k, v, *outs[r], do, plan, dQ=grads[r][0], dK=grads[r][1],
                                  dV=grads[r][2], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for s, q, k, v, do, plan, O, L, want, ws, grads, outs in jobs:
        for r in range(4):
            assert torch.equal(outs[r][0], O) and torch.equal(outs[r][1], L)
            assert all(torch.equal(a, b) for a, b in zip(grads[r], want))


def test_large_scores():
    """Scores of some thousands: rows of one key, a moving maximum, exp far below 1."""
    lens = [200, 700]
    q, k, v, do, cu = packed_inputs(lens, 4, 2, 64, 193, std=20.0)
    _check(q, k, v, cu, lens, True, scale=1.0)
    _grads(q, k, v, do, cu, lens, True, scale=1.0)


def test_the_most_sequences():
    """65535 of them, nearly all empty, and one of the others the last."""
    nseq = 65535
    lens = [0] * nseq
    lens[100], lens[40000], lens[nseq - 1] = 70, 1, 130
    q, k, v, do, cu = packed_inputs(lens, 4, 2, 64, 195, rest=3)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    O, L = fa.fa_packed_forward(q, k, v, plan)
    grads = fa.fa_packed_backward(q, k, v, O, L, do, plan)
    want = packed64(q, k, v, [70, 1, 130], True, None, do)
    assert_close("O", O[:201], tuple(x[:201] for x in want["O"]))
    for name, t in zip(("dQ", "dK", "dV"), grads):
        assert_close(name, t[:201], tuple(x[:201] for x in want[name]))
        assert torch.all(t[201:] == 0)


@pytest.mark.parametrize("hq,hkv,d", [(64, 1, 8), (48, 1, 128), (24, 8, 16)])
def test_many_heads_of_one_key_head(hq, hkv, d):
    lens = [150, 3, 64]
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 196, rest=1)
    _check(q, k, v, cu, lens, True)
    _grads(q, k, v, do, cu, lens, False)


def test_offsets_beyond_32_bits():
    """More than 2^31 values in Q and O: the last sequences against 64 bits."""
    hq, hkv, d, n, count = 64, 1, 128, 500, 530
    total = n * count
    assert total * hq * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(197)
    mk = lambda h: torch.randn(total, h, d, generator=g, device="cuda",  # noqa: E731
                               dtype=torch.bfloat16)
    q, k, v, do = mk(hq), mk(hkv), mk(hkv), mk(hq)
    cu = (torch.arange(count + 1, device="cuda") * n).to(torch.int32)
    plan = fa.fa_packed_plan(cu, total)
    O, L = fa.fa_packed_forward(q, k, v, plan)
    grads = fa.fa_packed_backward(q, k, v, O, L, do, plan)
    for s in (0, count - 1):
        rows = slice(s * n, (s + 1) * n)
        want = packed64(q[rows], k[rows], v[rows], [n], True, None, do[rows])
        assert_close("O", O[rows], want["O"])
        assert_close("L", L[:, rows], want["L"])
        for name, t in zip(("dQ", "dK", "dV"), grads):
            assert_close(name, t[rows], want[name])


def test_backward_of_few_heads_in_a_graph_and_into_one_buffer():
    """Gradients with strides, replayed for another batch of the same sizes."""
    hq, hkv, d, total = 8, 2, 128, 1700
    cut = [0, hq * d, (hq + hkv) * d, (hq + 2 * hkv) * d]
    parts = lambda x: [x[:, a:b].unflatten(1, (-1, d)) for a, b in zip(cut, cut[1:])]  # noqa: E731
    q, k, v, do, cu = packed_inputs([1100, 500], hq, hkv, d, 187, rest=100)
    wide = torch.cat([x.flatten(1) for x in (q, k, v)], 1)
    dwide = torch.full_like(wide, 9.0)
    plan = fa.fa_packed_plan(cu, total)
    ws = fa.alloc_packed_workspace(plan, hq, d)
    O, L = torch.zeros_like(q), torch.zeros(hq, total, device="cuda")
    dq, dk, dv = parts(dwide)

    def step():
        fa.fa_packed_plan(cu, total, plan=plan)
        fa.fa_packed_forward(*parts(wide), plan, O=O, L=L)
        fa.fa_packed_backward(*parts(wide), O, L, do, plan, dQ=dq, dK=dk, dV=dv, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([1100, 500], [20, 1600], [500, 500]):
        cu.copy_(torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32))
        dwide.fill_(9.0)
        ws.fill_(255)  # contents on entry do not matter
        graph.replay()
        torch.cuda.synchronize()
        n = sum(lens)
        want = packed64(q, k, v, lens, True, None, do)
        for name, t in zip(("dQ", "dK", "dV"), (dq, dk, dv)):
            assert_close(name, t[:n], tuple(x[:n] for x in want[name]))
        assert torch.all(dwide[n:] == 9.0)


def test_backward_matches_dense():
    B, n, h, d = 3, 384, 4, 128
    q, k, v, do, cu = packed_inputs([n] * B, h, h, d, 121)
    plan = fa.fa_packed_plan(cu, B * n)
    O, L = fa.fa_packed_forward(q, k, v, plan)
    got = fa.fa_packed_backward(q, k, v, O, L, do, plan)
    dense = [x.view(B, n, h, d).transpose(1, 2).contiguous() for x in (q, k, v, O, do)]
    Ld = L.view(h, B, n).transpose(0, 1).contiguous()
    want = fa.fa_backward(*dense[:4], Ld, dense[4], causal=True)
    for a, b in zip(got, want):
        assert torch.equal(a.view(B, n, h, d).transpose(1, 2), b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_backward_sequences_do_not_leak(d, causal):
    lens = [100, 60, 130, 1]
    q, k, v, do, cu = packed_inputs(lens, 4, 2, d, 141, rest=70)
    plan = fa.fa_packed_plan(cu, q.shape[0], causal)

    def grads():
        O, L = fa.fa_packed_forward(q, k, v, plan)
        return fa.fa_packed_backward(q, k, v, O, L, do, plan)

    clean = grads()
    for t in (q, k, v, do):
        t[100:160] = math.nan
        t[291:] = math.inf
    keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    keep[100:160] = False
    for a, b in zip(grads(), clean):
        assert torch.equal(a[keep], b[keep])


def test_gradients_into_one_buffer_leave_the_rest():
    """Q, K, V and their gradients as slices of one projection and of its gradient."""
    lens, hq, hkv, d = [50, 210, 7], 6, 2, 64
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 131, rest=12)
    cut = [0, hq * d, (hq + hkv) * d, (hq + 2 * hkv) * d]
    parts = lambda x: [x[:, a:b].unflatten(1, (-1, d)) for a, b in zip(cut, cut[1:])]  # noqa: E731
    wide = torch.cat([x.flatten(1) for x in (q, k, v)], 1)
    dwide = torch.full_like(wide, 9.0)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    O, L = fa.fa_packed_forward(*parts(wide), plan)
    dq, dk, dv = parts(dwide)
    fa.fa_packed_backward(*parts(wide), O, L, do, plan, dQ=dq, dK=dk, dV=dv)
    want = fa.fa_packed_backward(q, k, v, O, L, do, plan)
    for a, b in zip((dq, dk, dv), want):
        assert torch.equal(a[:267], b[:267])
    assert torch.all(dwide[267:] == 9.0)


def test_second_derivatives_are_refused():
    q, k, v, do, cu = packed_inputs([30], 2, 1, 64, 199)
    q.requires_grad_()
    out = fa.flash_attention_packed(q, k, v, fa.fa_packed_plan(cu, 30))
    (dq,) = torch.autograd.grad(out, q, do, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dq.float().sum(), q)


def test_autograd_and_differences():
    """flash_attention_packed's gradients against central differences of the 64-bit
    attention along random directions, and against fa_packed_backward."""
    lens, hq, hkv, d = [17, 1, 40], 4, 2, 32
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 151, rest=3)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    out = fa.flash_attention_packed(*leaves, plan)
    out.backward(do)
    n = sum(lens)

    def loss(*x):
        return float((packed64(*x, lens, True)["O"][0][:n] * do[:n].double()).sum())

    want = packed64(q, k, v, lens, True, None, do)
    g = torch.Generator(device="cuda").manual_seed(5)
    for i, name in enumerate(("dQ", "dK", "dV")):
        step = torch.randn(leaves[i].shape, generator=g, device="cuda", dtype=torch.float64)
        x = [y.double() for y in (q, k, v)]
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-5 * step, x[i] - 1e-5 * step
        slope = (loss(*up) - loss(*down)) / 2e-5
        got = float((leaves[i].grad[:n].double() * step[:n]).sum())
        room = float((want[name][1][:n] * step[:n].abs()).sum())
        assert abs(slope - got) <= room + 1e-5 * abs(slope)
        assert torch.all(leaves[i].grad[n:] == 0)
    # A plan that was written for another batch in between is refused.
    out = fa.flash_attention_packed(*leaves, plan)
    fa.fa_packed_plan(cu, q.shape[0], plan=plan)
    with pytest.raises(RuntimeError):
        out.backward(do)


def test_backward_in_a_graph():
    lens = [40, 260, 3]
    q, k, v, do, cu = packed_inputs(lens, 4, 2, 64, 161)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    O, L = fa.fa_packed_forward(q, k, v, plan)
    want = fa.fa_packed_backward(q, k, v, O, L, do, plan)
    got = [torch.empty_like(x) for x in (q, k, v)]
    ws = fa.alloc_packed_workspace(plan, 4, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_packed_forward(q, k, v, plan, O=O, L=L)
        fa.fa_packed_backward(q, k, v, O, L, do, plan, dQ=got[0], dK=got[1], dV=got[2],
                              workspace=ws)
    ws.fill_(255)  # contents on entry do not matter
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_in_a_graph():
    """Forward and backward pass through autograd, captured after a warm-up on a side stream
    whose graph is gone, replayed for other values and another batch of the same sizes."""
    lens, total = [40, 260], 310
    q, k, v, do, cu = packed_inputs(lens, 4, 2, 64, 163, rest=10)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, v)]
    plan = fa.fa_packed_plan(cu, total)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.flash_attention_packed(*leaves, plan).backward(do)
    torch.cuda.current_stream().wait_stream(side)
    for x in leaves:
        x.grad = None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.flash_attention_packed(*leaves, plan).backward(do)
    lens = [300, 5]
    cu.copy_(torch.tensor([0, 300, 305], dtype=torch.int32))
    fa.fa_packed_plan(cu, total, plan=plan)
    with torch.no_grad():
        for x, y in zip(leaves, (q, k, v)):
            x.copy_(y.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = packed64(*(x.detach() for x in leaves), lens, True, None, do)
    for name, x in zip(("dQ", "dK", "dV"), leaves):
        assert_close(name, x.grad[:305], tuple(t[:305] for t in want[name]))
        assert torch.all(x.grad[305:] == 0)
