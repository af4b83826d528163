"""Packed batches whose work lists take the long ways: ranks that several rounds of the deal
share, more tiles than the deal holds in shared memory, and more cost classes than a plan's
sort has."""
import math

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests.packed_ref import assert_close, attention64, packed64, packed_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def _many(long, short):
    """Sequences around a long one, of 1 to 23 rows, some of them empty."""
    lens = [(5 * i) % 24 for i in range(short)]
    lens.insert(short // 3, long)
    return lens


@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([2990], 64, 1, 40),                 # ten rounds of query blocks on 152 SMs
    ([2990, 1, 500], 48, 1, 128),
    (_many(3500, 1250), 4, 1, 64),       # more than 1024 tiles, and 33 rounds
    (_many(2500, 1200), 2, 1, 96)])
@pytest.mark.parametrize("causal", [True, False])
def test_backward_deals_in_many_rounds(lens, hq, hkv, d, causal):
    q, k, v, do, cu = packed_inputs(lens, hq, hkv, d, 311 + hq, rest=7)
    plan = fa.fa_packed_plan(cu, q.shape[0], causal)
    O, L = fa.fa_packed_forward(q, k, v, plan)
    # what is not written shows: each block is worked on
    grads = [torch.full_like(x, math.nan) for x in (q, k, v)]
    fa.fa_packed_backward(q, k, v, O, L, do, plan, dQ=grads[0], dK=grads[1], dV=grads[2])
    want = packed64(q, k, v, lens, causal, None, do)
    n = sum(lens)
    assert_close("O", O[:n], tuple(x[:n] for x in want["O"]))
    for name, t in zip(("dQ", "dK", "dV"), grads):
        assert_close(name, t[:n], tuple(x[:n] for x in want[name]))
        assert torch.isnan(t[n:].float()).all()
    # and worked on once, in an order that does not vary
    again = fa.fa_packed_backward(q, k, v, O, L, do, fa.fa_packed_plan(cu, q.shape[0], causal))
    for a, b in zip(grads, again):
        assert torch.equal(a[:n], b[:n])


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 64), (2, 2, 128)])
def test_a_sequence_of_many_cost_classes(hq, hkv, d):
    """Above 1024 tiles in one sequence the plan's sort merges classes: rows of every part of
    the long sequence, and of the one behind it, against 64 bits."""
    lens = [140001, 300]
    total = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(313)
    mk = lambda h: torch.randn(total, h, d, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = mk(hq), mk(hkv), mk(hkv)
    cu = torch.tensor([0, lens[0], total], dtype=torch.int32, device="cuda")
    O = torch.full_like(q, math.nan)
    L = torch.full((hq, total), math.nan, device="cuda")
    fa.fa_packed_forward(q, k, v, fa.fa_packed_plan(cu, total), O=O, L=L)
    assert torch.isfinite(O.float()).all() and torch.isfinite(L).all()
    rows = sorted({0, 1, 31, 32, 255, 256, lens[0] - 1, *range(137, lens[0], 4999)})
    per = hq // hkv
    for h in range(hkv):
        kh, vh = k[:lens[0], h].double(), v[:lens[0], h].double()
        for r in rows:
            want = attention64(q[r, h * per:(h + 1) * per].double()[:, None], kh[:r + 1],
                               vh[:r + 1], False, d ** -0.5)
            assert_close("O", O[r, h * per:(h + 1) * per], tuple(x[:, 0] for x in want["O"]))
            assert_close("L", L[h * per:(h + 1) * per, r], tuple(x[:, 0] for x in want["L"]))
    last = slice(lens[0], total)
    want = packed64(q[last], k[last], v[last], [lens[1]], True)
    assert_close("O", O[last], want["O"])
    assert_close("L", L[:, last], want["L"])
