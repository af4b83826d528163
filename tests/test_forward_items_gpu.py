"""Forward passes whose blocks go from work items with two tiles to items whose second tile is
empty, many times: the softmax warps of the empty tile have nothing to do with that item's
products, and must not lose count of them."""
import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests.packed_ref import assert_close, packed64, packed_inputs
from tests.test_decode_gpu import _batch, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("lens", [[130, 1], [1, 130], [129, 1, 200, 2, 256, 1, 131]])
@pytest.mark.parametrize("hq,hkv,d", [(4095, 1, 8), (2047, 89, 64), (1365, 1, 128)])
def test_packed_items_with_an_empty_tile(lens, hq, hkv, d):
    q, k, v, _, cu = packed_inputs(lens, hq, hkv, d, 17)
    plan = fa.fa_packed_plan(cu, q.shape[0])
    want = packed64(q, k, v, lens, True)
    O, L = fa.fa_packed_forward(q, k, v, plan)
    assert_close("O", O, want["O"])
    assert_close("L", L, want["L"])
    for _ in range(20):
        again = fa.fa_packed_forward(q, k, v, plan)
        assert torch.equal(again[0], O) and torch.equal(again[1], L)


@pytest.mark.parametrize("n", [257, 300, 641])
def test_dense_items_with_an_empty_tile(n):
    """The last pair of every head has one tile."""
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = (torch.randn(4, 512, n, 64, generator=g, device="cuda").to(torch.bfloat16)
               for _ in range(3))
    O, L = fa.fa_forward(q, k, v, causal=True)
    for h in (0, 100, 511):
        want = packed64(*(x[1, h, :, None] for x in (q, k, v)), [n], True)
        assert_close("O", O[1, h, :, None], want["O"])
        assert_close("L", L[1, h, None], want["L"])
    for _ in range(20):
        again = fa.fa_forward(q, k, v, causal=True)
        assert torch.equal(again[0], O) and torch.equal(again[1], L)


def test_decode_items_with_an_empty_tile():
    """Three row tiles of requests: the second pair's second tile is empty."""
    args, keys = _batch(140, [i % 7 for i in range(90)], 64, 16, 64, 16, 5)
    _check(args, keys, 16)
