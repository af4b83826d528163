"""Keys whose scores are all minus infinity (an infinite entry against queries of the other
sign) have weight 0: a row's result is that of its other keys, whatever the pieces that the
keys are split into."""
import math

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests.packed_ref import assert_close, attention64, packed_inputs
from tests.test_decode_gpu import _batch, _reference, _wide

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def _hide(args, keys, prefix, shared, own, offset=0.0):
    """Gives the shared keys `shared` and the requests' own keys `own` (ranges) scores of
    minus infinity, and returns the keys that are left. All scores are lowered by about
    `offset` / 8 (d = 64) first."""
    q, kc, _, pages, _, table, _ = args
    page = kc.shape[2]
    q[..., 0] = -q[..., 0].abs() - 0.5
    if offset:
        q[..., 1], kc[..., 1] = -16.0, offset / 16.0
    left = []
    for b, (k, v) in enumerate(keys):
        keep = torch.ones(k.shape[0], dtype=torch.bool)
        places = [(pages, i, i) for i in shared]
        places += [(table[b], i, prefix + i) for i in own if prefix + i < k.shape[0]]
        for pgs, i, at in places:
            kc[int(pgs[i // page]), :, i % page, 0] = math.inf
            keep[at] = False
        if offset:
            k = k.clone()
            k[..., 1] = offset / 16.0
        left.append((k[keep], v[keep]))
        assert left[-1][0].shape[0] > 0
    return left


@pytest.mark.parametrize("B,hq,hkv,d", [(3, 8, 2, 64), (2, 4, 1, 128), (20, 8, 2, 128),
                                        (40, 8, 2, 64), (20, 8, 2, 40)])
@pytest.mark.parametrize("shared,own", [((0, 300), (0, 0)), ((0, 0), (0, 70)), ((0, 150), (0, 64)),
                                        ((128, 256), (64, 128))])
def test_decode_parts_without_a_finite_score(B, hq, hkv, d, shared, own):
    """The forms that join parts of the keys: 16 and 32 rows, one row tile and two."""
    args, keys = _batch(300, [(70, 130, 200)[i % 3] for i in range(B)], hq, hkv, d, 16, 5 + B)
    if shared == (0, 0):  # own keys of the shortest requests: all of them
        keys = _hide(args, keys, 300, range(0), range(*own))
    else:
        keys = _hide(args, keys, 300, range(*shared), range(*own))
    want = _reference(args[0], keys, hkv)
    for call in (args, _wide(args)):
        O, L = fa.fa_prefix_decode(*call)
        assert_close("O", O, want["O"])
        assert_close("L", L, want["L"])


def test_decode_of_only_infinite_keys_is_not_a_number():
    """Weights of exp(-inf - -inf): as in the dense form."""
    args, keys = _batch(40, [30, 5, 66], 4, 2, 64, 16, 3)
    args[0][..., 0] = -1.0
    args[1][..., 0] = math.inf
    for call in (args, _wide(args)):
        O, L = fa.fa_prefix_decode(*call)
        assert torch.isnan(O.float()).all() and torch.all(L == -math.inf)


@pytest.mark.parametrize("n,hq,hkv,d", [(700, 8, 1, 64), (700, 1, 1, 128), (300, 4, 2, 64)])
@pytest.mark.parametrize("hidden", [(0, 64), (0, 128), (64, 128), (0, 290), (128, 300)])
def test_forward_steps_without_a_finite_score(n, hq, hkv, d, hidden):
    """The packed forward pass, in single tiles and in pairs."""
    q, k, v, _, cu = packed_inputs([n, 90], hq, hkv, d, 7)
    q[..., 0] = -q[..., 0].abs() - 0.5
    k[hidden[0]:hidden[1], :, 0] = math.inf
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[hidden[0]:hidden[1]] = False
    plan = fa.fa_packed_plan(cu, q.shape[0], causal=False)
    O, L = fa.fa_packed_forward(q, k, v, plan)
    g = hq // hkv
    for h in range(hkv):
        hs = slice(h * g, (h + 1) * g)
        want = attention64(q[:n, hs].double().transpose(0, 1), k[:n][keep, h].double(),
                           v[:n][keep, h].double(), False, d ** -0.5)
        assert_close("O", O[:n, hs], tuple(x.transpose(0, 1) for x in want["O"]))
        assert_close("L", L[hs, :n], want["L"])


@pytest.mark.parametrize("hidden", [(128, 256), (0, 128), (896, 1024)])
def test_decode_in_one_launch_joins_far_below_zero(hidden):
    """A block of the cluster without a finite score, beside blocks whose scores lie far below
    0: it adds nothing to their sums."""
    args, keys = _batch(1024, [20, 24], 8, 2, 64, 16, 11)
    keys = _hide(args, keys, 1024, range(*hidden), range(0), offset=2048.0)
    want = _reference(args[0], keys, 2)
    assert float(want["L"][0].max()) < -200.0
    for call in (args, _wide(args)):
        O, L = fa.fa_prefix_decode(*call)
        assert_close("O", O, want["O"])
        assert_close("L", L, want["L"])
