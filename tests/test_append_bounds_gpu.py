"""fa_cache_append with bounds that are not 0 = cu[0] <= ... <= cu[nseq] <= total: reported,
and no row goes to a request that does not own it."""
import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests.packed_ref import packed_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def _append(bounds, total, page=16, hkv=2, d=64):
    """Appends `total` rows; returns (status, row t's request and position or None). Request
    i's page is i, its start 0."""
    _, k, v, _, _ = packed_inputs([total], 1, hkv, d, 67)
    n = len(bounds) - 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kc = torch.zeros((n, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    fa.fa_cache_append(k, v, i32(bounds), i32([0] * n), i32([[i] for i in range(n)]), kc, vc)
    status = fa.fa_get_device_status()
    flat = kc.transpose(1, 2).reshape(n * page, hkv * d)
    written = [r for r in range(n * page) if bool(flat[r].any())]
    places = {}
    for r in written:
        (t,) = [t for t in range(total) if torch.equal(flat[r], k[t].flatten())]
        places.setdefault(t, []).append((r // page, r % page))
        assert torch.equal(vc[r // page, :, r % page], v[t])
    return status, places


@pytest.mark.parametrize("bounds", [
    [0, 5, 3, 10],            # decreasing: rows 3 and 4 lie in two requests
    [0, 8, 2, 4, 10],         # row 4 .. 7 as well
    [1, 5, 10],               # row 0 belongs to none
    [0, 5, 11],               # more rows than there are
    [0, -2, 10], [0, 2 ** 31 - 1, 10], [0, 10, 4]])
def test_bad_bounds_are_reported(bounds):
    status, places = _append(bounds, 10)
    assert status == -8
    assert fa.fa_get_device_status() == 0
    for t, at in places.items():
        for req, pos in at:
            assert bounds[req] <= t < bounds[req + 1] and pos == t - bounds[req]


@pytest.mark.parametrize("bounds", [[0, 10], [0, 0, 4, 4, 9, 9], [0, 0], [0, 3, 10, 10]])
def test_good_bounds(bounds):
    status, places = _append(bounds, 10)
    assert status == 0
    want = {t: [(i, t - bounds[i])] for i in range(len(bounds) - 1)
            for t in range(bounds[i], bounds[i + 1])}
    assert places == want


def test_bad_bounds_among_many_requests():
    """A decrease that no row's search meets."""
    n = 3000
    bounds = [0] * n + [4]
    bounds[1700] = -1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.ones(4, 1, 8, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((1, 1, 16, 8), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    fa.fa_cache_append(k, k, i32(bounds), i32([0] * n), i32([[0]] * n), kc, vc)
    assert fa.fa_get_device_status() == -8
