"""Argument checks of the paged-cache entry points (no GPU: every call is refused before
any CUDA work, or reaches the device check)."""
import pytest
import torch

import exact_io_aware_27_gb300 as fa
from exact_io_aware_27_gb300 import api
from tests.test_packed_abi import REACHED, at


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.lib()


def test_append(lib):
    def f(K=at(0), V=at(1), sk=128, sv=128, total=50, cu=at(2), starts=at(3), nseq=4,
          table=at(4), max_pages=8, Kc=at(5), Vc=at(6), pages=40, Hkv=2, page=16, d=64):
        return lib.fa_cache_append(K, V, sk, sv, total, cu, starts, nseq, table, max_pages, Kc, Vc,
                                   pages, Hkv, page, d, None)

    for bad in (dict(K=None), dict(V=None), dict(cu=None), dict(starts=None), dict(table=None),
                dict(Kc=None), dict(Vc=None), dict(total=0), dict(nseq=0), dict(nseq=70000),
                dict(max_pages=0), dict(max_pages=1 << 28), dict(pages=0), dict(Hkv=0),
                dict(page=8), dict(page=24), dict(page=2048), dict(sk=120), dict(sv=132),
                dict(pages=1 << 30), dict(Vc=at(5)), dict(Kc=at(0)), dict(Vc=at(4))):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    assert f(d=20) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(K=at(0) + 8), dict(Vc=at(6) + 2), dict(cu=at(2) + 2), dict(table=at(4) + 1)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    if not torch.cuda.is_available():
        assert f() in REACHED
        assert f(V=at(0) + 256, sk=256, sv=256) in REACHED  # side by side in one projection


def test_prefix_decode(lib):
    size = lib.fa_prefix_workspace_bytes
    assert size(0, 8, 2, 64, 10, 10) == 0 and size(2, 8, 3, 64, 10, 10) == 0
    assert size(2, 258, 2, 64, 10, 10) == 0 and size(9000, 8, 2, 64, 10, 10) == 0
    assert size(2, 8, 2, 64, -1, 10) == 0 and size(2, 8, 2, 20, 10, 10) == 0
    # a larger capacity never needs less
    sizes = [size(5, 8, 2, 64, 16 * i, 16 * j) for i in range(0, 200, 9) for j in (0, 7, 400)]
    assert all(a <= b for a, b in zip(sizes, sizes[3:])) and sizes[0] < sizes[-1]
    ws = size(3, 8, 2, 64, 80, 128)

    def f(Q=at(0), Kc=at(1), Vc=at(2), pp=at(3), npp=5, plen=at(4), table=at(5), max_pages=8,
          lens=at(6), B=3, Hq=8, Hkv=2, d=64, pages=40, page=16, scale=0.125, O=at(7), L=at(8),
          w=at(9), wb=ws):
        return lib.fa_prefix_decode(Q, Kc, Vc, pp, npp, plen, table, max_pages, lens, B, Hq, Hkv,
                                    d, pages, page, scale, O, L, w, wb, None)

    for bad in (dict(Q=None), dict(Kc=None), dict(Vc=None), dict(pp=None), dict(plen=None),
                dict(table=None), dict(lens=None), dict(O=None), dict(L=None), dict(w=None),
                dict(B=0), dict(B=9000), dict(Hq=7), dict(Hq=258), dict(npp=-1),
                dict(max_pages=-1), dict(npp=1 << 28), dict(page=48), dict(pages=0),
                dict(scale=0.0), dict(O=at(0)), dict(L=at(7)), dict(w=at(1)), dict(O=at(9))):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    assert f(d=132) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(Q=at(0) + 8), dict(w=at(9) + 8), dict(lens=at(6) + 2), dict(L=at(8) + 2)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    assert f(wb=ws - 1) == api.FA_ERR_WORKSPACE_TOO_SMALL
    if not torch.cuda.is_available():
        assert f() in REACHED
        assert f(npp=0, pp=None, plen=None, wb=1 << 24) in REACHED
        assert f(max_pages=0, table=None) in REACHED


def test_binding_refuses(lib):
    kv = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_cache_append(x, x, i, i, i[None], kv, kv)  # not on a GPU
    with pytest.raises(ValueError):
        fa.fa_prefix_decode(x, kv, kv, None, None, i[:, None], i)
    with pytest.raises(TypeError):
        fa.fa_prefix_decode(x, None, kv, None, None, i[:, None], i)
    with pytest.raises(ValueError):
        fa.alloc_prefix_workspace(0, 8, 2, 64, 10, 10, "cpu")
