"""Argument checks of the packed-sequence entry points (no GPU: every call is refused
before any CUDA work, or reaches the device check)."""
import pytest
import torch

import exact_io_aware_27_gb300 as fa
from exact_io_aware_27_gb300 import api
from exact_io_aware_27_gb300 import packed

BASE = 1 << 20  # aligned addresses that are never followed


def at(i):
    return BASE + (i << 26)


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.lib()


REACHED = (api.FA_ERR_CUDA, api.FA_ERR_UNSUPPORTED_DEVICE)


def test_plan(lib):
    size = lib.fa_packed_plan_bytes(5, 1000)
    # header, lists of 256-, 128- (two), 64- and 32-row tiles, four scans
    assert size == 64 + 16 * (3 + 5 + 2 * (7 + 5) + 15 + 5 + 31 + 5) + 6 * 4 * 4
    assert lib.fa_packed_plan_bytes(0, 10) == 0
    assert lib.fa_packed_plan_bytes(70000, 10) == 0
    assert lib.fa_packed_plan_bytes(1, 0) == 0
    assert lib.fa_packed_plan_bytes(1, (1 << 24) + 1) == 0
    f = lambda cu=at(0), nseq=5, total=1000, plan=at(1), size=size: lib.fa_packed_plan(  # noqa: E731
        cu, nseq, total, 1, plan, size, None)
    assert f(cu=None) == api.FA_ERR_INVALID_ARG
    assert f(plan=None) == api.FA_ERR_INVALID_ARG
    assert f(total=0) == api.FA_ERR_INVALID_ARG
    assert f(cu=at(0) + 2) == api.FA_ERR_MISALIGNED
    assert f(plan=at(1) + 8) == api.FA_ERR_MISALIGNED
    assert f(size=size - 1) == api.FA_ERR_WORKSPACE_TOO_SMALL
    assert f(cu=at(1) + 64) == api.FA_ERR_INVALID_ARG  # cu_seqlens inside the plan


def test_forward(lib):
    def f(Q=at(0), K=at(1), V=at(2), sq=512, sk=128, sv=128, total=100, Hq=8, Hkv=2, d=64,
          scale=0.125, plan=at(3), nseq=3, O=at(4), L=at(5), fill=0):
        return lib.fa_packed_forward(Q, K, V, sq, sk, sv, total, Hq, Hkv, d, 1, scale, plan, nseq,
                                     O, L, fill, None)

    for bad in (dict(Q=None), dict(V=None), dict(plan=None), dict(O=None), dict(L=None),
                dict(total=0), dict(nseq=0), dict(Hkv=3), dict(Hkv=0), dict(Hq=0),
                dict(sq=504), dict(sq=516), dict(sk=120), dict(sv=1 << 31), dict(scale=0.0),
                dict(scale=float("nan")), dict(fill=4), dict(O=at(0)), dict(L=at(4)),
                dict(O=at(3)), dict(total=1 << 24, nseq=65535, Hq=65535, Hkv=1, sq=65535 * 64)):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    for d in (0, 4, 12, 136):
        assert f(d=d) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(Q=at(0) + 8), dict(plan=at(3) + 4), dict(O=at(4) + 2), dict(L=at(5) + 2)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    if not torch.cuda.is_available():
        assert f() in REACHED
        # slices of one projection, side by side in its rows
        assert f(K=at(0) + 1024, V=at(0) + 1280, sq=768, sk=768, sv=768) in REACHED
        assert f(sq=1 << 30, total=1) in REACHED


def test_backward(lib):
    rows = (7 + 3) * 128 * 4 * 8
    assert rows <= lib.fa_packed_workspace_bytes(3, 1000, 4) <= rows + 34 * 10 ** 6
    assert lib.fa_packed_workspace_bytes(3, 100, 4) <= (3 * 128 * 4 * 8) + 10 ** 5
    assert lib.fa_packed_workspace_bytes(0, 1000, 4) == 0
    ws = lib.fa_packed_workspace_bytes(3, 100, 8)

    def f(Q=at(0), K=at(1), V=at(2), sq=512, sk=128, sv=128, O=at(3), L=at(4), dO=at(5), d=64,
          scale=0.125, plan=at(6), dQ=at(7), dK=at(8), dV=at(9), sdq=512, sdk=128, sdv=128,
          fill=0, w=at(10), wb=ws, Hkv=2):
        return lib.fa_packed_backward(Q, K, V, sq, sk, sv, O, L, dO, 100, 8, Hkv, d, 1, scale,
                                      plan, 3, dQ, dK, dV, sdq, sdk, sdv, fill, w, wb, None)

    for bad in (dict(K=None), dict(O=None), dict(L=None), dict(dO=None), dict(dQ=None),
                dict(dV=None), dict(w=None), dict(plan=None), dict(Hkv=3), dict(fill=8),
                dict(scale=-1.0), dict(sdq=256), dict(sdk=132), dict(dQ=at(0)), dict(dK=at(8) + 64,
                dV=at(8)), dict(w=at(7)), dict(dV=at(6)), dict(w=at(5))):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    assert f(d=20) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(dK=at(8) + 8), dict(w=at(10) + 8), dict(L=at(4) + 2)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    assert f(wb=ws - 1) == api.FA_ERR_WORKSPACE_TOO_SMALL
    if not torch.cuda.is_available():
        assert f() in REACHED
        one = dict(dQ=at(7), dK=at(7) + 1024, dV=at(7) + 1280, sdq=768, sdk=768, sdv=768)
        assert f(**one) in REACHED  # gradients side by side in one buffer
        one["dV"] -= 16
        assert f(**one) == api.FA_ERR_INVALID_ARG


def test_binding_refuses(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_packed_plan(cu, 4)  # not on a GPU
    with pytest.raises(TypeError):
        fa.fa_packed_forward(x, x, x, None)
    plan = packed.PackedPlan(torch.zeros(8, dtype=torch.uint8), 1, 4, True)
    L = torch.zeros(2, 4)
    with pytest.raises(TypeError):
        fa.fa_packed_forward(None, x, x, plan)
    with pytest.raises(ValueError):
        fa.fa_packed_forward(x, x, x, plan)  # not on a GPU
    with pytest.raises(ValueError):
        fa.fa_packed_forward(x, x, x, plan, stream=0)
    with pytest.raises(ValueError):
        fa.fa_packed_backward(x, x, x, x, L, x, plan)
    with pytest.raises(TypeError):
        fa.fa_packed_backward(x, x, x, x, L, x, None)
