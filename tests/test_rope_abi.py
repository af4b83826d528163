"""Argument checks of the entry points between projection and attention and of the cache in
4 bits (no GPU: every call is refused before any CUDA work, or reaches the device check)."""
import ctypes

import pytest
import torch

import exact_io_aware_27_gb300 as fa
from exact_io_aware_27_gb300 import api
from tests.test_packed_abi import REACHED, at


class Rope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_int), ("rot", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("eps", ctypes.c_float)]


def how(qw=at(20), kw=at(21), cs=at(22), positions=100, rot=64, eps=1e-6):
    return Rope(qw, kw, cs, positions, rot, 0, eps)


BAD_HOW = (dict(positions=0), dict(rot=4), dict(rot=12), dict(rot=72), dict(eps=-1.0),
           dict(eps=float("nan")), dict(eps=float("inf")))


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.lib()


def test_forward(lib):
    def f(Q=at(0), K=at(1), sq=512, sk=128, total=50, Hq=8, Hkv=2, d=64, pos=at(2), h=how(),
          Qo=at(3), Ko=at(4), sqo=512, sko=128):
        return lib.fa_qk_norm_rope(Q, K, sq, sk, total, Hq, Hkv, d, pos,
                                   ctypes.byref(h) if h else None, Qo, Ko, sqo, sko, None)

    for bad in (dict(Q=None), dict(K=None), dict(Qo=None), dict(Ko=None), dict(pos=None),
                dict(h=None), dict(total=0), dict(total=(1 << 24) + 1), dict(Hq=0), dict(Hkv=0),
                dict(Hq=70000), dict(sq=504), dict(sk=132), dict(sqo=511), dict(sko=1 << 31),
                dict(Qo=at(1)), dict(Ko=at(0)), dict(Ko=at(3)), dict(Qo=at(0), sqo=520),
                dict(Qo=at(0) + 1024), dict(Ko=at(2)), dict(Qo=at(22)),
                *(dict(h=how(**b)) for b in BAD_HOW)):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    for d in (0, 4, 20, 136):
        assert f(d=d, sq=4096, sk=4096, sqo=4096, sko=4096) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(Q=at(0) + 8), dict(Ko=at(4) + 2), dict(pos=at(2) + 2),
                dict(h=how(qw=at(20) + 4)), dict(h=how(cs=at(22) + 8))):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    if not torch.cuda.is_available():
        for good in (dict(), dict(Qo=at(0), Ko=at(1)), dict(h=how(None, None)),
                     dict(h=how(cs=None, rot=3, positions=-1), pos=None),
                     dict(K=at(0) + 1024, sq=768, sk=768),  # side by side in one projection
                     dict(Q=at(0), K=at(0) + 1024, sq=768, sk=768, Qo=at(0), Ko=at(0) + 1024,
                          sqo=768, sko=768)):
            assert f(**good) in REACHED, good


def test_backward(lib):
    size = lib.fa_qk_norm_rope_workspace_bytes
    assert size(0, 2, 64) == 0 and size(8, 0, 64) == 0 and size(8, 2, 20) == 0
    ws = size(8, 2, 64)
    assert ws > 0

    def f(dQo=at(0), dKo=at(1), sdq=512, sdk=128, Q=at(2), K=at(3), sq=512, sk=128, total=50, Hq=8,
          Hkv=2, d=64, pos=at(4), h=how(), dQ=at(5), dK=at(6), oq=512, ok=128, wq=at(7), wk=at(8),
          w=at(9), wb=ws):
        return lib.fa_qk_norm_rope_backward(dQo, dKo, sdq, sdk, Q, K, sq, sk, total, Hq, Hkv, d,
                                            pos, ctypes.byref(h), dQ, dK, oq, ok, wq, wk, w, wb,
                                            None)

    for bad in (dict(dQo=None), dict(dKo=None), dict(Q=None), dict(K=None), dict(pos=None),
                dict(dQ=None), dict(dK=None), dict(wq=None), dict(wk=None), dict(w=None),
                dict(total=0), dict(sdq=500), dict(ok=130), dict(sq=8), dict(dQ=at(0)),
                dict(dK=at(3)), dict(w=at(5)), dict(wq=at(8)), dict(dQ=at(20)),
                *(dict(h=how(**b)) for b in BAD_HOW)):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    assert f(d=12, sdq=4096) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(dQo=at(0) + 2), dict(w=at(9) + 4), dict(wq=at(7) + 2)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    assert f(wb=ws - 1) == api.FA_ERR_WORKSPACE_TOO_SMALL
    if not torch.cuda.is_available():
        assert f() in REACHED
        none = dict(h=how(None, None), Q=None, K=None, wq=None, wk=None, w=None, wb=0)
        assert f(**none) in REACHED
        assert f(h=how(kw=None), K=None, wk=None) in REACHED


@pytest.mark.parametrize("four", [False, True])
def test_append(lib, four):
    def f(Q=at(0), K=at(1), V=at(2), sq=512, sk=128, sv=128, total=50, Hq=8, cu=at(3), starts=at(4),
          nseq=4, table=at(5), max_pages=8, h=how(), Qo=at(6), fill=0, Kc=at(7), Vc=at(8), pages=40,
          Hkv=2, page=16, d=64):
        head = (Q, K, V, sq, sk, sv, total, Hq, cu, starts, nseq, table, max_pages,
                ctypes.byref(h) if h else None, Qo, fill)
        tail = (pages, Hkv, page, d, None)
        return (lib.fa_cache4_append(*head, Kc, *tail) if four
                else lib.fa_rope_append(*head, Kc, Vc, *tail))

    bads = [dict(K=None), dict(V=None), dict(cu=None), dict(starts=None), dict(table=None),
            dict(Kc=None), dict(total=0), dict(nseq=0), dict(nseq=70000), dict(max_pages=0),
            dict(max_pages=1 << 28), dict(pages=0), dict(Hkv=0), dict(page=8), dict(page=24),
            dict(page=2048), dict(sk=120), dict(sv=132), dict(sq=64), dict(pages=1 << 30),
            dict(Kc=at(0)), dict(Kc=at(5)), dict(Qo=at(1)), dict(Qo=at(0)), dict(Q=None),
            dict(Qo=None), dict(Hq=0), dict(Hq=-1), dict(fill=2), dict(h=None), dict(Kc=at(22)),
            *(dict(h=how(**b)) for b in BAD_HOW)]
    if not four:
        bads += [dict(Vc=None), dict(Vc=at(7)), dict(Vc=at(6))]
    for bad in bads:
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    assert f(d=20) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(K=at(1) + 8), dict(Kc=at(7) + 2), dict(cu=at(3) + 2), dict(Qo=at(6) + 8)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    if not torch.cuda.is_available():
        for good in (dict(), dict(Q=None, Qo=None, Hq=0, sq=0), dict(h=how(None, None, None)),
                     dict(K=at(0) + 1024, V=at(0) + 1280, sq=768, sk=768, sv=768)):
            assert f(**good) in REACHED, good


def test_row_bytes(lib):
    assert [lib.fa_cache4_row_bytes(d) for d in (8, 64, 72, 128)] == [72, 72, 144, 144]
    assert [lib.fa_cache4_row_bytes(d) for d in (0, -8, 12, 136)] == [0] * 4


def test_read(lib):
    def f(cache=at(0), pages=40, Hkv=2, page=16, d=64, cu=at(1), starts=at(2), nseq=4, table=at(3),
          max_pages=8, total=50, K=at(4), V=at(5), fill=1):
        return lib.fa_cache4_read(cache, pages, Hkv, page, d, cu, starts, nseq, table, max_pages,
                                  total, K, V, fill, None)

    for bad in (dict(cache=None), dict(cu=None), dict(starts=None), dict(table=None), dict(K=None),
                dict(V=None), dict(total=0), dict(nseq=0), dict(pages=0), dict(page=12),
                dict(max_pages=0), dict(fill=3), dict(K=at(0)), dict(V=at(4)), dict(V=at(1))):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    assert f(d=132) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(cache=at(0) + 8), dict(K=at(4) + 2), dict(table=at(3) + 1)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    if not torch.cuda.is_available():
        assert f() in REACHED


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 8, 64), (32, 4, 128), (40, 2, 128), (7, 1, 40)])
def test_decode_workspace_holds_for_fewer_requests_and_keys(lib, Hq, Hkv, d):
    size = lib.fa_cache4_workspace_bytes
    for B in (1, 39, 41, 330, 8192):
        sizes = [size(B, Hq, Hkv, d, n) for n in (0, 1, 16, 100, 1000, 1 << 14, 1 << 19, 1 << 20,
                                                  1 << 21, 1 << 24, 1 << 27)]
        assert sizes == sorted(sizes)
    for n in (0, 16, 1000, 1 << 21):
        sizes = [size(B, Hq, Hkv, d, n) for B in (*range(1, 400), 4000, 8192)]
        assert sizes == sorted(sizes)


def test_decode(lib):
    size = lib.fa_cache4_workspace_bytes
    assert size(0, 8, 2, 64, 10) == 0 and size(2, 8, 3, 64, 10) == 0
    assert size(2, 258, 2, 64, 10) == 0 and size(9000, 8, 2, 64, 10) == 0
    assert size(2, 8, 2, 64, -1) == 0 and size(2, 8, 2, 20, 10) == 0
    sizes = [size(5, 8, 2, 64, 16 * i) for i in range(0, 400, 7)]
    assert sizes == sorted(sizes) and sizes[0] < sizes[-1]
    ws = size(3, 8, 2, 64, 128)

    def f(Q=at(0), cache=at(1), table=at(2), max_pages=8, lens=at(3), B=3, Hq=8, Hkv=2, d=64,
          pages=40, page=16, scale=0.125, O=at(4), L=at(5), w=at(6), wb=ws):
        return lib.fa_cache4_decode(Q, cache, table, max_pages, lens, B, Hq, Hkv, d, pages, page,
                                    scale, O, L, w, wb, None)

    for bad in (dict(Q=None), dict(cache=None), dict(table=None), dict(lens=None), dict(O=None),
                dict(L=None), dict(w=None), dict(B=0), dict(B=9000), dict(Hq=7), dict(Hq=258),
                dict(max_pages=-1), dict(max_pages=1 << 28), dict(page=48), dict(pages=0),
                dict(scale=0.0), dict(scale=float("nan")), dict(O=at(0)), dict(L=at(4)),
                dict(w=at(1)), dict(O=at(6))):
        assert f(**bad) == api.FA_ERR_INVALID_ARG, bad
    assert f(d=132) == api.FA_ERR_UNSUPPORTED_HEAD_DIM
    for bad in (dict(Q=at(0) + 8), dict(w=at(6) + 8), dict(lens=at(3) + 2), dict(L=at(5) + 2)):
        assert f(**bad) == api.FA_ERR_MISALIGNED, bad
    assert f(wb=ws - 1) == api.FA_ERR_WORKSPACE_TOO_SMALL
    if not torch.cuda.is_available():
        assert f() in REACHED
        assert f(max_pages=0, table=None) in REACHED


def test_binding_refuses(lib):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    kv = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    c4 = torch.zeros(4, 2, 1, 1152, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(x, x)  # not on a GPU
    with pytest.raises(TypeError):
        fa.fa_qk_norm_rope(x, None)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_backward(x, x, x, x)
    with pytest.raises(ValueError):
        fa.fa_rope_append(x, x, x, i, i, i[None], kv, kv)
    with pytest.raises(ValueError):
        fa.fa_cache4_append(x, x, x, i, i, i[None], c4)
    with pytest.raises(ValueError):
        fa.fa_cache4_read(c4, i, i, i[None], 3, 64)
    with pytest.raises(ValueError):
        fa.fa_cache4_decode(x, c4, i[:, None], i)
    for bad in ((0, 2, 16, 64), (4, 0, 16, 64), (4, 2, 8, 64), (4, 2, 48, 64), (4, 2, 16, 20)):
        with pytest.raises(ValueError):
            fa.alloc_cache4(*bad, "cpu")
    assert fa.alloc_cache4(4, 2, 32, 80, "cpu").shape == (4, 2, 2, 2304)
    with pytest.raises(ValueError):
        fa.alloc_cache4_workspace(0, 8, 2, 64, 10, "cpu")
    with pytest.raises(ValueError):
        fa.alloc_qk_norm_rope_workspace(0, 2, 64, "cpu")
