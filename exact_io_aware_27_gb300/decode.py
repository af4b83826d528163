"""Binding of the paged-cache entry points of ``include/fa.h``.

K_cache and V_cache are bf16 [pages, Hkv, page, d] (page a power of two from 16 to 1024).
Position p of request i lies in row p % page of page block_table[i, p // page].

    fa_cache_append(K, V, cu_seqlens, starts, block_table, K_cache, V_cache)
    O, L = fa_prefix_decode(Q, K_cache, V_cache, prefix_pages, prefix_len, block_table, lens)

appends new rows to the cache, and attends from one new token per request to the prefix
that all requests share (read once for all of them) and to the request's own tokens.
Lengths and tables are int32 tensors on the device; nothing waits for the device.
"""
from __future__ import annotations

import torch

from .api import _check, _out, _scale, _workspace_bytes, lib
from .packed import _BF16, _elsewhere, _int32, _placed, _raw_stream, _row_stride


def _cache(K_cache, V_cache):
    for name, t in (("K_cache", K_cache), ("V_cache", V_cache)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda or t.dtype is not _BF16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [pages, Hkv, page, d]")
    if K_cache.shape != V_cache.shape or K_cache.get_device() != V_cache.get_device():
        raise ValueError("K_cache and V_cache must have one shape and one device")
    return K_cache.shape


def _table(block_table, requests, device):
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 tensor [requests, max_pages]")
    _int32("block_table", block_table, (requests, block_table.shape[1]), device)
    return block_table.shape[1]


def fa_cache_append(K, V, cu_seqlens, starts, block_table, K_cache, V_cache, stream=None):
    """Writes rows [cu_seqlens[i], cu_seqlens[i + 1]) of K and V [total, Hkv, d] to the
    cache positions starts[i], starts[i] + 1, ... of request i, in place. K and V may be
    slices of one projection (any row stride)."""
    num_pages, Hkv, page, d = _cache(K_cache, V_cache)
    device = K_cache.device
    ldk, ldv = _row_stride("K", K), _row_stride("V", V)
    total = K.shape[0]
    if K.shape != V.shape or K.shape[1:] != (Hkv, d):
        raise ValueError(f"K and V must be [total, {Hkv}, {d}]")
    if K.get_device() != device.index or V.get_device() != device.index:
        raise ValueError("all tensors of a call must be on the same device")
    if not isinstance(starts, torch.Tensor) or starts.dim() != 1:
        raise ValueError("starts must be an int32 tensor [requests]")
    nseq = starts.shape[0]
    _int32("starts", starts, (nseq,), device)
    _int32("cu_seqlens", cu_seqlens, (nseq + 1,), device)
    max_pages = _table(block_table, nseq, device)
    if _elsewhere(device, stream):
        with _placed(device, stream):
            return fa_cache_append(K, V, cu_seqlens, starts, block_table, K_cache, V_cache)
    _check("fa_cache_append",
           lib().fa_cache_append(K.data_ptr(), V.data_ptr(), ldk, ldv, total,
                                 cu_seqlens.data_ptr(), starts.data_ptr(), nseq,
                                 block_table.data_ptr(), max_pages, K_cache.data_ptr(),
                                 V_cache.data_ptr(), num_pages, Hkv, page, d,
                                 _raw_stream(device.index)))


def alloc_prefix_workspace(B: int, Hq: int, Hkv: int, d: int, prefix_capacity: int,
                           own_capacity: int, device) -> torch.Tensor:
    """Workspace of fa_prefix_decode for B requests, a prefix of at most prefix_capacity
    keys (the listed pages' rows) and own_capacity keys a request (a table row's)."""
    size = int(lib().fa_prefix_workspace_bytes(B, Hq, Hkv, d, prefix_capacity, own_capacity))
    if size == 0:
        raise ValueError("invalid sizes for the decode workspace")
    return torch.empty(size, dtype=torch.uint8, device=device)


def fa_prefix_decode(Q, K_cache, V_cache, prefix_pages, prefix_len, block_table, lens,
                     scale: float | None = None, O=None, L=None, workspace=None, stream=None):
    """O [B, Hq, d] bf16 and L [B, Hq] fp32 (natural-log logsumexp) for the queries
    Q [B, Hq, d] of one new token per request, over the first prefix_len[0] positions of
    prefix_pages (int32 [n]; both may be None for no prefix) and the first lens[b]
    positions of block_table[b]."""
    num_pages, Hkv, page, d = _cache(K_cache, V_cache)
    device = K_cache.device
    if not isinstance(Q, torch.Tensor):
        raise TypeError("Q must be a torch.Tensor")
    if (Q.dtype is not _BF16 or Q.dim() != 3 or Q.shape[2] != d or Q.device != device
            or not Q.is_contiguous()):
        raise ValueError(f"Q must be a contiguous bf16 tensor [B, Hq, {d}] on {device}")
    B, Hq, _ = Q.shape
    _int32("lens", lens, (B,), device)
    max_pages = _table(block_table, B, device)
    shared = 0
    if prefix_pages is not None:
        if not isinstance(prefix_pages, torch.Tensor) or prefix_pages.dim() != 1:
            raise ValueError("prefix_pages must be an int32 tensor [n]")
        shared = prefix_pages.shape[0]
        _int32("prefix_pages", prefix_pages, (shared,), device)
        _int32("prefix_len", prefix_len, (1,), device)
    if _elsewhere(device, stream):
        with _placed(device, stream):
            return fa_prefix_decode(Q, K_cache, V_cache, prefix_pages, prefix_len, block_table,
                                    lens, scale, O, L, workspace)
    if O is None:
        O = torch.empty_like(Q)
    else:
        _out("O", O, (B, Hq, d), _BF16, device)
    if L is None:
        L = torch.empty((B, Hq), dtype=torch.float32, device=device)
    else:
        _out("L", L, (B, Hq), torch.float32, device)
    if workspace is None:
        workspace = alloc_prefix_workspace(B, Hq, Hkv, d, shared * page, max_pages * page, device)
    size = _workspace_bytes(workspace, device)
    _check("fa_prefix_decode",
           lib().fa_prefix_decode(Q.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(),
                                  prefix_pages.data_ptr() if shared else None, shared,
                                  prefix_len.data_ptr() if shared else None,
                                  block_table.data_ptr() if max_pages else None, max_pages,
                                  lens.data_ptr(), B, Hq, Hkv, d, num_pages, page,
                                  _scale(scale, d), O.data_ptr(), L.data_ptr(),
                                  workspace.data_ptr(), size, _raw_stream(device.index)))
    return O, L
