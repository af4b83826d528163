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

from .api import lib
from .packed import _binding, _on_stream


def fa_cache_append(K, V, cu_seqlens, starts, block_table, K_cache, V_cache, stream=None):
    """Writes rows [cu_seqlens[i], cu_seqlens[i + 1]) of K and V [total, Hkv, d] to the
    cache positions starts[i], starts[i] + 1, ... of request i, in place. K and V may be
    slices of one projection (any row stride). Bounds that decrease or leave the rows, and
    places out of range, are reported by fa_get_device_status()."""
    if stream is not None:
        with _on_stream(K_cache, stream):
            return fa_cache_append(K, V, cu_seqlens, starts, block_table, K_cache, V_cache)
    _binding().cache_append(K, V, cu_seqlens, starts, block_table, K_cache, V_cache)


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
    if stream is not None:
        with _on_stream(K_cache, stream):
            return fa_prefix_decode(Q, K_cache, V_cache, prefix_pages, prefix_len, block_table,
                                    lens, scale, O, L, workspace)
    return _binding().prefix_decode(Q, K_cache, V_cache, prefix_pages, prefix_len, block_table,
                                    lens, scale, O, L, workspace)
