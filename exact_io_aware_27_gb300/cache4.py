"""Binding of the paged cache in 4 bits of ``include/fa.h``.

    cache = alloc_cache4(pages, Hkv, page, d, device)
    Qo = fa_cache4_append(Q, K, V, cu_seqlens, starts, block_table, cache, cos_sin, ...)
    O, L = fa_cache4_decode(Qo, cache, block_table, lens)            # one token a request
    K, V = fa_cache4_read(cache, cu_seqlens, starts, block_table, total, d)

The cache is one uint8 tensor [pages, Hkv, page / 16, bytes of 16 rows]: 72 bytes a row, head
and group of 64 channels for K and V together, against 256 in bf16. Every row has a scale and
a minimum per group, and a code of 0 to 15 per channel. Position p of request i lies in row
p % page of page block_table[i, p // page], as in the bf16 cache. fa_cache4_append norms and
turns queries and keys like fa_rope_append; fa_cache4_read gives rows back in bf16, for
attention of several tokens to what the cache holds. fa_packed_forward has as many queries as
keys in each sequence: a prompt's next chunk goes through it with rows of zeros for the queries
before the chunk, whose products are computed too.
"""
from __future__ import annotations

import torch

from .api import lib
from .packed import _binding, _on_stream


def alloc_cache4(num_pages: int, Hkv: int, page: int, d: int, device) -> torch.Tensor:
    """An empty cache of num_pages pages of `page` rows (a power of two from 16 to 1024)."""
    row = int(lib().fa_cache4_row_bytes(d))
    if row == 0 or num_pages < 1 or Hkv < 1 or page not in (16, 32, 64, 128, 256, 512, 1024):
        raise ValueError("invalid sizes for a cache in 4 bits")
    return torch.zeros((num_pages, Hkv, page // 16, 16 * row), dtype=torch.uint8, device=device)


def fa_cache4_append(Q, K, V, cu_seqlens, starts, block_table, cache, cos_sin=None, q_weight=None,
                     k_weight=None, eps: float = 1e-6, interleaved: bool = False, Qo=None,
                     stream=None):
    """fa_rope_append into a cache in 4 bits: rows [cu_seqlens[i], cu_seqlens[i + 1]) of K
    (normed and turned) and V go to positions starts[i], starts[i] + 1, ... of request i.
    Returns Q normed and turned (None for Q = None)."""
    if stream is not None:
        with _on_stream(cache, stream):
            return fa_cache4_append(Q, K, V, cu_seqlens, starts, block_table, cache, cos_sin,
                                    q_weight, k_weight, eps, interleaved, Qo)
    return _binding().cache4_append(Q, K, V, cu_seqlens, starts, block_table, cache, cos_sin,
                                    q_weight, k_weight, eps, interleaved, Qo)


def fa_cache4_read(cache, cu_seqlens, starts, block_table, total: int, d: int, K=None, V=None,
                   stream=None):
    """K and V [total, Hkv, d] bf16: rows [cu_seqlens[i], cu_seqlens[i + 1]) are positions
    starts[i], starts[i] + 1, ... of request i. Rows behind the last request are 0 in tensors
    allocated here and left as they were in tensors that are passed in (both or neither)."""
    if stream is not None:
        with _on_stream(cache, stream):
            return fa_cache4_read(cache, cu_seqlens, starts, block_table, total, d, K, V)
    return _binding().cache4_read(cache, cu_seqlens, starts, block_table, total, d, K, V)


def alloc_cache4_workspace(B: int, Hq: int, Hkv: int, d: int, capacity: int,
                           device) -> torch.Tensor:
    """Workspace of fa_cache4_decode for B requests of at most `capacity` keys (a table
    row's)."""
    size = int(lib().fa_cache4_workspace_bytes(B, Hq, Hkv, d, capacity))
    if size == 0:
        raise ValueError("invalid sizes for the decode workspace")
    return torch.empty(size, dtype=torch.uint8, device=device)


def fa_cache4_decode(Q, cache, block_table, lens, scale: float | None = None, O=None, L=None,
                     workspace=None, stream=None):
    """O [B, Hq, d] bf16 and L [B, Hq] fp32 (natural-log logsumexp) for the queries Q [B, Hq, d]
    of one new token per request, over the first lens[b] positions of block_table[b]. Query
    head h reads key/value head h // (Hq / Hkv)."""
    if stream is not None:
        with _on_stream(cache, stream):
            return fa_cache4_decode(Q, cache, block_table, lens, scale, O, L, workspace)
    return _binding().cache4_decode(Q, cache, block_table, lens, scale, O, L, workspace)
