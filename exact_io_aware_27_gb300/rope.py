"""Binding of the entry points of ``include/fa.h`` between projection and attention: norms of
queries and keys for each head, with the position rotation in the same pass.

    cos_sin = rope_table(positions, rot)                   # once
    Qo, Ko = fa_qk_norm_rope(Q, K, positions, cos_sin, q_weight, k_weight)
    dQ, dK, dq_weight, dk_weight = fa_qk_norm_rope_backward(dQo, dKo, Q, K, positions, ...)

qk_norm_rope(...) is the two of them under autograd, for use before flash_attention_packed;
fa_rope_append is fa_cache_append with the same on the way into the paged cache.

Q [total, Hq, d] and K [total, Hkv, d] may be slices of one projection (any row stride).
q_weight and k_weight (bf16 [d]) scale the normed rows; without one, that tensor is not
normed. cos_sin (fp32 [positions, rot]) has a position's cosines, then its sines; without it
nothing is turned. Pairs are channels (i, i + rot / 2), or (2 i, 2 i + 1) with `interleaved`.
"""
from __future__ import annotations

import torch

from .api import lib
from .packed import _binding, _on_stream


def rope_table(positions: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The usual table, fp32 [positions, rot]: position p turns pair i by p / base^(2 i / rot).
    Angles are computed in 64 bits, since 32 lose the far positions'."""
    if positions < 1 or rot < 8 or rot % 8 != 0:
        raise ValueError("positions must be at least 1 and rot a multiple of 8")
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    at = torch.arange(positions, dtype=torch.float64, device=device)
    angle = at[:, None] * base ** (-i / rot)
    return torch.cat([torch.cos(angle), torch.sin(angle)], dim=1).float()


def fa_qk_norm_rope(Q, K, positions=None, cos_sin=None, q_weight=None, k_weight=None,
                    eps: float = 1e-6, interleaved: bool = False, Qo=None, Ko=None, stream=None):
    """(Qo, Ko): Q and K normed and turned, row t by the angles of positions[t] (int32 on the
    device). Qo may be Q and Ko K: the rows are then changed in place. Positions that cos_sin
    does not have are reported by fa_get_device_status() and their rows not written."""
    if stream is not None:
        with _on_stream(Q, stream):
            return fa_qk_norm_rope(Q, K, positions, cos_sin, q_weight, k_weight, eps, interleaved,
                                   Qo, Ko)
    return _binding().qk_norm_rope(Q, K, positions, cos_sin, q_weight, k_weight, eps, interleaved,
                                   Qo, Ko)


def alloc_qk_norm_rope_workspace(Hq: int, Hkv: int, d: int, device) -> torch.Tensor:
    """Workspace of fa_qk_norm_rope_backward (for any number of rows)."""
    size = int(lib().fa_qk_norm_rope_workspace_bytes(Hq, Hkv, d))
    if size == 0:
        raise ValueError("invalid sizes for the workspace")
    return torch.empty(size, dtype=torch.uint8, device=device)


def fa_qk_norm_rope_backward(dQo, dKo, Q, K, positions=None, cos_sin=None, q_weight=None,
                             k_weight=None, eps: float = 1e-6, interleaved: bool = False, dQ=None,
                             dK=None, workspace=None, stream=None):
    """(dQ, dK, dq_weight, dk_weight) for gradients dQo and dKo of fa_qk_norm_rope's outputs on
    the same inputs. The weights' gradients are fp32 [d], None for a weight that is None."""
    if stream is not None:
        with _on_stream(Q, stream):
            return fa_qk_norm_rope_backward(dQo, dKo, Q, K, positions, cos_sin, q_weight, k_weight,
                                            eps, interleaved, dQ, dK, workspace)
    return _binding().qk_norm_rope_backward(dQo, dKo, Q, K, positions, cos_sin, q_weight, k_weight,
                                            eps, interleaved, dQ, dK, workspace)


def _dense_rows(t):
    """A gradient as the kernels take it: heads and columns dense, rows 16 bytes aligned."""
    rows, heads, d = t.shape
    ok = (t.stride(2) == 1 and t.stride(1) == d and t.stride(0) >= heads * d
          and t.stride(0) % 8 == 0 and t.data_ptr() % 16 == 0)
    # a copy, also of one that is dense but starts between two 16-byte boundaries
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class QKNormRope(torch.autograd.Function):
    """Autograd wrapper of fa_qk_norm_rope and its backward; saves Q and K."""

    @staticmethod
    def forward(ctx, Q, K, positions, cos_sin, q_weight, k_weight, eps, interleaved):
        ctx.save_for_backward(Q, K, positions, cos_sin, q_weight, k_weight)
        ctx.eps, ctx.interleaved = eps, interleaved
        return fa_qk_norm_rope(Q, K, positions, cos_sin, q_weight, k_weight, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dQo, dKo):
        Q, K, positions, cos_sin, q_weight, k_weight = ctx.saved_tensors
        dQ, dK, dwq, dwk = fa_qk_norm_rope_backward(
            _dense_rows(dQo), _dense_rows(dKo), Q, K, positions, cos_sin, q_weight, k_weight,
            ctx.eps, ctx.interleaved)
        cast = lambda g, w: None if g is None else g.to(w.dtype)  # noqa: E731
        return dQ, dK, None, None, cast(dwq, q_weight), cast(dwk, k_weight), None, None


def qk_norm_rope(Q, K, positions=None, cos_sin=None, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False):
    """fa_qk_norm_rope, differentiable (once) in Q, K and the weights. As with
    flash_attention_packed, drop every eager graph that reaches the same leaves before
    capturing a backward pass in a CUDA graph, or capture the two calls."""
    return QKNormRope.apply(Q, K, positions, cos_sin, q_weight, k_weight, eps, interleaved)


def fa_rope_append(Q, K, V, cu_seqlens, starts, block_table, K_cache, V_cache, cos_sin=None,
                   q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                   Qo=None, stream=None):
    """fa_cache_append of K normed and turned, by the angles of the cache positions that its
    rows go to, and of V as it is; returns Q normed and turned by the same positions,
    [total, Hq, d] (None for Q = None). Rows without a position are 0 in a Qo allocated here,
    and left as they were in one that is passed in."""
    if stream is not None:
        with _on_stream(K_cache, stream):
            return fa_rope_append(Q, K, V, cu_seqlens, starts, block_table, K_cache, V_cache,
                                  cos_sin, q_weight, k_weight, eps, interleaved, Qo)
    return _binding().rope_append(Q, K, V, cu_seqlens, starts, block_table, K_cache, V_cache,
                                  cos_sin, q_weight, k_weight, eps, interleaved, Qo)
