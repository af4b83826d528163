"""Binding of the packed-sequence entry points of ``include/fa.h``.

A packed batch holds its sequences one after another in one tensor: Q [total, Hq, d],
K and V [total, Hkv, d] (bf16), with bounds cu_seqlens, int32 [nseq + 1] on the device.
Query head h reads key/value head h // (Hq / Hkv).

    plan = fa_packed_plan(cu_seqlens, Q.shape[0])     # once per batch
    O, L = fa_packed_forward(Q, K, V, plan)           # every layer
    dQ, dK, dV = fa_packed_backward(Q, K, V, O, L, dO, plan)

flash_attention_packed(Q, K, V, plan) is the two of them under autograd.

Q, K and V may be slices of one projection [total, (Hq + 2 Hkv) d]: rows may lie any
stride apart, heads and columns are dense.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from . import _build
from .api import FAError, _check, lib

_fast = None


def _binding():
    """The marshalling module (csrc/fa_binding.cpp). Raises if it has not been built."""
    global _fast
    if _fast is None:
        lib()
        if not os.path.exists(_build.BINDING):
            raise RuntimeError(
                f"{_build.BINDING} is not built; run "
                "`python -c 'import __graft_entry__ as g; g.build()'` first")
        loader = importlib.machinery.ExtensionFileLoader("_fa_binding", _build.BINDING)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location("_fa_binding", _build.BINDING, loader=loader))
        loader.exec_module(module)
        module.set_error(FAError)
        _fast = module
    return _fast


def _on_stream(t, stream):
    """The context of a call on `stream`, a torch stream or a raw handle of the tensor's
    device: what the call allocates belongs to that stream."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = (torch.cuda.ExternalStream(handle, device=t.device) if handle
                  else torch.cuda.default_stream(t.device))
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


class PackedPlan:
    """The work lists of one packed batch, on the device (fa_packed_plan)."""

    __slots__ = ("buffer", "nseq", "total", "causal", "version")

    def __init__(self, buffer, nseq, total, causal):
        self.buffer, self.nseq, self.total, self.causal = buffer, nseq, total, causal
        self.version = 0  # times it has been written over

    @property
    def device(self):
        return self.buffer.device


def fa_packed_plan(cu_seqlens, total: int, causal: bool = True, plan: PackedPlan | None = None,
                   stream=None) -> PackedPlan:
    """Plan of the batch with sequence bounds `cu_seqlens` (int32 [nseq + 1] on the
    device, 0 = cu[0] <= ... <= cu[nseq] <= total) in tensors of `total` rows, for causal
    attention or not; at least one sequence and one row. `plan`: an earlier plan of the same
    sizes to write over, for example where the call is captured in a graph."""
    if (not isinstance(cu_seqlens, torch.Tensor) or not cu_seqlens.is_cuda
            or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1
            or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 CUDA tensor")
    device, nseq, total = cu_seqlens.device, cu_seqlens.numel() - 1, int(total)
    size = int(lib().fa_packed_plan_bytes(nseq, total))
    if size == 0:
        raise ValueError(f"invalid sizes for a plan: {nseq} sequences, {total} rows")
    if plan is not None and (plan.nseq, plan.total, plan.device) != (nseq, total, device):
        raise ValueError("plan was made for other sizes or another device")
    with (torch.cuda.device(device) if stream is None else _on_stream(cu_seqlens, stream)):
        buffer = (torch.empty(size, dtype=torch.uint8, device=device) if plan is None
                  else plan.buffer)
        _check("fa_packed_plan",
               lib().fa_packed_plan(cu_seqlens.data_ptr(), nseq, total, int(bool(causal)),
                                    buffer.data_ptr(), size,
                                    torch.cuda.current_stream(device).cuda_stream))
    if plan is None:
        return PackedPlan(buffer, nseq, total, bool(causal))
    plan.causal = bool(causal)
    plan.version += 1
    return plan


def _plan(plan):
    if not isinstance(plan, PackedPlan):
        raise TypeError("plan must be a PackedPlan")
    return plan


def fa_packed_forward(Q, K, V, plan: PackedPlan, scale: float | None = None, O=None, L=None,
                      stream=None):
    """O [total, Hq, d] bf16 and L [Hq, total] fp32 (natural-log logsumexp). Rows behind
    the last sequence are 0 in an O allocated here and -inf in an L allocated here, and
    left as they were in tensors that are passed in."""
    if stream is not None:
        with _on_stream(Q, stream):
            return fa_packed_forward(Q, K, V, plan, scale, O, L)
    p = _plan(plan)
    return _binding().packed_forward(Q, K, V, p.buffer, p.nseq, p.total, p.causal, scale, O, L)


def alloc_packed_workspace(plan: PackedPlan, Hq: int, d: int) -> torch.Tensor:
    """Workspace of fa_packed_backward for the plan's batch and Hq query heads (of any
    head dimension d; it does not change the size)."""
    size = int(lib().fa_packed_workspace_bytes(plan.nseq, plan.total, Hq))
    if size == 0:
        raise ValueError("invalid sizes for the backward workspace")
    return torch.empty(size, dtype=torch.uint8, device=plan.device)


def fa_packed_backward(Q, K, V, O, L, dO, plan: PackedPlan, scale: float | None = None, dQ=None,
                       dK=None, dV=None, workspace=None, stream=None):
    """dQ [total, Hq, d], dK and dV [total, Hkv, d] (bf16) for the gradient dO of the
    forward's O. Rows behind the last sequence are 0 in gradients allocated here and left
    as they were in tensors that are passed in, which may be slices of one
    [total, (Hq + 2 Hkv) d] buffer."""
    if stream is not None:
        with _on_stream(Q, stream):
            return fa_packed_backward(Q, K, V, O, L, dO, plan, scale, dQ, dK, dV, workspace)
    p = _plan(plan)
    return _binding().packed_backward(Q, K, V, p.buffer, p.nseq, p.total, p.causal, scale, O, L,
                                      dO, dQ, dK, dV, workspace)


class FlashAttentionPacked(torch.autograd.Function):
    """Autograd wrapper of fa_packed_forward and fa_packed_backward; saves Q, K, V, O
    and L."""

    @staticmethod
    def forward(ctx, Q, K, V, plan, scale=None):
        O, L = fa_packed_forward(Q, K, V, plan, scale)
        ctx.save_for_backward(Q, K, V, O, L)
        ctx.plan, ctx.version = plan, plan.version
        ctx.scale = scale
        return O

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, L = ctx.saved_tensors
        if ctx.plan.version != ctx.version:
            raise RuntimeError("the plan was written for another batch between the forward and "
                               "the backward pass")
        dQ, dK, dV = fa_packed_backward(Q, K, V, O, L, dO.contiguous(), ctx.plan, ctx.scale)
        return dQ, dK, dV, None, None


def flash_attention_packed(Q, K, V, plan: PackedPlan, scale: float | None = None):
    """Attention over the plan's packed sequences, differentiable (once) in Q, K and V. The
    plan has to hold this batch until the backward pass has run: writing it over in between
    is refused, but for the replay of a captured fa_packed_plan, which Python does not see
    and which gives the gradients of the other batch's bounds. To capture a backward pass
    in a CUDA graph, first drop every eager graph that reaches the same leaves (autograd ties
    a leaf to the stream that first used it, and does not survive waiting for another stream
    during a capture), or capture fa_packed_forward and fa_packed_backward."""
    return FlashAttentionPacked.apply(Q, K, V, plan, scale)
