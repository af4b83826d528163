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

import torch

from .api import _check, _out, _scale, _workspace_bytes, lib

_BF16 = torch.bfloat16
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream  # current stream of a device, as a handle


def _elsewhere(device, stream) -> bool:
    """True when a call has to enter _placed first: `stream` is given, or the tensors are
    not on the current device. The common call is neither, and costs no context."""
    return stream is not None or device.index != _current_device()


def _placed(device, stream):
    """The context a call allocates and launches in: the tensors' device, and `stream`
    (a torch stream or a raw handle of that device) when one is given."""
    if stream is None:
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                  else torch.cuda.default_stream(device))
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _row_stride(name, t):
    """Elements from row to row of a bf16 [rows, heads, d] CUDA tensor whose heads and
    columns are dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype is not _BF16 or t.dim() != 3:
        raise ValueError(f"{name} must be a bf16 CUDA tensor [rows, heads, d]")
    rows, heads, d = t.shape
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (heads > 1 and s1 != d):
        raise ValueError(f"{name} must be dense in its heads and columns")
    if rows <= 1:
        return heads * d
    if s0 < heads * d or s0 % 8:
        raise ValueError(f"{name} must have a row stride that is a multiple of 8 and at least "
                         "heads * d")
    return s0


def _int32(name, t, shape, device):
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or tuple(t.shape) != shape
            or not t.is_contiguous() or t.device != device):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape} on {device}")


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
    attention or not. `plan`: an earlier plan of the same sizes to write over, for example
    where the call is captured in a graph."""
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be a 1-D int32 CUDA tensor")
    device, nseq, total = cu_seqlens.device, cu_seqlens.numel() - 1, int(total)
    _int32("cu_seqlens", cu_seqlens, (nseq + 1,), device)
    size = int(lib().fa_packed_plan_bytes(nseq, total))
    if size == 0:
        raise ValueError(f"invalid sizes for a plan: {nseq} sequences, {total} rows")
    if plan is not None and (plan.nseq, plan.total, plan.device) != (nseq, total, device):
        raise ValueError("plan was made for other sizes or another device")
    if _elsewhere(device, stream):
        with _placed(device, stream):
            return fa_packed_plan(cu_seqlens, total, causal, plan)
    buffer = torch.empty(size, dtype=torch.uint8, device=device) if plan is None else plan.buffer
    _check("fa_packed_plan",
           lib().fa_packed_plan(cu_seqlens.data_ptr(), nseq, total, int(bool(causal)),
                                buffer.data_ptr(), size, _raw_stream(device.index)))
    if plan is None:
        return PackedPlan(buffer, nseq, total, bool(causal))
    plan.causal = bool(causal)
    plan.version += 1
    return plan


def _packed_inputs(Q, K, V, plan):
    """Checks Q, K, V against each other and the plan; returns their row strides and
    (Hq, Hkv, d)."""
    if not isinstance(plan, PackedPlan):
        raise TypeError("plan must be a PackedPlan")
    strides = _row_stride("Q", Q), _row_stride("K", K), _row_stride("V", V)
    total, Hq, d = Q.shape
    rows, Hkv, dk = K.shape
    if K.shape != V.shape or rows != total or dk != d:
        raise ValueError("K and V must be [total, Hkv, d] with Q's rows and d")
    if Hkv == 0 or Hq % Hkv:
        raise ValueError("the number of query heads must be a multiple of the key/value heads")
    if total != plan.total:
        raise ValueError(f"the plan is for {plan.total} rows, Q has {total}")
    at = Q.get_device()
    if K.get_device() != at or V.get_device() != at or plan.buffer.get_device() != at:
        raise ValueError("all tensors of a call must be on the same device")
    return strides, Hq, Hkv, d


def fa_packed_forward(Q, K, V, plan: PackedPlan, scale: float | None = None, O=None, L=None,
                      stream=None):
    """O [total, Hq, d] bf16 and L [Hq, total] fp32 (natural-log logsumexp). Rows behind
    the last sequence are 0 in an O allocated here and -inf in an L allocated here, and
    left as they were in tensors that are passed in."""
    (ldq, ldk, ldv), Hq, Hkv, d = _packed_inputs(Q, K, V, plan)
    total, device = plan.total, Q.device
    if _elsewhere(device, stream):
        with _placed(device, stream):
            return fa_packed_forward(Q, K, V, plan, scale, O, L)
    fill = 0
    if O is None:
        O, fill = torch.empty((total, Hq, d), dtype=_BF16, device=device), 1
    else:
        _out("O", O, (total, Hq, d), _BF16, device)
    if L is None:
        L, fill = torch.empty((Hq, total), dtype=torch.float32, device=device), fill | 2
    else:
        _out("L", L, (Hq, total), torch.float32, device)
    _check("fa_packed_forward",
           lib().fa_packed_forward(Q.data_ptr(), K.data_ptr(), V.data_ptr(), ldq, ldk, ldv, total,
                                   Hq, Hkv, d, plan.causal, _scale(scale, d),
                                   plan.buffer.data_ptr(), plan.nseq, O.data_ptr(), L.data_ptr(),
                                   fill, _raw_stream(device.index)))
    return O, L


def alloc_packed_workspace(plan: PackedPlan, Hq: int, d: int) -> torch.Tensor:
    """Workspace of fa_packed_backward for the plan's batch and Hq query heads (of any
    head dimension d; it does not change the size)."""
    size = int(lib().fa_packed_workspace_bytes(plan.nseq, plan.total, Hq))
    if size == 0:
        raise ValueError("invalid sizes for the backward workspace")
    return torch.empty(size, dtype=torch.uint8, device=plan.device)


def _gradient(name, like, t):
    """(tensor, row stride, allocated here) of a gradient with the shape of `like`."""
    if t is None:
        return torch.empty(like.shape, dtype=_BF16, device=like.device), \
            like.shape[1] * like.shape[2], True
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != like.shape or t.device != like.device:
        raise ValueError(f"{name} must have the shape {tuple(like.shape)} on {like.device}")
    return t, _row_stride(name, t), False


def fa_packed_backward(Q, K, V, O, L, dO, plan: PackedPlan, scale: float | None = None, dQ=None,
                       dK=None, dV=None, workspace=None, stream=None):
    """dQ [total, Hq, d], dK and dV [total, Hkv, d] (bf16) for the gradient dO of the
    forward's O. Rows behind the last sequence are 0 in gradients allocated here and left
    as they were in tensors that are passed in, which may be slices of one
    [total, (Hq + 2 Hkv) d] buffer."""
    (ldq, ldk, ldv), Hq, Hkv, d = _packed_inputs(Q, K, V, plan)
    total, device = plan.total, Q.device
    for name, t in (("O", O), ("dO", dO)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if (t.dtype is not _BF16 or t.shape != Q.shape or not t.is_contiguous()
                or t.device != device):
            raise ValueError(f"{name} must be a contiguous bf16 tensor of Q's shape on {device}")
    if (not isinstance(L, torch.Tensor) or L.dtype != torch.float32 or L.device != device
            or tuple(L.shape) != (Hq, total) or not L.is_contiguous()):
        raise ValueError("L must be a contiguous fp32 [Hq, total] tensor on the inputs' device")
    if _elsewhere(device, stream):
        with _placed(device, stream):
            return fa_packed_backward(Q, K, V, O, L, dO, plan, scale, dQ, dK, dV, workspace)
    dQ, lddq, new_q = _gradient("dQ", Q, dQ)
    dK, lddk, new_k = _gradient("dK", K, dK)
    dV, lddv, new_v = _gradient("dV", V, dV)
    if workspace is None:
        workspace = alloc_packed_workspace(plan, Hq, d)
    size = _workspace_bytes(workspace, device)
    _check("fa_packed_backward",
           lib().fa_packed_backward(Q.data_ptr(), K.data_ptr(), V.data_ptr(), ldq, ldk, ldv,
                                    O.data_ptr(), L.data_ptr(), dO.data_ptr(), total, Hq, Hkv, d,
                                    plan.causal, _scale(scale, d), plan.buffer.data_ptr(),
                                    plan.nseq, dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), lddq,
                                    lddk, lddv, new_q | new_k << 1 | new_v << 2,
                                    workspace.data_ptr(), size, _raw_stream(device.index)))
    return dQ, dK, dV


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
    def backward(ctx, dO):
        Q, K, V, O, L = ctx.saved_tensors
        if ctx.plan.version != ctx.version:
            raise RuntimeError("the plan was written for another batch between the forward and "
                               "the backward pass")
        dQ, dK, dV = fa_packed_backward(Q, K, V, O, L, dO.contiguous(), ctx.plan, ctx.scale)
        return dQ, dK, dV, None, None


def flash_attention_packed(Q, K, V, plan: PackedPlan, scale: float | None = None):
    """Attention over the plan's packed sequences, differentiable in Q, K and V. The plan
    has to hold this batch until the backward pass has run."""
    return FlashAttentionPacked.apply(Q, K, V, plan, scale)
