"""Thin torch.autograd wrappers: `compressor` over the Compressor's two C-ABI
calls, `rope` over csa_rope and its transpose, `norm_rope` over csa_norm_rope
and `prompt_attend` over csa_prompt_attend and their gradients.

`compressor(...)` returns `out` and, on backward, calls csa_compress_bwd for
dkv, dscore and dape (cuDNN-frontend "CSA Fused Compressor", sections
"High-level wrappers" and "Semantics"). Both directions run in
libcsa_compress.so; this module only routes tensors.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import csa_compress_bwd, csa_compress_fwd
from .norm_rope import csa_norm_rope, csa_norm_rope_bwd
from .prompt import csa_prompt_attend, csa_prompt_attend_bwd
from .rope import csa_rope


class CompressorFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, kv, score, ape, cu_seqlens, cu_seqlens_comp, capacity: int, ratio: int,
                coff: int, head_dim: int, exact: bool = False):
        out = csa_compress_fwd(kv, score, ape, cu_seqlens, cu_seqlens_comp, capacity, ratio, coff,
                               head_dim, exact=exact)
        ctx.save_for_backward(kv, score, ape, cu_seqlens, cu_seqlens_comp)
        ctx.meta = (capacity, ratio, coff, head_dim, exact)
        return out

    @staticmethod
    def backward(ctx, grad_out):
        kv, score, ape, cu, cuc = ctx.saved_tensors
        capacity, ratio, coff, head_dim, exact = ctx.meta
        dkv, dscore, dape = csa_compress_bwd(kv, score, ape, cu, cuc, capacity, ratio, coff, head_dim,
                                             grad_out.contiguous(), exact=exact)
        return dkv, dscore, dape, None, None, None, None, None, None, None


def compressor(kv: torch.Tensor, score: torch.Tensor, ape: torch.Tensor, cu_seqlens: torch.Tensor,
               cu_seqlens_comp: torch.Tensor, ratio: int, coff: int, head_dim: int,
               capacity: Optional[int] = None, exact: bool = False) -> torch.Tensor:
    """Differentiable fused Compressor. `capacity` defaults to cu_seqlens_comp[-1],
    which reads the device (a host synchronisation); pass a static capacity to
    keep the call free of synchronisation (e.g. for CUDA-graph capture).
    exact=True runs both directions in the exact mode (windows of at most 8
    slots)."""
    if capacity is None:
        capacity = int(cu_seqlens_comp[-1].item())
    return CompressorFunction.apply(kv, score, ape, cu_seqlens, cu_seqlens_comp, capacity, ratio,
                                    coff, head_dim, exact)


class RopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, freqs, positions, cu_seqlens_comp, ratio: int, offset: int, layout: str,
                amplitude: float, transpose: bool):
        ctx.save_for_backward(freqs, positions, cu_seqlens_comp)
        ctx.meta = (ratio, offset, layout, amplitude, transpose)
        return csa_rope(x, freqs, positions, cu_seqlens_comp=cu_seqlens_comp, ratio=ratio,
                        offset=offset, layout=layout, amplitude=amplitude, transpose=transpose)

    @staticmethod
    def backward(ctx, grad):
        # the operator is linear: its gradient is its transpose, itself differentiable
        freqs, positions, cuc = ctx.saved_tensors
        ratio, offset, layout, amplitude, transpose = ctx.meta
        if grad.stride(-1) != 1:
            grad = grad.contiguous()
        if grad.requires_grad and torch.is_grad_enabled():  # a graph of the gradient is wanted
            dx = RopeFunction.apply(grad, freqs, positions, cuc, ratio, offset, layout, amplitude,
                                    not transpose)
        else:
            dx = csa_rope(grad, freqs, positions, cu_seqlens_comp=cuc, ratio=ratio, offset=offset,
                          layout=layout, amplitude=amplitude, transpose=not transpose)
        return dx, None, None, None, None, None, None, None, None


def rope(x: torch.Tensor, freqs: torch.Tensor, positions: Optional[torch.Tensor] = None, *,
         cu_seqlens_comp: Optional[torch.Tensor] = None, ratio: int = 1, offset: int = 0,
         layout: str = "interleaved", amplitude: float = 1.0,
         transpose: bool = False) -> torch.Tensor:
    """Differentiable csa_rope (same arguments, no in-place form): the gradient
    with respect to x is the transposed turn of grad_out, in one launch.
    freqs and positions are constants. As with every operator of torch, a
    backward pass is captured into a CUDA graph only while no eager graph of
    the same leaf tensors is alive (torch ties a leaf's accumulation node to
    the stream it was made on and would make the capture wait for it)."""
    return RopeFunction.apply(x, freqs, positions, cu_seqlens_comp, ratio, offset, layout,
                              amplitude, transpose)


def _rows_contiguous(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """Kernels read rows whose last dimension is contiguous."""
    return t if t is None or t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class NormRopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp, how):
        ctx.save_for_backward(q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp)
        ctx.how = how
        return csa_norm_rope(q, q_weight, freqs, positions, k=k, k_weight=k_weight,
                             cu_seqlens_comp=cu_seqlens_comp, **how)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, k_grad):
        q, q_weight, k, k_weight, freqs, positions, cuc = ctx.saved_tensors
        dq, dqw, dk, dkw = csa_norm_rope_bwd(q, q_weight, freqs, _rows_contiguous(grad), positions, k=k,
                                             k_weight=k_weight, k_grad=_rows_contiguous(k_grad),
                                             cu_seqlens_comp=cuc, **ctx.how)
        return dq, dqw, dk, dkw, None, None, None, None


def norm_rope(q: torch.Tensor, q_weight: torch.Tensor, freqs: torch.Tensor,
              positions: Optional[torch.Tensor] = None, *, k: Optional[torch.Tensor] = None,
              k_weight: Optional[torch.Tensor] = None, cu_seqlens_comp: Optional[torch.Tensor] = None,
              ratio: int = 1, offset: int = 0, layout: str = "interleaved", amplitude: float = 1.0,
              eps: float = 1e-6):
    """Differentiable csa_norm_rope (same arguments, no in-place form): (out,
    k_out), k_out None without k, with gradients of q, k and their weights; freqs
    and positions are constants. The gradient is not itself differentiable.
    Captured into a CUDA graph under the condition that `rope` states."""
    how = dict(ratio=ratio, offset=offset, layout=layout, amplitude=amplitude, eps=eps)
    return NormRopeFunction.apply(q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp, how)


def _vectors_apart(t: torch.Tensor) -> bool:
    """Whether csa_prompt_attend_bwd takes a gradient as it lies in memory: 16-byte
    aligned rows, no dimension broadcast."""
    return (t.stride(2) == 1 and t.data_ptr() % 16 == 0
            and all(t.shape[i] == 1 or t.stride(i) > 0 and t.stride(i) % 8 == 0 for i in (0, 1)))


class PromptAttendFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, sm_scale: float, window):
        rest = torch.empty_like(q, memory_format=torch.contiguous_format)
        out, lse = csa_prompt_attend(q, k, v, cu_q, sm_scale, cu_k=cu_k, window=window, rest=rest)
        ctx.save_for_backward(q, k, v, cu_q, cu_k, out, lse, rest)
        ctx.how = (sm_scale, window)
        ctx.set_materialize_grads(False)
        return out, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_lse):
        if grad is None and grad_lse is None:
            return None, None, None, None, None, None, None
        q, k, v, cu_q, cu_k, out, lse, rest = ctx.saved_tensors
        sm_scale, window = ctx.how
        if grad is None:
            grad = torch.zeros_like(out)
        elif not _vectors_apart(grad):
            grad = grad.clone(memory_format=torch.contiguous_format)
        if grad_lse is not None:
            grad_lse = grad_lse.contiguous()
        dq, dk, dv = csa_prompt_attend_bwd(q, k, v, out, lse, grad, cu_q, sm_scale, cu_k=cu_k, window=window,
                                           rest=rest, grad_lse=grad_lse)
        return dq, dk, dv, None, None, None, None


def prompt_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, sm_scale: float, *,
                  cu_k: Optional[torch.Tensor] = None, window: Optional[int] = None):
    """Differentiable csa_prompt_attend (same arguments, no outputs of the caller's):
    (out, lse), both with gradients to q, k and v. A gradient that arrives broadcast
    or unaligned is copied first. The gradient is not itself differentiable.
    For the gradient it keeps q, k, v, out, lse and what out's rounding left off, a tensor
    of out's size; where none is wanted that is not made. Captured into a CUDA graph
    under the condition that `rope` states."""
    if not (torch.is_grad_enabled() and any(getattr(t, "requires_grad", False) for t in (q, k, v))):
        return csa_prompt_attend(q, k, v, cu_q, sm_scale, cu_k=cu_k, window=window)
    return PromptAttendFunction.apply(q, k, v, cu_q, cu_k, sm_scale, window)
