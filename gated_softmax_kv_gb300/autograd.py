"""Thin torch.autograd wrappers: `compressor` over the Compressor's two C-ABI
calls, and `rope` over csa_rope and its transpose.

`compressor(...)` returns `out` and, on backward, calls csa_compress_bwd for
dkv, dscore and dape (cuDNN-frontend "CSA Fused Compressor", sections
"High-level wrappers" and "Semantics"). Both directions run in
libcsa_compress.so; this module only routes tensors.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import csa_compress_bwd, csa_compress_fwd
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
