"""Python binding of include/csa_norm_rope.h (argument marshalling only): norms of
queries and keys for each head with the rotary positions in the same pass."""
from __future__ import annotations

import ctypes

from .binding import _check, _check_detail, _raise, load
from .launch import changed, on_device, output_overlaps
from .rope import LAYOUTS, _dtype_code


class _Side(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "weight", "grad", "y", "dweight")]
                + [(n, ctypes.c_int64) for n in ("xt", "xh", "gt", "gh", "yt", "yh")]
                + [("heads", ctypes.c_int32)])


class _How(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("cu_rows", ctypes.c_void_p),
                ("tokens", ctypes.c_int64), ("position_bits", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("ratio", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("offset", ctypes.c_int32), ("layout", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("amplitude", ctypes.c_float), ("eps", ctypes.c_float)]


def _strides(t, name):
    """(heads, token stride, head stride) of [tokens, heads, head_dim] or [tokens, head_dim]."""
    s = t.stride()
    if len(s) not in (2, 3):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] or [tokens, head_dim]")
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return (t.shape[1], s[0], s[1]) if len(s) == 3 else (1, s[0], 0)


def _how(x, weight, freqs, positions, cu_seqlens_comp, ratio, offset, layout, amplitude, eps):
    """(the C description, the device) of a call, from its first side."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    code = _dtype_code(x.dtype)
    if code is None:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {x.dtype}")
    dev = x.get_device()
    if dev < 0:
        _check_detail(x, "q", x.dtype, 0, None)
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
    _check(freqs, "freqs", torch.float64, dev, 1)
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (x.dtype, torch.float32):
        raise TypeError("weights must be tensors of q's type or float32")
    T = x.shape[0] if x.dim() else 0
    pos, bits, cu, nseq = None, 0, None, 0
    if positions is not None:
        if cu_seqlens_comp is not None:
            raise ValueError("positions and cu_seqlens_comp exclude each other")
        if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be an int32 or int64 tensor")
        _check(positions, "positions", positions.dtype, dev, 1)
        if positions.shape[0] != T:
            raise ValueError("positions must be [tokens]")
        # an empty tensor has no address, and nothing of it is read
        pos, bits = positions.data_ptr() if T else freqs.data_ptr(), 8 * positions.element_size()
    elif cu_seqlens_comp is not None:
        _check(cu_seqlens_comp, "cu_seqlens_comp", torch.int32, dev, 1)
        nseq = cu_seqlens_comp.shape[0] - 1
        if nseq < 1:
            raise ValueError("cu_seqlens_comp must be [num_seqs + 1]")
        cu = cu_seqlens_comp.data_ptr()
    else:
        raise ValueError("positions or cu_seqlens_comp must be given")
    if x.dim() not in (2, 3) or 0 in x.shape[1:]:
        raise ValueError("q must be [tokens, heads, head_dim] or [tokens, head_dim], with heads and columns")
    return _How(freqs.data_ptr(), pos, cu, T, bits, nseq, ratio, x.shape[-1], 2 * freqs.shape[0], offset,
                LAYOUTS[layout], code, _dtype_code(weight.dtype), amplitude, eps), dev


def _fits(x, weight, names, how, dev, like, wlike):
    """Checks a side against the first one's types and sizes."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dtype != like.dtype or x.get_device() != dev:
        raise TypeError(f"{names[0]} must be a tensor of q's type and device")
    heads, ts, hs = _strides(x, names[0])
    if x.shape[0] != how.tokens or x.shape[-1] != how.head_dim or heads < 1:
        raise ValueError(f"{names[0]} must have q's tokens and head_dim, and heads")
    _check(weight, names[1], wlike.dtype, dev, 1)
    if weight.shape[0] != how.head_dim:
        raise ValueError(f"{names[1]} must be [head_dim]")
    return _Side(x=x.data_ptr(), weight=weight.data_ptr(), xt=ts, xh=hs, heads=heads)


def _target(out, x, name, others, dev):
    """An output of the caller's: x's shape, type and device; an input itself, or apart."""
    import torch
    if not isinstance(out, torch.Tensor) or out.dtype != x.dtype or out.get_device() != dev:
        raise TypeError(f"{name} must be a tensor of its input's type and device")
    if out.shape != x.shape:
        raise ValueError(f"{name} must have its input's shape")
    if output_overlaps(out, x) or any(o is not None and _meets(out, o) for o in others):
        raise ValueError(f"{name} overlaps another tensor: it must be its input itself, with the same strides, or apart")


def _meets(a, b) -> bool:
    """Whether a and b share memory, by the elements' span: views of the same rows
    that interleave (queries and keys side by side) do not."""
    if a.numel() == 0 or b.numel() == 0:
        return False
    if a.data_ptr() == b.data_ptr():
        return True
    if not output_overlaps(a, b):
        return False
    # the same token stride: apart where the two stretches of a token's row are
    if a.dim() == b.dim() == 3 and a.stride(0) == b.stride(0) > 0:
        row = a.stride(0) * a.element_size()
        span = [1 + sum((n - 1) * s for n, s in zip(t.shape[1:], t.stride()[1:])) for t in (a, b)]
        at = (b.data_ptr() - a.data_ptr()) % row // a.element_size()
        return not (at >= span[0] and at + span[1] <= a.stride(0))
    return True


def csa_norm_rope(q, q_weight, freqs, positions=None, *, k=None, k_weight=None, cu_seqlens_comp=None,
                  ratio: int = 1, offset: int = 0, layout: str = "interleaved", amplitude: float = 1.0,
                  eps: float = 1e-6, out=None, k_out=None, stream=None):
    """Norms every head of q (and of k) over its columns, weighs the columns and
    turns [offset, offset + 2 * len(freqs)) of them by position * freqs
    (include/csa_norm_rope.h); returns (out, k_out), k_out None without k.

    q, k: [tokens, heads, head_dim] or [tokens, head_dim], bf16, fp16 or fp32, the
    last dimension contiguous; views of one projection's output work. Weights:
    [head_dim], of q's type or fp32, both the same. freqs, positions,
    cu_seqlens_comp, ratio, offset, layout and amplitude as in csa_rope (packed
    tokens: their cu_seqlens and ratio 1). out=q and k_out=k work in place;
    without them contiguous tensors are made. Not recorded by autograd:
    autograd.norm_rope is.
    """
    import torch
    how, dev = _how(q, q_weight, freqs, positions, cu_seqlens_comp, ratio, offset, layout, amplitude, eps)
    a = _fits(q, q_weight, ("q", "q_weight"), how, dev, q, q_weight)
    b = None
    if k is not None:
        b = _fits(k, k_weight, ("k", "k_weight"), how, dev, q, q_weight)
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out go with k")
    given = [t for t in (out, k_out) if t is not None]
    with on_device(dev, stream) as launch:
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _target(out, q, "out", (k,), dev)
        if k is not None:
            if k_out is None:
                k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
            else:
                _target(k_out, k, "k_out", (q, out), dev)
            _, b.yt, b.yh = _strides(k_out, "k_out")
            b.y = k_out.data_ptr()
        _, a.yt, a.yh = _strides(out, "out")
        a.y = out.data_ptr()
        st = load().csa_norm_rope(ctypes.byref(how), ctypes.byref(a), None if b is None else ctypes.byref(b),
                                  launch.handle)
        if st != 0:
            _raise(st)
        launch.used(q, k, q_weight, k_weight, freqs, positions, cu_seqlens_comp, out, k_out)
    if given:
        changed(*given)
    return out, k_out


def csa_norm_rope_bwd(q, q_weight, freqs, grad, positions=None, *, k=None, k_weight=None, k_grad=None,
                      cu_seqlens_comp=None, ratio: int = 1, offset: int = 0, layout: str = "interleaved",
                      amplitude: float = 1.0, eps: float = 1e-6, stream=None):
    """The gradient of csa_norm_rope with the same arguments: grad and k_grad are
    those of out and k_out; returns (dq, dq_weight, dk, dk_weight), the last two
    None without k. The gradients are contiguous, the weights' in their type."""
    import torch
    how, dev = _how(q, q_weight, freqs, positions, cu_seqlens_comp, ratio, offset, layout, amplitude, eps)
    a = _fits(q, q_weight, ("q", "q_weight"), how, dev, q, q_weight)
    b = None
    if k is not None:
        b = _fits(k, k_weight, ("k", "k_weight"), how, dev, q, q_weight)
    elif k_weight is not None or k_grad is not None:
        raise ValueError("k_weight and k_grad go with k")
    with on_device(dev, stream) as launch:
        made = []
        for s, x, w, g, name in ((a, q, q_weight, grad, "grad"), (b, k, k_weight, k_grad, "k_grad")):
            if s is None:
                made += [None, None]
                continue
            if not isinstance(g, torch.Tensor) or g.dtype != x.dtype or g.get_device() != dev or g.shape != x.shape:
                raise TypeError(f"{name} must be a tensor of its input's shape, type and device")
            _, s.gt, s.gh = _strides(g, name)
            dx, dw = torch.empty_like(x, memory_format=torch.contiguous_format), torch.empty_like(w)
            _, s.yt, s.yh = _strides(dx, "dx")
            s.grad, s.y, s.dweight = g.data_ptr(), dx.data_ptr(), dw.data_ptr()
            made += [dx, dw]
        st = load().csa_norm_rope_bwd(ctypes.byref(how), ctypes.byref(a), None if b is None else ctypes.byref(b),
                                      launch.handle)
        if st != 0:
            _raise(st)
        launch.used(q, k, q_weight, k_weight, freqs, positions, cu_seqlens_comp, grad, k_grad, *made)
    return tuple(made)
