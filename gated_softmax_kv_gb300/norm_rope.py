"""Python binding of include/csa_norm_rope.h (argument marshalling only): norms of
queries and keys for each head with the rotary positions in the same pass."""
from __future__ import annotations

import struct

from .binding import _check, _check_detail, _raise, load
from .launch import changed, on_device, output_overlaps
from .rope import LAYOUTS, _dtype_code

# csa_norm_side_t: x, weight, grad, y, dweight; (token, head) strides of x, grad and y; heads
_side = struct.Struct("@5P6qi4x").pack
# csa_norm_rope_t: freqs, positions, cu_rows; tokens; nine numbers; amplitude and eps
_how = struct.Struct("@3Pq9i2f4x").pack


def _strides(t, name):
    """(heads, token stride, head stride) of [tokens, heads, head_dim] or [tokens, head_dim]."""
    s = t.stride()
    if len(s) not in (2, 3):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] or [tokens, head_dim]")
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return (t.shape[1], s[0], s[1]) if len(s) == 3 else (1, s[0], 0)


def _describe(q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp, ratio, offset, layout, amplitude, eps):
    """(the C description, q's and k's (heads, token stride, head stride), the device) of a
    call. Reading attributes is most of the host's time: each is read once, and the
    checks that name a fault run where there is one."""
    import torch
    try:
        dt, dev, wt = q.dtype, q.get_device(), q_weight.dtype
        code, wcode, (pairs,) = _dtype_code(dt), _dtype_code(wt), freqs.shape
        T, D, a, b = q.shape[0], q.shape[-1], _strides(q, "q"), None
        fine = (dev >= 0 and code is not None and (wt is dt or wcode == 2) and q_weight.shape == (D,) and a[0] > 0 and D > 0
                and q_weight.get_device() == dev and q_weight.is_contiguous() and freqs.dtype is torch.float64
                and freqs.get_device() == dev and freqs.is_contiguous() and layout in LAYOUTS)
        if fine and k is not None:
            b = _strides(k, "k")
            fine = (k.dtype is dt and k.get_device() == dev and k.shape[0] == T and k.shape[-1] == D and b[0] > 0
                    and k_weight.dtype is wt and k_weight.get_device() == dev and k_weight.is_contiguous()
                    and k_weight.shape == (D,))
        where = positions if positions is not None else cu_seqlens_comp
        (length,), kind = where.shape, where.dtype
        fine = (fine and where.get_device() == dev and where.is_contiguous()
                and (kind is torch.int32 and length > 1 if positions is None else
                     cu_seqlens_comp is None and length == T and (kind is torch.int64 or kind is torch.int32)))
    except (AttributeError, ValueError, TypeError):
        fine = False
    if not fine:
        _refuse(q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp, layout)
        a, b = _strides(q, "q"), None if k is None else _strides(k, "k")
        T, D, dev = q.shape[0], q.shape[-1], q.get_device()
        code, wcode, pairs = _dtype_code(q.dtype), _dtype_code(q_weight.dtype), freqs.shape[0]
    if positions is None:
        pos, bits, cu, nseq = 0, 0, cu_seqlens_comp.data_ptr(), cu_seqlens_comp.shape[0] - 1
    else:  # an empty tensor has no address, and nothing of it is read
        pos, bits, cu, nseq = positions.data_ptr() if T else freqs.data_ptr(), 8 * positions.element_size(), 0, 0
    return _how(freqs.data_ptr(), pos, cu, T, bits, nseq, ratio, D, 2 * pairs, offset, LAYOUTS[layout], code, wcode,
                amplitude, eps), a, b, dev


def _refuse(q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp, layout):
    """Names what a call's tensors are not; returns where they are unusual but fine."""
    import torch
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if _dtype_code(q.dtype) is None:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {q.dtype}")
    dev = q.get_device()
    if dev < 0:
        _check_detail(q, "q", q.dtype, 0, None)
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
    _check(freqs, "freqs", torch.float64, dev, 1)
    if not isinstance(q_weight, torch.Tensor) or q_weight.dtype not in (q.dtype, torch.float32):
        raise TypeError("weights must be tensors of q's type or float32")
    if q.dim() not in (2, 3) or 0 in q.shape[1:]:
        raise ValueError("q must be [tokens, heads, head_dim] or [tokens, head_dim], with heads and columns")
    T, D = q.shape[0], q.shape[-1]
    if positions is not None:
        if cu_seqlens_comp is not None:
            raise ValueError("positions and cu_seqlens_comp exclude each other")
        if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be an int32 or int64 tensor")
        _check(positions, "positions", positions.dtype, dev, 1)
        if positions.shape[0] != T:
            raise ValueError("positions must be [tokens]")
    elif cu_seqlens_comp is not None:
        _check(cu_seqlens_comp, "cu_seqlens_comp", torch.int32, dev, 1)
        if cu_seqlens_comp.shape[0] < 2:
            raise ValueError("cu_seqlens_comp must be [num_seqs + 1]")
    else:
        raise ValueError("positions or cu_seqlens_comp must be given")
    for x, w, names in ((q, q_weight, ("q", "q_weight")), (k, k_weight, ("k", "k_weight"))):
        if x is None:
            continue
        if not isinstance(x, torch.Tensor) or x.dtype != q.dtype or x.get_device() != dev:
            raise TypeError(f"{names[0]} must be a tensor of q's type and device")
        if _strides(x, names[0])[0] < 1 or x.shape[0] != T or x.shape[-1] != D:
            raise ValueError(f"{names[0]} must have q's tokens and head_dim, and heads")
        _check(w, names[1], q_weight.dtype, dev, 1)
        if w.shape[0] != D:
            raise ValueError(f"{names[1]} must be [head_dim]")


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
    if k is None and (k_weight is not None or k_out is not None):
        raise ValueError("k_weight and k_out go with k")
    how, (heads, xt, xh), side, dev = _describe(q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp, ratio, offset,
                                                layout, amplitude, eps)
    given = [t for t in (out, k_out) if t is not None]
    with on_device(dev, stream) as launch:
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            yt, yh = heads * q.shape[-1], q.shape[-1]
        else:
            _target(out, q, "out", (k,), dev)
            _, yt, yh = _strides(out, "out")
        a = _side(q.data_ptr(), q_weight.data_ptr(), 0, out.data_ptr(), 0, xt, xh, 0, 0, yt, yh, heads)
        b = None
        if k is not None:
            heads, xt, xh = side
            if k_out is None:
                k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
                yt, yh = heads * k.shape[-1], k.shape[-1]
            else:
                _target(k_out, k, "k_out", (q, out), dev)
                _, yt, yh = _strides(k_out, "k_out")
            b = _side(k.data_ptr(), k_weight.data_ptr(), 0, k_out.data_ptr(), 0, xt, xh, 0, 0, yt, yh, heads)
        st = load().csa_norm_rope(how, a, b, launch.handle)
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
    if k is None and (k_weight is not None or k_grad is not None):
        raise ValueError("k_weight and k_grad go with k")
    how, q_side, k_side, dev = _describe(q, q_weight, k, k_weight, freqs, positions, cu_seqlens_comp, ratio, offset, layout,
                                         amplitude, eps)
    with on_device(dev, stream) as launch:
        made, sides = [], []
        for s, x, w, g, name in ((q_side, q, q_weight, grad, "grad"), (k_side, k, k_weight, k_grad, "k_grad")):
            if x is None:
                made += [None, None]
                sides.append(None)
                continue
            if not isinstance(g, torch.Tensor) or g.dtype != x.dtype or g.get_device() != dev or g.shape != x.shape:
                raise TypeError(f"{name} must be a tensor of its input's shape, type and device")
            (heads, xt, xh), (_, gt, gh), D = s, _strides(g, name), x.shape[-1]
            dx, dw = torch.empty_like(x, memory_format=torch.contiguous_format), torch.empty_like(w)
            sides.append(_side(x.data_ptr(), w.data_ptr(), g.data_ptr(), dx.data_ptr(), dw.data_ptr(), xt, xh, gt, gh,
                               heads * D, D, heads))
            made += [dx, dw]
        st = load().csa_norm_rope_bwd(how, *sides, launch.handle)
        if st != 0:
            _raise(st)
        launch.used(q, k, q_weight, k_weight, freqs, positions, cu_seqlens_comp, grad, k_grad, *made)
    return tuple(made)
