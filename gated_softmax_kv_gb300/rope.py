"""Python binding of include/csa_rope.h (argument marshalling only) and the
frequency tables that it takes."""
from __future__ import annotations

import math
from typing import Optional

from .binding import _check, _check_detail, _raise, load
from .launch import changed, on_device, output_overlaps

LAYOUTS = {"interleaved": 0, "half": 1}
_codes = {}


def _dtype_code(dtype) -> Optional[int]:
    """CSA_BF16, CSA_FP16, CSA_FP32; None for other types."""
    if not _codes:
        import torch
        _codes.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    return _codes.get(dtype)


def csa_rope(x, freqs, positions=None, *, cu_seqlens_comp=None, ratio: int = 1, offset: int = 0,
             layout: str = "interleaved", amplitude: float = 1.0, transpose: bool = False,
             out=None, stream=None):
    """Turns the columns [offset, offset + 2 * len(freqs)) of every head of x
    by position * freqs (include/csa_rope.h); returns out.

    x: [tokens, heads, head_dim] or [tokens, head_dim], bf16, fp16 or fp32, the
    last dimension contiguous. freqs: fp64 [rope_dim / 2], radians a position
    (csa_rope_freqs makes it). positions: int32 or int64 [tokens]; without it,
    those of compressed rows, from cu_seqlens_comp and ratio. layout:
    "interleaved" pairs columns 2i, 2i + 1; "half" pairs i, i + rope_dim / 2.
    transpose=True gives the gradient (for amplitude 1 also the inverse).
    out=x turns in place; without out a contiguous tensor is made. Not recorded
    by autograd: autograd.rope is.
    """
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dtype, shape, strides = x.dtype, x.shape, x.stride()
    code = _dtype_code(dtype)
    if code is None:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {dtype}")
    if len(shape) == 3:
        T, heads, D = shape
        xt, xh, last = strides
    elif len(shape) == 2:
        (T, D), heads = shape, 1
        (xt, last), xh = strides, 0
    else:
        raise ValueError("x must be [tokens, heads, head_dim] or [tokens, head_dim]")
    dev = x.get_device()
    if dev < 0:
        _check_detail(x, "x", dtype, 0, None)
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
    _check(freqs, "freqs", torch.float64, dev, 1)
    pos_ptr, bits, cu_ptr, nseq = None, 0, None, 0
    if positions is not None:
        if cu_seqlens_comp is not None:
            raise ValueError("positions and cu_seqlens_comp exclude each other")
        if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be an int32 or int64 tensor")
        _check(positions, "positions", positions.dtype, dev, 1)
        if positions.shape[0] != T:
            raise ValueError("positions must be [tokens]")
        # an empty tensor has no address, and nothing of it is read
        pos_ptr, bits = positions.data_ptr() if T else freqs.data_ptr(), 8 * positions.element_size()
    elif cu_seqlens_comp is not None:
        _check(cu_seqlens_comp, "cu_seqlens_comp", torch.int32, dev, 1)
        nseq = cu_seqlens_comp.shape[0] - 1
        if nseq < 1:
            raise ValueError("cu_seqlens_comp must be [num_seqs + 1]")
        cu_ptr = cu_seqlens_comp.data_ptr()
    else:
        raise ValueError("positions or cu_seqlens_comp must be given")
    if heads < 1 or D < 1:
        raise ValueError("x has no heads or no columns")
    if last != 1 and D > 1:
        raise ValueError("the last dimension of x must be contiguous")
    given = out is not None
    with on_device(dev, stream) as launch:
        if out is None:
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
            yt, yh = heads * D, D
        else:
            if not isinstance(out, torch.Tensor) or out.dtype != dtype or out.get_device() != dev:
                raise TypeError("out must be a tensor of x's type and device")
            ys = out.stride()
            if out.shape != shape or (ys[-1] != 1 and D > 1):
                raise ValueError("out must have x's shape and a contiguous last dimension")
            if output_overlaps(out, x):
                raise ValueError("out overlaps x: it must be x itself, with the same strides, or apart")
            yt, yh = ys[0], ys[1] if len(ys) == 3 else 0
        st = load().csa_rope(x.data_ptr(), out.data_ptr(), freqs.data_ptr(), pos_ptr, bits, cu_ptr,
                             nseq, ratio, T, heads, D, xt, xh, yt, yh, 2 * freqs.shape[0], offset,
                             LAYOUTS[layout], code, amplitude, transpose, launch.handle)
        if st != 0:
            _raise(st)
        launch.used(x, out, freqs, positions, cu_seqlens_comp)
    if given:
        changed(out)
    return out


def csa_rope_freqs(rope_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                   original_positions: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                   device="cuda"):
    """(freqs fp64 [rope_dim / 2] on `device`, amplitude) for csa_rope.

    f_i = base^(-2i / rope_dim), then by `scaling` for contexts `factor` times
    `original_positions` long:
      none    f_i
      linear  f_i / factor (positions interpolated)
      ntk     the base raised by factor^(rope_dim / (rope_dim - 2)), which
              leaves the fastest pair alone and stretches the slowest by factor
      yarn    by parts (Peng et al., "YaRN", 2023): pairs that turn more than
              beta_fast times over original_positions are left alone, those
              that turn less than beta_slow times are interpolated, a linear
              ramp over the pair index between; amplitude 0.1 ln(factor) + 1
    """
    import torch
    if rope_dim < 2 or rope_dim % 2:
        raise ValueError("rope_dim must be even and positive")
    if not base > 1.0:
        raise ValueError("base must be above 1")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError("scaling must be none, linear, ntk or yarn")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    if scaling == "yarn" and not (original_positions > 0 and beta_fast >= beta_slow > 0):
        raise ValueError("yarn needs original_positions > 0 and beta_fast >= beta_slow > 0")
    half = rope_dim // 2
    if scaling == "ntk" and rope_dim > 2:
        base = base * factor ** (rope_dim / (rope_dim - 2))
    f = [base ** (-2.0 * i / rope_dim) for i in range(half)]
    amplitude = 1.0
    if scaling == "linear":
        f = [v / factor for v in f]
    elif scaling == "yarn":
        def index_of(turns):  # the (real) pair index that turns so often
            return rope_dim * math.log(original_positions / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(index_of(beta_fast)), 0)
        hi = min(math.ceil(index_of(beta_slow)), rope_dim - 1)
        for i in range(half):
            stretch = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f[i] = f[i] / factor * stretch + f[i] * (1.0 - stretch)
        amplitude = 0.1 * math.log(factor) + 1.0
    return torch.tensor(f, dtype=torch.float64, device=device), amplitude
