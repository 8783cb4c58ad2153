"""Python binding of include/csa_prompt.h (argument marshalling only): causal
attention over packed sequences, and its gradient."""
from __future__ import annotations

import ctypes

from .binding import _check, _check_detail, _raise, load
from .launch import _span, changed, on_device

FILL_OUT, FILL_LSE = 1, 2


class _Prompt(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "cu_q", "cu_k")]
                + [(n, ctypes.c_int64) for n in ("num_q", "num_k", "qt", "qh", "kt", "kh", "vt", "vh")]
                + [(n, ctypes.c_int32) for n in ("num_seqs", "heads", "kv_heads", "head_dim", "dtype", "window")]
                + [("sm_scale", ctypes.c_float)])


_codes = {}


def _dtype_code(dtype):
    """CSA_BF16, CSA_FP16; None for other types."""
    if not _codes:
        import torch
        _codes.update({torch.bfloat16: 0, torch.float16: 1})
    return _codes.get(dtype)


def _rows(t, name, like, dev):
    """The (token, head) strides of a [tokens, heads, head_dim] tensor of q's type."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype} as q is, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    s = t.stride()
    if len(s) != 3 or t.shape[2] != like.shape[2] or (s[2] != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with q's head_dim and a contiguous last dimension")
    return s[0], s[1]


def _describe(q, k, v, cu_q, cu_k, sm_scale, window):
    """(the C description, the device) of a call."""
    import torch
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    code = _dtype_code(q.dtype)
    if code is None:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    dev = q.get_device()
    if dev < 0:
        _check_detail(q, "q", q.dtype, 0, 3)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    qt, qh = _rows(q, "q", q, dev)
    kt, kh = _rows(k, "k", q, dev)
    vt, vh = _rows(v, "v", q, dev)
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    T, H, D = q.shape
    N, KV, _ = k.shape
    if KV < 1 or H < 1 or H % KV != 0:
        raise ValueError("q's heads must be a multiple of k's")
    _check(cu_q, "cu_q", torch.int32, dev, 1)
    n = cu_q.shape[0] - 1
    if n < 1:
        raise ValueError("cu_q must be [num_seqs + 1]")
    if cu_k is not None:
        _check(cu_k, "cu_k", torch.int32, dev, 1)
        if cu_k.shape[0] != n + 1:
            raise ValueError("cu_k must be as long as cu_q")
    elif N != T:
        raise ValueError("without cu_k, k must have q's tokens")
    if window is not None and window < 1:
        raise ValueError("window must be at least 1, or None for all keys")
    # a window of 2^31 tokens and more is none: a sequence has fewer
    return _Prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), None if cu_k is None else cu_k.data_ptr(),
                   T, N, qt, qh, kt, kh, vt, vh, n, H, KV, D, code,
                   0 if window is None or window >= 2 ** 31 else window, sm_scale), dev


def _apart(t, name, *others):
    a, b = _span(t)
    for o in others:
        if o is not None:
            c, d = _span(o)
            if a < d and c < b:
                raise ValueError(f"{name} overlaps another tensor of the call")


def csa_prompt_attend(q, k, v, cu_q, sm_scale: float, *, cu_k=None, window=None, out=None, lse=None, rest=None,
                      stream=None):
    """Causal attention of packed queries q [tokens, heads, head_dim] over packed
    keys and values [keys, kv_heads, head_dim] (bf16 or fp16; views of one
    projection's output work); returns (out, lse) (include/csa_prompt.h).

    cu_q, cu_k: int32 [num_seqs + 1], where sequences begin and end; without cu_k
    the keys are the queries' own tokens. With more keys than queries the queries
    are the last tokens of their sequence: a chunk of a prompt, or a single token,
    behind what is held. window: how many tokens a query sees, its own included
    (None: all). lse (natural logarithm, fp32 [tokens, heads]) lets the result be
    merged with csa_cache_attend's over compressed rows.

    Rows of no sequence (a static capacity's) are 0, and -inf in lse, in tensors
    that the call makes, and left as they were in those that it is given. rest (of
    out's shape) takes what out's rounding left off, for the gradient. Not recorded
    by autograd: autograd.prompt_attend is.
    """
    import torch
    p, dev = _describe(q, k, v, cu_q, cu_k, sm_scale, window)
    T, H, _ = q.shape
    fill, given = 0, [t for t in (out, lse, rest) if t is not None]
    with on_device(dev, stream) as launch:
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            fill |= FILL_OUT
        else:
            _check(out, "out", q.dtype, dev, 3)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
            _apart(out, "out", q, k, v)
        if lse is None:
            lse = torch.empty((T, H), dtype=torch.float32, device=dev)
            fill |= FILL_LSE
        else:
            _check(lse, "lse", torch.float32, dev, 2)
            if tuple(lse.shape) != (T, H):
                raise ValueError("lse must be [tokens, heads]")
            _apart(lse, "lse", q, k, v, out)
        if rest is not None:
            _check(rest, "rest", q.dtype, dev, 3)
            if rest.shape != q.shape:
                raise ValueError("rest must have q's shape")
            _apart(rest, "rest", q, k, v, out, lse)
        st = load().csa_prompt_attend(ctypes.byref(p), out.data_ptr(), None if rest is None else rest.data_ptr(),
                                      lse.data_ptr(), fill, launch.handle)
        if st != 0:
            _raise(st)
        launch.used(q, k, v, cu_q, cu_k, out, lse, rest)
    if given:
        changed(*given)
    return out, lse


def csa_prompt_attend_bwd(q, k, v, out, lse, grad, cu_q, sm_scale: float, *, cu_k=None, window=None, rest=None,
                          grad_lse=None, stream=None):
    """The gradient of csa_prompt_attend: out, lse and rest are the forward's, grad
    (and grad_lse) those of out (and of lse); returns contiguous (dq, dk, dv), 0 for
    rows of no sequence."""
    import torch
    p, dev = _describe(q, k, v, cu_q, cu_k, sm_scale, window)
    T, H, _ = q.shape
    gt, gh = _rows(grad, "grad", q, dev)
    if grad.shape != q.shape:
        raise ValueError("grad must have q's shape")
    _check(out, "out", q.dtype, dev, 3)
    _check(lse, "lse", torch.float32, dev, 2)
    if out.shape != q.shape or tuple(lse.shape) != (T, H):
        raise ValueError("out and lse must be the forward's")
    if rest is not None:
        _check(rest, "rest", q.dtype, dev, 3)
        if rest.shape != q.shape:
            raise ValueError("rest must be the forward's")
    if grad_lse is not None:
        _check(grad_lse, "grad_lse", torch.float32, dev, 2)
        if grad_lse.shape != lse.shape:
            raise ValueError("grad_lse must have lse's shape")
    with on_device(dev, stream) as launch:
        dq, dk, dv = (torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v))
        st = load().csa_prompt_attend_bwd(
            ctypes.byref(p), out.data_ptr(), None if rest is None else rest.data_ptr(), lse.data_ptr(), grad.data_ptr(), gt, gh,
            None if grad_lse is None else grad_lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), launch.handle)
        if st != 0:
            _raise(st)
        launch.used(q, k, v, cu_q, cu_k, out, lse, rest, grad, grad_lse, dq, dk, dv)
    return dq, dk, dv
