"""Python binding of include/csa_prompt.h (argument marshalling only): causal
attention over packed sequences, and its gradient."""
from __future__ import annotations

import struct

from .binding import _check, _check_detail, _raise, load
from .launch import _span, changed, on_device

FILL_OUT, FILL_LSE = 1, 2

# csa_prompt_t: five pointers, two counts and six strides, six numbers, the scale
_pack = struct.Struct("@5P8q6if4x").pack


class _Types:
    """torch's types, looked up once."""

    def __getattr__(self, name):
        import torch
        self.i32, self.f32 = torch.int32, torch.float32
        self.codes = {torch.bfloat16: 0, torch.float16: 1}  # CSA_BF16, CSA_FP16
        self.contiguous = {"memory_format": torch.contiguous_format}
        self.empty, self.empty_like = torch.empty, torch.empty_like
        return self.__dict__[name]


_types = _Types()


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
    """(the C description, the device) of a call. Reading attributes is most of the
    host's time: each is read once, and the checks that name a fault run where there
    is one."""
    try:
        dt, dev, i32 = q.dtype, q.get_device(), _types.i32
        code = _types.codes.get(dt)
        (T, H, D), (qt, qh, q1), ks, (kt, kh, k1), (vt, vh, v1), (n,) = (q.shape, q.stride(), k.shape, k.stride(),
                                                                         v.stride(), cu_q.shape)
        N, KV, cols = ks
        fine = (code is not None and dev >= 0 and k.dtype is dt and v.dtype is dt and k.get_device() == dev
                and v.get_device() == dev and q1 == k1 == v1 == 1 and cols == D and v.shape == ks and KV > 0 and H > 0
                and H % KV == 0 and n > 1 and cu_q.dtype is i32 and cu_q.get_device() == dev and cu_q.is_contiguous()
                and (N == T if cu_k is None else
                     cu_k.dtype is i32 and cu_k.get_device() == dev and cu_k.is_contiguous() and tuple(cu_k.shape) == (n,))
                and (window is None or window >= 1))
    except (AttributeError, ValueError, TypeError):
        fine = False
    if not fine:
        _refuse(q, k, v, cu_q, cu_k, window)
        (T, H, D), (qt, qh, _), (N, KV, _), (kt, kh, _), (vt, vh, _) = q.shape, q.stride(), k.shape, k.stride(), v.stride()
        code, dev, n = _types.codes[q.dtype], q.get_device(), cu_q.shape[0]
    # a window of 2^31 tokens and more is none: a sequence has fewer
    return _pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), 0 if cu_k is None else cu_k.data_ptr(), T, N, qt,
                 qh, kt, kh, vt, vh, n - 1, H, KV, D, code, 0 if window is None or window >= 2 ** 31 else window,
                 sm_scale), dev


def _refuse(q, k, v, cu_q, cu_k, window):
    """Names what a call's tensors are not; returns where they are unusual but fine."""
    import torch
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    code = _types.codes.get(q.dtype)
    if code is None:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    dev = q.get_device()
    if dev < 0:
        _check_detail(q, "q", q.dtype, 0, 3)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _rows(t, name, q, dev)
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    T, H, _ = q.shape
    N, KV, _ = k.shape
    if KV < 1 or H < 1 or H % KV != 0:
        raise ValueError("q's heads must be a multiple of k's")
    _check(cu_q, "cu_q", torch.int32, dev, 1)
    n = cu_q.shape[0]
    if n < 2:
        raise ValueError("cu_q must be [num_seqs + 1]")
    if cu_k is not None:
        _check(cu_k, "cu_k", torch.int32, dev, 1)
        if cu_k.shape[0] != n:
            raise ValueError("cu_k must be as long as cu_q")
    elif N != T:
        raise ValueError("without cu_k, k must have q's tokens")
    if window is not None and window < 1:
        raise ValueError("window must be at least 1, or None for all keys")


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
    Lists that pass the tensors leave the queries of those sequences without keys.

    Rows of no sequence (a static capacity's) are 0, and -inf in lse, in tensors
    that the call makes, and left as they were in those that it is given. rest (of
    out's shape) takes what out's rounding left off, for the gradient. Not recorded
    by autograd: autograd.prompt_attend is.
    """
    p, dev = _describe(q, k, v, cu_q, cu_k, sm_scale, window)
    T, H, _ = q.shape
    fill, given = 0, [t for t in (out, lse, rest) if t is not None]
    with on_device(dev, stream) as launch:
        if out is None:
            out = _types.empty_like(q, **_types.contiguous)
            fill |= FILL_OUT
        else:
            _check(out, "out", q.dtype, dev, 3)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
            _apart(out, "out", q, k, v)
        if lse is None:
            lse = _types.empty((T, H), dtype=_types.f32, device=dev)
            fill |= FILL_LSE
        else:
            _check(lse, "lse", _types.f32, dev, 2)
            if tuple(lse.shape) != (T, H):
                raise ValueError("lse must be [tokens, heads]")
            _apart(lse, "lse", q, k, v, out)
        if rest is not None:
            _check(rest, "rest", q.dtype, dev, 3)
            if rest.shape != q.shape:
                raise ValueError("rest must have q's shape")
            _apart(rest, "rest", q, k, v, out, lse)
        st = load().csa_prompt_attend(p, out.data_ptr(), None if rest is None else rest.data_ptr(),
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
    p, dev = _describe(q, k, v, cu_q, cu_k, sm_scale, window)
    T, H, _ = q.shape
    gt, gh = _rows(grad, "grad", q, dev)
    if grad.shape != q.shape:
        raise ValueError("grad must have q's shape")
    _check(out, "out", q.dtype, dev, 3)
    _check(lse, "lse", _types.f32, dev, 2)
    if out.shape != q.shape or tuple(lse.shape) != (T, H):
        raise ValueError("out and lse must be the forward's")
    if rest is not None:
        _check(rest, "rest", q.dtype, dev, 3)
        if rest.shape != q.shape:
            raise ValueError("rest must be the forward's")
    if grad_lse is not None:
        _check(grad_lse, "grad_lse", _types.f32, dev, 2)
        if grad_lse.shape != lse.shape:
            raise ValueError("grad_lse must have lse's shape")
    with on_device(dev, stream) as launch:
        dq, dk, dv = (_types.empty_like(t, **_types.contiguous) for t in (q, k, v))
        st = load().csa_prompt_attend_bwd(
            p, out.data_ptr(), None if rest is None else rest.data_ptr(), lse.data_ptr(), grad.data_ptr(), gt, gh,
            None if grad_lse is None else grad_lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), launch.handle)
        if st != 0:
            _raise(st)
        launch.used(q, k, v, cu_q, cu_k, out, lse, rest, grad, grad_lse, dq, dk, dv)
    return dq, dk, dv
