"""Python binding of include/csa_cache.h (argument marshalling only): the
paged 8-bit cache of compressed rows, its attention and its pages.

The cache is two tensors: `cache` float8_e4m3fn [num_pages, num_heads,
page_size, head_dim] and `scales` fp32 [num_pages, num_heads, page_size /
block]. Sequences are `page_table` int32 [num_seqs, max_pages] (-1: no page),
`seq_lens` int32 [num_seqs] and, for the page functions, `page_refs` int32
[num_pages]. An empty cache is zeros, a table of -1, and zeros.
"""
from __future__ import annotations

import ctypes

from .binding import _check, _check_detail, _raise, load
from .launch import changed, on_device, output_overlaps

CACHE_STATUS = {1: "a sequence index outside the table", 2: "an index twice, or both child and parent",
                4: "a child that holds rows or pages", 8: "fewer free pages than needed",
                16: "more rows than a table row has room for", 32: "a held page outside the pool"}


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("block", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class _Types:
    """torch's types, looked up once."""

    def __getattr__(self, name):
        import torch
        self.e4m3, self.f32, self.i32 = torch.float8_e4m3fn, torch.float32, torch.int32
        self.queries = {torch.bfloat16: 0, torch.float16: 1}
        self.rows = {**self.queries, torch.float32: 2}
        self.contiguous = {"memory_format": torch.contiguous_format}
        self.empty, self.empty_like = torch.empty, torch.empty_like
        return self.__dict__[name]


_types = _Types()


def _fine(cache, scales, rows, codes, dev, *ints) -> bool:
    """Whether a cache, packed rows and int32 tensors are of the right types and
    layouts and on the device. The checks that name the fault run where not:
    reading attributes is most of the host's time of a call."""
    i32 = _types.i32
    for t in ints:
        if t.dtype is not i32 or t.get_device() != dev or not t.is_contiguous():
            return False
    return (dev >= 0 and cache.dtype is _types.e4m3 and cache.is_contiguous()
            and scales.dtype is _types.f32 and scales.get_device() == dev and scales.is_contiguous()
            and rows.dtype in codes and rows.get_device() == dev)


def _cache(cache, scales):
    """(the C description, the device) of a cache."""
    import torch
    dev = cache.get_device() if isinstance(cache, torch.Tensor) else -1
    if dev < 0:
        _check_detail(cache, "cache", torch.float8_e4m3fn, 0, 4)
    _check(cache, "cache", torch.float8_e4m3fn, dev, 4)
    _check(scales, "scales", torch.float32, dev, 3)
    p, h, page, d = cache.shape
    blocks = scales.shape[2]
    if scales.shape[0] != p or scales.shape[1] != h or blocks < 1 or page % blocks != 0:
        raise ValueError("scales must be [num_pages, num_heads, page_size / block]")
    return _Cache(cache.data_ptr(), scales.data_ptr(), p, h, page, page // blocks, d), dev


def _tables(page_table, seq_lens, dev):
    import torch
    _check(page_table, "page_table", torch.int32, dev, 2)
    _check(seq_lens, "seq_lens", torch.int32, dev, 1)
    n, width = page_table.shape
    if seq_lens.shape[0] != n or n < 1 or width < 1:
        raise ValueError("page_table must be [num_seqs, max_pages] and seq_lens [num_seqs]")
    return n, width


def _list(a, b, names, dev):
    import torch
    _check(a, names[0], torch.int32, dev, 1)
    _check(b, names[1], torch.int32, dev, 1)
    if a.shape != b.shape:
        raise ValueError(f"{names[0]} and {names[1]} must be equally long")
    return a.shape[0]


def _word(status, dev, name="status"):
    import torch
    _check(status, name, torch.int32, dev, 1)
    if status.shape[0] != 1:
        raise ValueError(f"{name} must be one int32 word")


def _rows(t, name, dtypes, dev):
    """A packed [tokens, heads, head_dim] input whose last dimension is contiguous."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if t.dim() != 3 or t.shape[1] < 1 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with a contiguous last dimension")


def csa_cache_append(rows, cache, scales, page_table, seq_lens, cu_rows, stream=None) -> None:
    """Quantises rows [num_rows, num_heads, head_dim] (bf16, fp16 or fp32) into
    the cache: sequence s gets rows cu_rows[s] .. cu_rows[s + 1] - 1 behind its
    seq_lens[s] rows. seq_lens is not changed: add the lengths afterwards. Not
    recorded by autograd."""
    try:
        dev = cache.get_device()
        (pages, heads, page, D), (sp, sh, blocks) = cache.shape, scales.shape
        (n, width), (lens,), (cu,) = page_table.shape, seq_lens.shape, cu_rows.shape
        (T, H, cols), (rs, hs, last) = rows.shape, rows.stride()
        fine = (sp == pages and sh == heads == H and cols == D and blocks >= 1 and page % blocks == 0
                and n == lens == cu - 1 and n >= 1 and width >= 1 and heads >= 1 and last == 1
                and _fine(cache, scales, rows, _types.rows, dev, page_table, seq_lens, cu_rows))
    except (AttributeError, ValueError):
        fine = False
    if fine:
        c = _Cache(cache.data_ptr(), scales.data_ptr(), pages, heads, page, page // blocks, D)
    else:
        c, dev = _cache(cache, scales)
        n, width = _tables(page_table, seq_lens, dev)
        _check(cu_rows, "cu_rows", _types.i32, dev, 1)
        _rows(rows, "rows", tuple(_types.rows), dev)
        if cu_rows.shape[0] != n + 1:
            raise ValueError("cu_rows must be [num_seqs + 1]")
        if rows.shape[1] != c.num_heads or rows.shape[2] != c.head_dim:
            raise ValueError("rows must be [num_rows, num_heads, head_dim] of the cache")
        (T, H, _), (rs, hs, _) = rows.shape, rows.stride()
    # the stride of a dimension of one element is never stepped: 0
    if T <= 1:
        rs = 0
    if H <= 1:
        hs = 0
    with on_device(dev, stream) as launch:
        st = load().csa_cache_append(ctypes.byref(c), rows.data_ptr(), _types.rows[rows.dtype],
                                     T, rs, hs, page_table.data_ptr(), n, width,
                                     seq_lens.data_ptr(), cu_rows.data_ptr(), launch.handle)
        if st != 0:
            _raise(st)
        launch.used(rows, cache, scales, page_table, seq_lens, cu_rows)


def csa_cache_attend(q, cache, scales, page_table, seq_lens, cu_q, kv_heads: int, sm_scale: float,
                     shared: bool = False, visible=None, out=None, lse=None, stream=None):
    """Attention of packed queries q [tokens, heads, head_dim] (bf16 or fp16)
    over the cache; returns (out, lse). kv_heads cache heads are keys; with
    shared=True they are the values too, else the next kv_heads heads are.
    visible (int32 [tokens]): rows that each query sees, all where None. lse
    (natural logarithm, fp32 [tokens, heads]) lets the result be merged with
    attention over other rows. Tokens at or behind cu_q[-1] are not written.
    Not recorded by autograd: out and lse carry no gradient to q, whether or not
    it requires one (the 8-bit rows have none to take)."""
    try:
        dev = cache.get_device()
        (pages, heads, page, D), (sp, sh, blocks) = cache.shape, scales.shape
        (n, width), (lens,), (cu,) = page_table.shape, seq_lens.shape, cu_q.shape
        (T, H, cols), (qt, qh, last) = q.shape, q.stride()
        fine = (sp == pages and sh == heads and cols == D and blocks >= 1 and page % blocks == 0
                and n == lens == cu - 1 and n >= 1 and width >= 1 and H >= 1 and last == 1
                and _fine(cache, scales, q, _types.queries, dev, page_table, seq_lens, cu_q))
    except (AttributeError, ValueError):
        fine = False
    if fine:
        c = _Cache(cache.data_ptr(), scales.data_ptr(), pages, heads, page, page // blocks, D)
    else:
        c, dev = _cache(cache, scales)
        n, width = _tables(page_table, seq_lens, dev)
        _check(cu_q, "cu_q", _types.i32, dev, 1)
        _rows(q, "q", tuple(_types.queries), dev)
        if cu_q.shape[0] != n + 1:
            raise ValueError("cu_q must be [num_seqs + 1]")
        (T, H, D), (qt, qh, _) = q.shape, q.stride()
        if D != c.head_dim:
            raise ValueError("q must be [tokens, heads, head_dim] with the cache's head_dim")
    if visible is not None:
        _check(visible, "visible", _types.i32, dev, 1)
        if visible.shape[0] != T:
            raise ValueError("visible must be [tokens]")
    # the stride of a dimension of one element is never stepped: 0
    if T <= 1:
        qt = 0
    if H <= 1:
        qh = 0
    given = [t for t in (out, lse) if t is not None]
    with on_device(dev, stream) as launch:
        if out is None:
            out = _types.empty_like(q, **_types.contiguous)
        else:
            _check(out, "out", q.dtype, dev, 3)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
            if out.data_ptr() == q.data_ptr() and T > 0 or output_overlaps(out, q):
                raise ValueError("out overlaps q")
        if lse is None:
            lse = _types.empty((T, H), dtype=_types.f32, device=dev)
        else:
            _check(lse, "lse", _types.f32, dev, 2)
            if tuple(lse.shape) != (T, H):
                raise ValueError("lse must be [tokens, heads]")
        st = load().csa_cache_attend(
            ctypes.byref(c), q.data_ptr(), _types.queries[q.dtype], T, H, qt, qh, kv_heads,
            int(shared), sm_scale, page_table.data_ptr(), n, width, seq_lens.data_ptr(),
            cu_q.data_ptr(), None if visible is None or T == 0 else visible.data_ptr(),
            out.data_ptr(), lse.data_ptr() if T else None, launch.handle)
        if st != 0:
            _raise(st)
        launch.used(q, cache, scales, page_table, seq_lens, cu_q, visible, out, lse)
    if given:
        changed(*given)
    return out, lse


def csa_cache_copy_pages(cache, scales, src, dst, stream=None) -> None:
    """Copies pages src[i] -> dst[i] (int32 [n]); destinations distinct, none a source."""
    c, dev = _cache(cache, scales)
    n = _list(src, dst, ("src", "dst"), dev)
    with on_device(dev, stream) as launch:
        st = load().csa_cache_copy_pages(ctypes.byref(c), src.data_ptr(), dst.data_ptr(), n,
                                         launch.handle)
        if st != 0:
            _raise(st)
        launch.used(cache, scales, src, dst)


def csa_cache_fork(page_table, seq_lens, page_refs, parents, children, page_size: int, status,
                   stream=None) -> None:
    """Makes the empty sequence children[i] an equal of parents[i] that shares
    its pages. Bits of CACHE_STATUS go to the int32 word `status`."""
    import torch
    dev = page_table.get_device() if isinstance(page_table, torch.Tensor) else -1
    if dev < 0:
        _check_detail(page_table, "page_table", torch.int32, 0, 2)
    n, width = _tables(page_table, seq_lens, dev)
    _check(page_refs, "page_refs", torch.int32, dev, 1)
    k = _list(parents, children, ("parents", "children"), dev)
    _word(status, dev)
    with on_device(dev, stream) as launch:
        st = load().csa_cache_fork(page_table.data_ptr(), seq_lens.data_ptr(), page_refs.data_ptr(),
                                   n, width, page_refs.shape[0], page_size, parents.data_ptr(),
                                   children.data_ptr(), k, status.data_ptr(), launch.handle)
        if st != 0:
            _raise(st)
        launch.used(page_table, seq_lens, page_refs, parents, children, status)


def csa_cache_reserve(cache, scales, page_table, seq_lens, page_refs, seqs, rows, status,
                      stream=None) -> None:
    """Makes room for rows[i] more rows of sequence seqs[i]: new pages, and
    copies of shared pages that will be written. All or nothing; bits of
    CACHE_STATUS go to the int32 word `status`."""
    import torch
    c, dev = _cache(cache, scales)
    n, width = _tables(page_table, seq_lens, dev)
    _check(page_refs, "page_refs", torch.int32, dev, 1)
    if page_refs.shape[0] != c.num_pages:
        raise ValueError("page_refs must be [num_pages]")
    k = _list(seqs, rows, ("seqs", "rows"), dev)
    _word(status, dev)
    with on_device(dev, stream) as launch:
        st = load().csa_cache_reserve(ctypes.byref(c), page_table.data_ptr(), seq_lens.data_ptr(),
                                      page_refs.data_ptr(), n, width, seqs.data_ptr(),
                                      rows.data_ptr(), k, status.data_ptr(), launch.handle)
        if st != 0:
            _raise(st)
        launch.used(cache, scales, page_table, seq_lens, page_refs, seqs, rows, status)


def csa_cache_free(page_table, seq_lens, page_refs, seqs, stream=None) -> None:
    """Ends the sequences seqs: their pages are given back."""
    import torch
    dev = page_table.get_device() if isinstance(page_table, torch.Tensor) else -1
    if dev < 0:
        _check_detail(page_table, "page_table", torch.int32, 0, 2)
    n, width = _tables(page_table, seq_lens, dev)
    _check(page_refs, "page_refs", torch.int32, dev, 1)
    _check(seqs, "seqs", torch.int32, dev, 1)
    with on_device(dev, stream) as launch:
        st = load().csa_cache_free(page_table.data_ptr(), seq_lens.data_ptr(), page_refs.data_ptr(),
                                   n, width, page_refs.shape[0], seqs.data_ptr(), seqs.shape[0],
                                   launch.handle)
        if st != 0:
            _raise(st)
        launch.used(page_table, seq_lens, page_refs, seqs)


def csa_cache_compact(cache, scales, page_table, page_refs, live=None, stream=None) -> None:
    """Moves the held pages to the pool's front; live (one int32 word) gets
    their number."""
    import torch
    c, dev = _cache(cache, scales)
    _check(page_table, "page_table", torch.int32, dev, 2)
    _check(page_refs, "page_refs", torch.int32, dev, 1)
    n, width = page_table.shape
    if page_refs.shape[0] != c.num_pages:
        raise ValueError("page_refs must be [num_pages]")
    if live is not None:
        _word(live, dev, "live")
    with on_device(dev, stream) as launch:
        st = load().csa_cache_compact(ctypes.byref(c), page_table.data_ptr(), page_refs.data_ptr(),
                                      n, width, None if live is None else live.data_ptr(),
                                      launch.handle)
        if st != 0:
            _raise(st)
        launch.used(cache, scales, page_table, page_refs, live)
