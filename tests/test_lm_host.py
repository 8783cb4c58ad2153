"""Host-side checks of csa_rope.h and csa_cache.h (no GPU needed): arguments are
refused before anything is launched, the binding refuses wrong tensors, the
frequency tables, and the tests' own references."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import cache_ref
import gated_softmax_kv_gb300 as gsk
from gated_softmax_kv_gb300 import binding
from gated_softmax_kv_gb300.cache import _Cache

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# Well-aligned addresses that are never dereferenced: every call below is
# refused, or has nothing to do, before any CUDA call.
A = 0x10000
NULL, ALIGN, UNSUPPORTED, RANGE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    gsk.build()
    return binding.load()


def rope(lib, **kw):
    a = dict(x=A, y=2 * A, freqs=A, positions=A, bits=32, cu=None, nseq=0, ratio=1, tokens=0, heads=2,
             d=64, xt=128, xh=64, yt=128, yh=64, rope=32, offset=0, layout=0, dtype=0, amplitude=1.0,
             transpose=0)
    a.update(kw)
    return lib.csa_rope(a["x"], a["y"], a["freqs"], a["positions"], a["bits"], a["cu"], a["nseq"],
                        a["ratio"], a["tokens"], a["heads"], a["d"], a["xt"], a["xh"], a["yt"],
                        a["yh"], a["rope"], a["offset"], a["layout"], a["dtype"], a["amplitude"],
                        a["transpose"], None)


def test_rope_refusals(lib):
    assert rope(lib) == 0                                   # no tokens: valid, nothing launched
    assert rope(lib, positions=None, cu=A, nseq=1) == 0
    for bad in (dict(dtype=3), dict(dtype=-1), dict(layout=2), dict(rope=0), dict(rope=31),
                dict(rope=66), dict(offset=-2), dict(offset=34), dict(bits=16), dict(d=0)):
        assert rope(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(tokens=-1), dict(heads=0), dict(xt=-1), dict(yh=-64), dict(tokens=4, yt=0),
                dict(tokens=4, yh=32), dict(tokens=4, yt=64), dict(tokens=1 << 59),
                dict(tokens=1 << 40, xt=1 << 40), dict(positions=None, cu=A, nseq=0),
                dict(positions=None, cu=A, nseq=1, ratio=0), dict(x=A, y=A, xt=256, tokens=4)):
        assert rope(lib, **bad) == RANGE, bad
    for bad in (dict(freqs=None), dict(positions=None), dict(tokens=4, x=None), dict(tokens=4, y=None)):
        assert rope(lib, **bad) == NULL, bad
    for bad in (dict(x=A + 1), dict(y=A + 3), dict(x=A + 2, dtype=2), dict(freqs=A + 4),
                dict(positions=A + 2), dict(positions=A + 4, bits=64),
                dict(positions=None, cu=A + 2, nseq=1)):
        assert rope(lib, **bad) == ALIGN, bad


def cache_of(**kw):
    a = dict(data=A, scales=A, num_pages=8, num_heads=2, page_size=64, block=16, head_dim=128)
    a.update(kw)
    return _Cache(a["data"], a["scales"], a["num_pages"], a["num_heads"], a["page_size"], a["block"],
                  a["head_dim"])


BAD_CACHES = [(dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
              (dict(head_dim=1024), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
              (dict(page_size=8), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
              (dict(block=0), UNSUPPORTED), (dict(block=24), UNSUPPORTED), (dict(block=128), UNSUPPORTED),
              (dict(num_heads=0), UNSUPPORTED), (dict(num_heads=1025), UNSUPPORTED),
              (dict(num_pages=0), RANGE), (dict(num_pages=(1 << 24) + 1), RANGE), (dict(data=None), NULL),
              (dict(scales=None), NULL), (dict(data=A + 8), ALIGN), (dict(scales=A + 2), ALIGN)]


def append(lib, cache=None, **kw):
    a = dict(rows=A, dtype=0, n=0, rs=256, hs=128, table=A, nseq=1, width=4, lens=A, cu=A)
    a.update(kw)
    c = cache if cache is not None else cache_of()
    return lib.csa_cache_append(ctypes.byref(c), a["rows"], a["dtype"], a["n"], a["rs"], a["hs"],
                                a["table"], a["nseq"], a["width"], a["lens"], a["cu"], None)


def attend(lib, cache=None, **kw):
    a = dict(q=A, dtype=0, tokens=0, heads=4, qt=512, qh=128, kv=1, shared=0, table=A, nseq=1, width=4,
             lens=A, cu=A, visible=None, out=A, lse=A)
    a.update(kw)
    c = cache if cache is not None else cache_of()
    return lib.csa_cache_attend(ctypes.byref(c), a["q"], a["dtype"], a["tokens"], a["heads"], a["qt"],
                                a["qh"], a["kv"], a["shared"], 1.0, a["table"], a["nseq"], a["width"],
                                a["lens"], a["cu"], a["visible"], a["out"], a["lse"], None)


def reserve(lib, cache=None, **kw):
    a = dict(table=A, lens=A, refs=A, nseq=4, width=4, seqs=A, rows=A, n=0, status=A)
    a.update(kw)
    c = cache if cache is not None else cache_of()
    return lib.csa_cache_reserve(ctypes.byref(c), a["table"], a["lens"], a["refs"], a["nseq"],
                                 a["width"], a["seqs"], a["rows"], a["n"], a["status"], None)


@pytest.mark.parametrize("call", [append, attend, reserve])
def test_cache_envelope(lib, call):
    assert call(lib) == 0
    for kw, want in BAD_CACHES:
        assert call(lib, cache=cache_of(**kw)) == want, kw
    for d in (64, 128, 256, 512):
        for page in (16, 32, 64, 128, 256):
            for block in (1, 2, 16, page):
                assert call(lib, cache=cache_of(head_dim=d, page_size=page, block=block)) == 0


def test_append_refusals(lib):
    assert append(lib, rows=None) == 0                      # nothing to append
    assert append(lib, dtype=3) == UNSUPPORTED
    for bad in (dict(nseq=0), dict(nseq=262145), dict(width=0), dict(n=-1), dict(n=1 << 31), dict(rs=-8),
                dict(hs=-8), dict(rs=1 << 57), dict(hs=1 << 56)):
        assert append(lib, **bad) == RANGE, bad
    for bad in (dict(table=None), dict(lens=None), dict(cu=None), dict(n=4, rows=None)):
        assert append(lib, **bad) == NULL, bad
    for bad in (dict(rows=A + 8), dict(rs=4), dict(hs=12), dict(rs=2, dtype=2), dict(table=A + 2),
                dict(lens=A + 1), dict(cu=A + 2)):
        assert append(lib, **bad) == ALIGN, bad


def test_attend_refusals(lib):
    assert attend(lib, q=None, out=None, lse=None) == 0     # no tokens
    for bad in (dict(dtype=2), dict(kv=0), dict(kv=3, heads=6), dict(kv=2), dict(heads=0),
                dict(kv=2, heads=3, shared=1), dict(heads=65537)):
        assert attend(lib, **bad) == UNSUPPORTED, bad
    assert attend(lib, kv=2, shared=1) == 0
    for bad in (dict(nseq=0), dict(nseq=262145), dict(width=0), dict(tokens=-1), dict(tokens=1 << 30),
                dict(qt=-8), dict(qh=-8), dict(qt=1 << 57), dict(qh=1 << 56)):
        assert attend(lib, **bad) == RANGE, bad
    for bad in (dict(table=None), dict(lens=None), dict(cu=None), dict(tokens=1, q=None),
                dict(tokens=1, out=None)):
        assert attend(lib, **bad) == NULL, bad
    for bad in (dict(q=A + 8), dict(out=A + 8), dict(qt=4), dict(qh=2), dict(table=A + 2),
                dict(lens=A + 2), dict(cu=A + 2), dict(visible=A + 2), dict(lse=A + 2)):
        assert attend(lib, **bad) == ALIGN, bad


def test_page_call_refusals(lib):
    c = ctypes.byref(cache_of())
    copy = lib.csa_cache_copy_pages
    assert copy(c, None, None, 0, None) == 0
    assert copy(c, A, A, -1, None) == RANGE
    assert copy(c, None, A, 1, None) == NULL and copy(c, A, None, 1, None) == NULL
    assert copy(c, A + 2, A, 1, None) == ALIGN
    assert copy(None, A, A, 1, None) == NULL
    for kw, want in BAD_CACHES:
        assert copy(ctypes.byref(cache_of(**kw)), A, A, 1, None) == want

    def fork(table=A, lens=A, refs=A, nseq=4, width=4, pages=8, page=64, p=A, ch=A, n=0, status=A):
        return lib.csa_cache_fork(table, lens, refs, nseq, width, pages, page, p, ch, n, status, None)

    def free(table=A, lens=A, refs=A, nseq=4, width=4, pages=8, seqs=A, n=0):
        return lib.csa_cache_free(table, lens, refs, nseq, width, pages, seqs, n, None)

    def compact(table=A, refs=A, nseq=4, width=4, live=None, cache=c):
        return lib.csa_cache_compact(cache, table, refs, nseq, width, live, None)

    assert fork() == 0 and free() == 0
    assert fork(page=48) == UNSUPPORTED
    for f in (fork, free):
        for bad in (dict(nseq=0), dict(nseq=262145), dict(width=0), dict(pages=0), dict(n=-1)):
            assert f(**bad) == RANGE, bad
        for bad in (dict(table=None), dict(lens=None), dict(refs=None)):
            assert f(**bad) == NULL, bad
        for bad in (dict(table=A + 2), dict(lens=A + 1), dict(refs=A + 2)):
            assert f(**bad) == ALIGN, bad
    assert fork(n=1, p=None) == NULL and fork(n=1, ch=None) == NULL and fork(status=None) == NULL
    assert fork(status=A + 2) == ALIGN and fork(p=A + 2) == ALIGN
    assert free(n=1, seqs=None) == NULL and free(seqs=A + 2) == ALIGN
    for bad in (dict(nseq=0), dict(width=0)):
        assert compact(**bad) == RANGE and reserve(lib, **bad) == RANGE
    assert compact(table=None) == NULL and compact(refs=None) == NULL and compact(cache=None) == NULL
    assert compact(live=A + 2) == ALIGN
    assert reserve(lib, n=-1) == RANGE
    for bad in (dict(table=None), dict(lens=None), dict(refs=None), dict(n=1, seqs=None),
                dict(n=1, rows=None), dict(status=None)):
        assert reserve(lib, **bad) == NULL, bad
    for bad in (dict(table=A + 2), dict(seqs=A + 2), dict(rows=A + 2), dict(status=A + 2)):
        assert reserve(lib, **bad) == ALIGN, bad


def test_sizes_past_the_limits(lib):
    """Table rows wider than 2^31 rows need and lists longer than there can be sequences."""
    c, wide, long = ctypes.byref(cache_of()), (1 << 27) + 1, 262145
    assert append(lib, width=1 << 27) == 0 and append(lib, width=wide) == RANGE
    assert attend(lib, width=1 << 27) == 0 and attend(lib, width=wide) == RANGE
    assert reserve(lib, width=wide) == RANGE and reserve(lib, n=long) == RANGE
    for width, n in ((wide, 0), (4, long), ((1 << 31) - 1, 1)):
        assert lib.csa_cache_fork(A, A, A, 4, width, 8, 64, A, A, n, A, None) == RANGE
        assert lib.csa_cache_free(A, A, A, 4, width, 8, A, n, None) == RANGE
    assert lib.csa_cache_compact(c, A, A, 4, wide, None, None) == RANGE


def test_headers_compile_as_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    from gated_softmax_kv_gb300 import nvbuild
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(nvbuild.nvcc())), "include")
    src = tmp_path / "h.c"
    src.write_text('#include "csa_cache.h"\n#include "csa_rope.h"\n'
                   'int main(void) { csa_cache_t c; c.block = 1; return (int)sizeof(c) != 40 || c.block != 1; }\n')
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", cuda_inc, str(src), "-o", str(tmp_path / "h")], check=True)
    assert subprocess.run([str(tmp_path / "h")]).returncode == 0
    assert ctypes.sizeof(_Cache) == 40


def test_binding_refuses_wrong_tensors():
    f = torch.zeros(4, dtype=torch.float64)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        gsk.csa_rope([1.0], f, pos)
    with pytest.raises(TypeError):
        gsk.csa_rope(torch.zeros(3, 8, dtype=torch.float64), f, pos)
    with pytest.raises(ValueError):
        gsk.csa_rope(torch.zeros(8), f, pos)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_rope(torch.zeros(3, 8), f, pos)
    c8 = torch.zeros(2, 1, 16, 64).to(torch.float8_e4m3fn)
    sc = torch.ones(2, 1, 1)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    cu = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_cache_attend(q, c8, sc, t, n, cu, 1, 1.0, shared=True)
    with pytest.raises(TypeError):
        gsk.csa_cache_attend(q, c8.view(torch.uint8), sc, t, n, cu, 1, 1.0, shared=True)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_cache_append(q, c8, sc, t, n, cu)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_cache_fork(t, n, n, n, n, 16, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_cache_free(t, n, n, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_cache_compact(c8, sc, t, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_cache_copy_pages(c8, sc, n, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gsk.csa_cache_reserve(c8, sc, t, n, n, n, n, n)


def test_rope_freqs():
    f, a = gsk.csa_rope_freqs(64, device="cpu")
    assert f.dtype == torch.float64 and a == 1.0
    want = np.array([10000.0 ** (-2 * i / 64) for i in range(32)])
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-15)
    lin, a = gsk.csa_rope_freqs(64, scaling="linear", factor=8.0, device="cpu")
    np.testing.assert_allclose(lin.numpy(), want / 8, rtol=1e-15)
    assert a == 1.0
    ntk, a = gsk.csa_rope_freqs(64, scaling="ntk", factor=8.0, device="cpu")
    assert ntk[0] == 1.0 and a == 1.0
    np.testing.assert_allclose(float(ntk[-1]), want[-1] / 8, rtol=1e-12)
    y, a = gsk.csa_rope_freqs(64, scaling="yarn", factor=16.0, original_positions=4096, device="cpu")
    assert a == 0.1 * math.log(16.0) + 1.0
    turns = 4096 * want / (2 * math.pi)
    ratio = y.numpy() / want
    assert np.all(np.diff(ratio) <= 1e-15)
    np.testing.assert_allclose(ratio[turns > 40], 1.0, rtol=1e-15)      # fast pairs left alone
    np.testing.assert_allclose(ratio[turns < 0.7], 1 / 16, rtol=1e-12)  # slow pairs interpolated
    for bad in (dict(rope_dim=7), dict(rope_dim=0), dict(rope_dim=8, base=1.0),
                dict(rope_dim=8, scaling="other"), dict(rope_dim=8, factor=0.5),
                dict(rope_dim=8, scaling="yarn", original_positions=0),
                dict(rope_dim=8, scaling="yarn", beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            gsk.csa_rope_freqs(device="cpu", **bad)


def test_reference_quantiser_is_torchs():
    """The tests' own e4m3 against torch's conversion, every bf16 value within +-448."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[x.float().abs() <= 448].float()
    want = x.to(torch.float8_e4m3fn)
    got = cache_ref.quantise(x.double().numpy())
    np.testing.assert_array_equal(got, want.view(torch.uint8).numpy())
    back = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(back, cache_ref.TABLE)
    for amax in (0.0, 1e-40, 2.0 ** -112, 1.0, 447.9, 448.0, 448.01, 3.3e38):
        k = cache_ref.scale_exp(amax)
        assert amax <= 448 * 2.0 ** k and (k == -120 or amax > 448 * 2.0 ** (k - 1))
