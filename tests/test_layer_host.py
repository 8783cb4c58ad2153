"""Host-side checks of csa_norm_rope.h and csa_prompt.h (no GPU needed): arguments
are refused before anything is launched, the binding refuses wrong tensors, and the
tests' own gradients against differences."""
import ctypes

import numpy as np
import pytest

import layer_ref
import gated_softmax_kv_gb300 as gsk
from gated_softmax_kv_gb300 import binding, norm_rope, prompt

torch = pytest.importorskip("torch")

# Well-aligned addresses that are never dereferenced: every call below is refused, or
# has nothing to do, before any CUDA call.
A = 0x10000
NULL, ALIGN, UNSUPPORTED, RANGE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    gsk.build()
    return binding.load()


def side(**kw):
    a = dict(x=A, weight=A, grad=A, y=2 * A, dweight=A, xt=128, xh=64, gt=128, gh=64, yt=128, yh=64, heads=2)
    a.update(kw)
    return norm_rope._side(*(0 if v is None else v for v in a.values()))


def norm(lib, bwd=False, q=None, k=None, **kw):
    a = dict(freqs=A, positions=A, cu=0, tokens=0, bits=32, nseq=0, ratio=1, d=64, rope=32, offset=0, layout=0, dtype=0,
             weight_dtype=0, amplitude=1.0, eps=1e-6)
    a.update(kw)
    fn = lib.csa_norm_rope_bwd if bwd else lib.csa_norm_rope
    return fn(norm_rope._how(*(0 if v is None else v for v in a.values())), side() if q is None else q, k, None)


def test_norm_refusals(lib):
    assert norm(lib) == 0 and norm(lib, k=side()) == 0      # no tokens: valid, nothing launched
    assert norm(lib, positions=None, cu=A, nseq=1) == 0
    assert lib.csa_norm_rope(None, side(), None, None) == NULL and lib.csa_norm_rope(norm_rope._how(*[0] * 14, 0.0), None, None, None) == NULL
    for bad in (dict(dtype=3), dict(weight_dtype=1), dict(layout=2), dict(rope=0), dict(rope=31), dict(rope=66), dict(offset=-2),
                dict(offset=34), dict(bits=16), dict(d=0), dict(d=1025, rope=2)):
        assert norm(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(tokens=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(tokens=1 << 59),
                dict(positions=None, cu=A, nseq=0), dict(positions=None, cu=A, nseq=1, ratio=0)):
        assert norm(lib, **bad) == RANGE, bad
    for which in ("q", "k"):
        for bad in (dict(heads=0), dict(xt=-1), dict(yh=-64), dict(yt=0), dict(yh=32), dict(yt=64), dict(xt=1 << 60),
                    dict(x=A, y=A, xt=256)):
            assert norm(lib, tokens=4, **{which: side(**bad)}) == RANGE, bad
        for bad in (dict(weight=None), dict(x=None), dict(y=None)):
            assert norm(lib, tokens=4, **{which: side(**bad)}) == NULL, bad
        for bad in (dict(x=A + 1), dict(y=2 * A + 3), dict(weight=A + 1)):
            assert norm(lib, **{which: side(**bad)}) == ALIGN, bad
        for bad, want in ((dict(dweight=None), NULL), (dict(grad=None), NULL), (dict(gt=-1), RANGE), (dict(grad=A + 1), ALIGN),
                          (dict(dweight=A + 1), ALIGN), (dict(grad=2 * A, gt=64), RANGE)):
            assert norm(lib, bwd=True, tokens=4, **{which: side(**bad)}) == want, bad
    for bad in (dict(freqs=None), dict(positions=None)):
        assert norm(lib, **bad) == NULL, bad
    for bad in (dict(freqs=A + 4), dict(positions=A + 2), dict(positions=A + 4, bits=64), dict(positions=None, cu=A + 2, nseq=1)):
        assert norm(lib, **bad) == ALIGN, bad


def pack(**kw):
    a = dict(q=A, k=A, v=A, cu_q=A, cu_k=0, num_q=4, num_k=4, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64, nseq=1, heads=4,
             kv_heads=2, d=64, dtype=0, window=0, scale=0.125)
    a.update(kw)
    return prompt._pack(*(0 if v is None else v for v in a.values()))


def attend(lib, out=A, rest=None, lse=A, fill=0, **kw):
    return lib.csa_prompt_attend(pack(**kw), out, rest, lse, fill, None)


def back(lib, out=A, rest=None, lse=A, grad=A, gt=256, gh=64, glse=None, dq=A, dk=A, dv=A, **kw):
    return lib.csa_prompt_attend_bwd(pack(**kw), out, rest, lse, grad, gt, gh, glse, dq, dk, dv, None)


@pytest.mark.parametrize("call", [attend, back])
def test_prompt_refusals(lib, call):
    for bad in (dict(dtype=2), dict(dtype=-1), dict(d=0), dict(d=4), dict(d=132), dict(d=136), dict(heads=0), dict(heads=3),
                dict(kv_heads=0), dict(kv_heads=3), dict(heads=258), dict(heads=1 << 17, kv_heads=1 << 16)):
        assert call(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(num_q=-1), dict(num_k=-1), dict(nseq=0), dict(nseq=262145), dict(window=-1), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(qt=0), dict(qh=-64), dict(kt=0),
                dict(vh=0), dict(qt=1 << 40), dict(num_q=1 << 31, cu_k=A), dict(num_q=1 << 30, cu_k=A, heads=4),
                dict(num_k=5), dict(nseq=262144, kv_heads=65535, heads=65535)):
        assert call(lib, **bad) == RANGE, bad
    for bad in (dict(qt=260), dict(kh=4), dict(vt=6), dict(q=A + 8), dict(k=A + 2), dict(v=A + 4), dict(cu_q=A + 2), dict(cu_k=A + 1),
                dict(out=A + 8), dict(rest=A + 2), dict(lse=A + 2)):
        assert call(lib, **bad) == ALIGN, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(cu_q=None), dict(out=None), dict(lse=None)):
        assert call(lib, **bad) == NULL, bad


def test_prompt_refusals_of_one_direction(lib):
    assert attend(lib, num_q=0, num_k=0, q=None, k=None, v=None, out=None, lse=None) == 0
    assert back(lib, num_q=0, num_k=0, q=None, k=None, v=None, out=None, lse=None, grad=None, dq=None, dk=None, dv=None) == 0
    assert attend(lib, fill=4) == UNSUPPORTED and lib.csa_prompt_attend(None, A, None, A, 0, None) == NULL
    for bad, want in ((dict(grad=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL),
                      (dict(grad=A + 8), ALIGN), (dict(gh=4), ALIGN), (dict(gt=0), RANGE), (dict(dq=A + 4), ALIGN),
                      (dict(dk=A + 8), ALIGN), (dict(dv=A + 2), ALIGN), (dict(glse=A + 2), ALIGN)):
        assert back(lib, **bad) == want, bad


def test_bindings_refuse_tensors_of_the_host():
    x, w = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    f, pos, cu = torch.ones(16, dtype=torch.float64), torch.arange(4), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gsk.csa_norm_rope(x, w, f, pos)
    with pytest.raises(ValueError, match="CUDA"):
        gsk.csa_prompt_attend(x, x, x, cu, 0.1)
    with pytest.raises(TypeError):
        gsk.csa_norm_rope(x.double(), w, f, pos)
    with pytest.raises(TypeError):
        gsk.csa_prompt_attend(x.float(), x, x, cu, 0.1)
    for bad in (None, 3, [1.0]):
        with pytest.raises(TypeError):
            gsk.csa_prompt_attend(bad, x, x, cu, 0.1)
        with pytest.raises(TypeError):
            gsk.csa_norm_rope(bad, w, f, pos)


def test_structures_as_the_compiler_lays_them_out(tmp_path):
    """The packed descriptions have the C structures' sizes and last fields' places."""
    import os
    import shutil
    import struct
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None or not os.path.exists("/usr/local/cuda/include/cuda_runtime_api.h"):
        pytest.skip("no C compiler or CUDA headers")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "csa_norm_rope.h"\n#include "csa_prompt.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(csa_prompt_t), sizeof(csa_norm_side_t),\n'
                   "sizeof(csa_norm_rope_t), offsetof(csa_prompt_t, sm_scale), offsetof(csa_norm_side_t, heads),\n"
                   "offsetof(csa_norm_rope_t, eps)); return 0; }\n")
    subprocess.run([cc, "-I" + os.path.join(root, "include"), "-I/usr/local/cuda/include", str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert got[:3] == [len(prompt._pack(*[0] * 19, 1.0)), len(norm_rope._side(*[0] * 12)), len(norm_rope._how(*[0] * 13, 1.0, 2.0))]
    assert struct.unpack_from("@f", prompt._pack(*[0] * 19, 1.5), got[3]) == (1.5,)
    assert struct.unpack_from("@i", norm_rope._side(*[0] * 11, 7), got[4]) == (7,)
    assert struct.unpack_from("@f", norm_rope._how(*[0] * 13, 1.0, 2.5), got[5]) == (2.5,)


def slope(f, h):
    return (f(h) - f(-h)) / (2 * h)


def test_the_references_gradients_are_those_of_the_references():
    """Central differences in 64 bits: off by h^2 / 6 of a third derivative, of which
    three quarters go from h to h / 2, and 2^-53 of the terms over h."""
    r = np.random.default_rng(1)
    x, w, g, f, pos = r.normal(size=(3, 2, 16)), r.normal(size=16), r.normal(size=(3, 2, 16)), np.array([1.0, 0.3, 0.01]), [0, 5, 9]
    kw = dict(offset=4, layout="half", amplitude=1.3)
    dx, _, dw, _ = layer_ref.norm_rope_grad(x, w, g, f, pos, 1e-6, **kw)
    d, e = r.normal(size=x.shape), r.normal(size=w.shape)
    loss = lambda h: (layer_ref.norm_rope(x + h * d, w + h * e, f, pos, 1e-6, **kw)[0] * g).sum()  # noqa: E731
    a, b = slope(loss, 1e-4), slope(loss, 5e-5)
    assert abs((dx * d).sum() + (dw * e).sum() - b) <= abs(a - b) + 1e-9
    for cu_q, cu_k, window in (([0, 3, 8], [0, 3, 8], None), ([0, 3, 8], [0, 9, 11], 4)):
        q, k, v = r.normal(size=(8, 4, 8)), r.normal(size=(cu_k[-1], 2, 8)), r.normal(size=(cu_k[-1], 2, 8))
        g, gl = r.normal(size=q.shape), r.normal(size=q.shape[:2])
        out, lse, parts = layer_ref.prompt(q, k, v, cu_q, cu_k, 0.4, window)
        gl = np.where(np.isfinite(lse), gl, 0.0)
        grads, _ = layer_ref.prompt_grad(q, k, v, cu_q, cu_k, 0.4, parts, out, g, gl)
        d = [r.normal(size=t.shape) for t in (q, k, v)]

        def loss(h):
            o, l, _ = layer_ref.prompt(*(t + h * s for t, s in zip((q, k, v), d)), cu_q, cu_k, 0.4, window)
            return (o * g).sum() + (np.where(np.isfinite(l), l, 0.0) * gl).sum()

        a, b = slope(loss, 1e-4), slope(loss, 5e-5)
        assert abs(sum((t * s).sum() for t, s in zip(grads, d)) - b) <= abs(a - b) + 1e-9
