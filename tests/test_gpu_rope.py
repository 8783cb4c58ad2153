"""Rotary positions (csa_rope, autograd.rope) against the 64-bit turn.

Tolerance of an element: the angle is off by at most 2^-32 turns (fixed point)
and pi 2^-24 (the fraction of a turn as fp32), sincospif by 2 units in the
last place, the amplitude's product, the product and the sum by one rounding
each: (pi + 2 + 3) 2^-24 < 2^-20.9 of amplitude (|a| + |b|); then one rounding
to the type, eps / 2, and half a step of fp16's subnormals.
"""
import math
from fractions import Fraction

import numpy as np
import pytest

import cache_ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def close(got, want, mag):
    eps = torch.finfo(got.dtype).eps
    g = got.detach().double().cpu().numpy().reshape(want.shape)
    tol = 2.0 ** -20.9 * mag + eps / 2 * (np.abs(want) + 2.0 ** -20.9 * mag)
    tol = tol + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], g[bad][:3], want[bad][:3])


def make(T, H, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H, D), generator=g).to(DTYPES[dtype]).cuda()


def ref(x, freqs, positions, **kw):
    return cache_ref.rope(x.detach().double().cpu().numpy(), freqs.cpu().numpy(),
                          np.asarray(positions.cpu() if torch.is_tensor(positions) else positions),
                          kw.get("offset", 0), kw.get("layout", "interleaved"), kw.get("amplitude", 1.0),
                          kw.get("transpose", False))


SHAPES = [(1, 1, 64, 64, 0), (1, 64, 512, 64, 448), (7, 3, 128, 32, 96), (33, 5, 64, 32, 16), (130, 1, 512, 64, 448),
          (5, 17, 128, 128, 0), (300, 2, 24, 16, 8),      # vectors
          (9, 3, 10, 6, 2), (4, 1, 7, 2, 5), (3, 2, 66, 34, 31), (1, 1, 2, 2, 0)]   # any


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,H,D,n,off", SHAPES)
def test_turn_and_transpose(gsk, T, H, D, n, off, dtype, layout):
    x = make(T, H, D, dtype, T + D)
    f, _ = gsk.csa_rope_freqs(n)
    pos = torch.randint(0, 1_000_000, (T,), generator=torch.Generator().manual_seed(T)).to(
        torch.int64 if T % 2 else torch.int32).cuda()
    for tr in (False, True):
        kw = dict(offset=off, layout=layout, amplitude=1.25, transpose=tr)
        y = gsk.csa_rope(x, f, pos, **kw)
        want, mag = ref(x, f, pos, **kw)
        close(y, want, mag)
        keep = [c for c in range(D) if not off <= c < off + n]
        assert torch.equal(y[..., keep], x[..., keep])
    z = x.clone()
    assert gsk.csa_rope(z, f, pos, out=z, **kw) is z        # in place, the same bits
    assert torch.equal(z.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("pos", [0, 1, 7, 2 ** 20 + 1, 2 ** 31 - 1, -5, -2 ** 31])
def test_far_and_negative_positions(gsk, pos):
    """Angles of far positions, up to 2^32.6 rad."""
    f = torch.tensor([1.0, 0.5, 2.0 ** -10, 2.0 ** -31, 0.0, 3.0, -0.25, 2.0 ** -62], dtype=torch.float64,
                     device="cuda")
    x = make(1, 2, 16, "fp32", 3)
    y = gsk.csa_rope(x, f, torch.tensor([pos], device="cuda"))
    # the angle modulo a turn in rational arithmetic (pi to 50 digits), then the plain turn by it
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")
    turns = [(Fraction(pos) * Fraction(float(v)) / two_pi) % 1 for v in f.cpu()]
    ang = np.array([float(t) for t in turns]) * 2 * math.pi
    want, mag = cache_ref.rope(x.double().cpu().numpy(), ang, [1.0], 0, "interleaved", 1.0, False)
    close(y, want, mag)


def test_positions_of_compressed_rows(gsk):
    cu = [0, 5, 5, 6, 19]
    T, ratio = 23, 4                                        # four padding rows
    x = make(T, 1, 64, "bf16", 1).squeeze(1)                # [tokens, head_dim]
    f, a = gsk.csa_rope_freqs(32, scaling="yarn", factor=4.0)
    y = gsk.csa_rope(x, f, cu_seqlens_comp=torch.tensor(cu, dtype=torch.int32, device="cuda"), ratio=ratio,
                     offset=32, amplitude=a)
    pos = [0] * T
    for s in range(4):
        for t in range(cu[s], cu[s + 1]):
            pos[t] = (t - cu[s]) * ratio
    want, mag = ref(x[:, None], f, pos, offset=32, amplitude=a)
    close(y[:, None], want, mag)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_strides_and_alignments(gsk, layout):
    T, H, D, n = 13, 4, 64, 32
    f, _ = gsk.csa_rope_freqs(n)
    pos = torch.arange(T, device="cuda") * 3
    base = make(T, H + 2, D + 16, "bf16", 5)
    views = [base[:, 1:1 + H, :D], base[:, 1:1 + H, 8:8 + D], base[:, :H, 3:3 + D],   # aligned, aligned, odd
             make(H, T, D, "bf16", 6).transpose(0, 1), make(1, H, D, "bf16", 7).expand(T, H, D),
             make(T, 1, D, "bf16", 8).expand(T, H, D)]
    for x in views:
        want, mag = ref(x, f, pos, offset=16, layout=layout)
        close(gsk.csa_rope(x, f, pos, offset=16, layout=layout), want, mag)
        hold = torch.full((T, H + 1, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        out = hold[:, :H, 8:]
        close(gsk.csa_rope(x, f, pos, offset=16, layout=layout, out=out), want, mag)
        assert (hold[:, H] == 7).all() and (hold[:, :, :8] == 7).all()
    z = base.clone()                                        # in place on a slice
    gsk.csa_rope(z[:, 1:1 + H, 8:8 + D], f, pos, out=z[:, 1:1 + H, 8:8 + D], layout=layout)
    want, mag = ref(base[:, 1:1 + H, 8:8 + D], f, pos, layout=layout)
    close(z[:, 1:1 + H, 8:8 + D], want, mag)
    z[:, 1:1 + H, 8:8 + D] = base[:, 1:1 + H, 8:8 + D]
    assert torch.equal(z, base)


def test_infinities_and_nan_stay_in_their_pair(gsk):
    x = make(2, 1, 64, "fp32")
    x[0, 0, 3], x[1, 0, 10], x[1, 0, 40] = math.inf, math.nan, -math.inf
    f, _ = gsk.csa_rope_freqs(32)
    y = gsk.csa_rope(x, f, torch.tensor([1, 2], device="cuda"))
    bad = (~torch.isfinite(y)).nonzero().tolist()
    assert bad == [[0, 0, 2], [0, 0, 3], [1, 0, 10], [1, 0, 11], [1, 0, 40]]


def test_gradients(gsk):
    from gated_softmax_kv_gb300 import autograd
    T, H, D, n = 6, 2, 64, 32
    f, _ = gsk.csa_rope_freqs(n)
    pos = torch.arange(T, device="cuda") * 11
    for layout in ("interleaved", "half"):
        kw = dict(offset=32, layout=layout, amplitude=1.5)
        x = make(T, H, D, "fp32", 2).requires_grad_()
        g = make(T, H, D, "fp32", 3)
        y = autograd.rope(x, f, pos, **kw)
        (gx,) = torch.autograd.grad(y, x, g)
        want, mag = ref(g, f, pos, transpose=True, **kw)
        close(gx, want, mag)
        # against differences: the operator is linear, so (y(x + d) - y(x)) . g = gx . d
        d = make(T, H, D, "fp32", 4)
        dy, _ = ref(d, f, pos, **kw)
        lhs = (dy * g.double().cpu().numpy()).sum()
        rhs = (gx.detach().double() * d.double()).sum().item()
        # gx within 2^-20.9 mag + 2^-24 |want| of the formula's; fp64 sums are exact next to that
        tol = ((2.0 ** -20.9 * mag + 2.0 ** -23 * np.abs(want)) * np.abs(d.double().cpu().numpy())).sum()
        assert abs(lhs - rhs) <= tol
        # the gradient's own gradient is the turn again
        g2 = g.clone().requires_grad_()
        (gx2,) = torch.autograd.grad(autograd.rope(x, f, pos, **kw), x, g2, create_graph=True)
        (back,) = torch.autograd.grad(gx2, g2, d)
        want, mag = ref(d, f, pos, **kw)
        close(back, want, mag)
    # a broadcast gradient (a sum's) and a transposed one
    x = make(T, H, D, "bf16", 2).requires_grad_()
    autograd.rope(x, f, pos).sum().backward()
    want, mag = ref(torch.ones(T, H, D), f, pos, transpose=True)
    close(x.grad, want, mag)
    x.grad = None
    w = make(D, T, H, "bf16", 9).permute(1, 2, 0)
    (autograd.rope(x, f, pos) * w).sum().backward()
    want, mag = ref(w, f, pos, transpose=True)
    close(x.grad, want, mag)


def test_inverse_and_empty(gsk):
    f, _ = gsk.csa_rope_freqs(64)
    pos = torch.arange(40, device="cuda") * 1000
    x = make(40, 2, 64, "fp32")
    y = gsk.csa_rope(gsk.csa_rope(x, f, pos), f, pos, transpose=True)
    # two turns, each within 2^-20.9 (|a| + |b|) + 2^-24 |y| <= (2^-20.4 + 2^-24) of the pair's norm
    # an element, sqrt(2) of it over a pair that the second turn mixes
    norm = x.view(40, 2, 32, 2).norm(dim=-1, keepdim=True).expand(40, 2, 32, 2).reshape(40, 2, 64)
    assert ((y - x).abs() <= 2.5 * (2.0 ** -20.4 + 2.0 ** -24) * norm).all()
    e = gsk.csa_rope(x[:0], f, pos[:0])
    assert e.shape == (0, 2, 64)
    e = gsk.csa_rope(x[:0], f, cu_seqlens_comp=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert e.shape == (0, 2, 64)


def test_refusals(gsk):
    f, _ = gsk.csa_rope_freqs(32)
    pos = torch.arange(4, device="cuda")
    x = make(4, 2, 64, "bf16")
    for bad in (dict(layout="other"), dict(positions=pos[:3]), dict(positions=None), dict(out=x[:3])):
        with pytest.raises(ValueError):
            gsk.csa_rope(x, f, **{**dict(positions=pos), **bad})
    with pytest.raises(ValueError):
        gsk.csa_rope(x, f, pos, cu_seqlens_comp=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        gsk.csa_rope(x, f, pos.float())
    with pytest.raises(TypeError):
        gsk.csa_rope(x, f.float(), pos)
    with pytest.raises(ValueError):
        gsk.csa_rope(x.transpose(1, 2), f, pos)
    with pytest.raises(gsk.CsaError):
        gsk.csa_rope(x, f, pos, offset=33)
    big = make(5, 2, 64, "bf16")
    with pytest.raises(ValueError, match="overlaps"):
        gsk.csa_rope(big[:4], f, pos, out=big[1:])
    e = make(1, 2, 64, "bf16").expand(4, 2, 64)
    with pytest.raises(gsk.CsaError):
        gsk.csa_rope(e, f, pos, out=e)                      # output elements not distinct


def test_capture_other_stream_and_backward_in_a_graph(gsk):
    from gated_softmax_kv_gb300 import autograd
    f, _ = gsk.csa_rope_freqs(64)
    T = 100
    x = make(T, 2, 64, "bf16", 1).requires_grad_()
    g = make(T, 2, 64, "bf16", 2)
    pos = torch.arange(T, device="cuda")
    autograd.rope(x, f, pos).sum().backward()               # eager graphs of the leaf, gone before the capture
    x.grad = None
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(autograd.rope(x, f, pos), x, g)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        y = autograd.rope(x, f, pos)
        (gx,) = torch.autograd.grad(y, x, g)
    with torch.no_grad():
        x.copy_(make(T, 2, 64, "bf16", 5))
        g.copy_(make(T, 2, 64, "bf16", 6))
        pos.mul_(7)
    graph.replay()
    torch.cuda.synchronize()
    want, mag = ref(x, f, pos)
    close(y, want, mag)
    want, mag = ref(g, f, pos, transpose=True)
    close(gx, want, mag)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = gsk.csa_rope(x.detach(), f, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y2, y)


def test_long_and_wide(gsk):
    """Strides past 2^31 bytes."""
    T, D = 3, 64
    hold = torch.empty(2 * (2 ** 30 + 512) + 64, dtype=torch.bfloat16, device="cuda")
    x = hold.as_strided((T, 1, D), (2 ** 30 + 512, D, 1))
    x.copy_(make(T, 1, D, "bf16"))
    f, _ = gsk.csa_rope_freqs(64)
    pos = torch.tensor([1, 2, 3], device="cuda")
    want, mag = ref(x, f, pos)
    close(gsk.csa_rope(x, f, pos), want, mag)
    gsk.csa_rope(x, f, pos, out=x)
    close(x, want, mag)
