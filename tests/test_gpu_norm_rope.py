"""Norms of queries and keys with the rotary positions (csa_norm_rope, its
gradient, autograd.norm_rope) against the 64-bit formulas; layer_ref.py derives
the tolerances."""
import math

import numpy as np
import pytest

import layer_ref

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


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, name=""):
    assert got.shape == want.shape
    t = layer_ref.rounded(want, tol, torch.finfo(got.dtype).eps, 2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    g = np64(got)
    bad = ~(np.abs(g - want) <= t)
    assert not bad.any(), (name, np.argwhere(bad)[:3], g[bad][:3], want[bad][:3], t[bad][:3])


def make(shape, dtype, seed=0, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DTYPES[dtype]).cuda()


def weight(D, dtype, seed):
    return (1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(seed))).to(DTYPES[dtype]).cuda()


def check(gsk, q, wq, k, wk, f, pos, gq, gk, eps=1e-6, **kw):
    fn, p = np64(f), pos.cpu().numpy()
    y, z = gsk.csa_norm_rope(q, wq, f, pos, k=k, k_weight=wk, eps=eps, **kw)
    made = gsk.csa_norm_rope_bwd(q, wq, f, gq, pos, k=k, k_weight=wk, k_grad=gk, eps=eps, **kw)
    for x, w, g, o, dx, dw in ((q, wq, gq, y, made[0], made[1]), (k, wk, gk, z, made[2], made[3])):
        if x is None:
            assert o is None and dx is None and dw is None
            continue
        want, tol = layer_ref.norm_rope(np64(x), np64(w), fn, p, eps, **kw)
        close(o, want, tol, "y")
        a, ta, b, tb = layer_ref.norm_rope_grad(np64(x), np64(w), np64(g), fn, p, eps, **kw)
        close(dx, a, ta, "dx")
        close(dw, b, tb, "dw")


# tokens, heads of q, of k (0: none), columns, turned, offset
SHAPES = [(1, 1, 0, 512, 64, 448), (1, 64, 8, 128, 128, 0), (16, 64, 8, 128, 128, 0), (7, 3, 2, 64, 32, 32), (33, 5, 1, 96, 96, 0),
          (130, 2, 1, 256, 64, 64), (3, 1, 1, 1024, 64, 960), (40, 3, 3, 40, 16, 8), (2500, 4, 1, 128, 64, 0),       # vectors
          (9, 3, 2, 10, 6, 2), (4, 1, 0, 7, 2, 5), (3, 2, 1, 66, 34, 31), (1, 1, 1, 2, 2, 0), (5, 2, 1, 130, 130, 0)]  # any


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("T,H,K,D,n,off", SHAPES)
def test_formulas(gsk, T, H, K, D, n, off, dtype, wtype, layout):
    f, _ = gsk.csa_rope_freqs(n)
    pos = torch.randint(0, 1_000_000, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int64 if T % 2 else torch.int32).cuda()
    # tokens of different sizes
    size = torch.exp2(torch.arange(T) % 7 - 3.0).view(T, 1, 1).cuda()
    q, k = ((make((T, h, D), "fp32", T + h) * size).to(DTYPES[dtype]) if h else None for h in (H, K))
    check(gsk, q, weight(D, wtype, 1), k, weight(D, wtype, 2) if K else None, f, pos, make((T, H, D), dtype, 3),
          make((T, K, D), dtype, 4) if K else None, offset=off, layout=layout, amplitude=1.25)


def test_positions_of_packed_tokens_and_rows(gsk):
    cu = [0, 5, 5, 6, 19]
    T = 23                                                  # four rows behind the last sequence
    for ratio in (1, 4):
        pos = torch.zeros(T, dtype=torch.int64)
        for a, b in zip(cu, cu[1:]):
            pos[a:b] = torch.arange(b - a) * ratio
        x, w = make((T, 64), "bf16", 1), weight(64, "fp32", 2)
        f, a = gsk.csa_rope_freqs(32, scaling="yarn", factor=4.0)
        kw = dict(cu_seqlens_comp=torch.tensor(cu, dtype=torch.int32, device="cuda"), ratio=ratio, offset=32, amplitude=a)
        y, none = gsk.csa_norm_rope(x, w, f, **kw)
        assert none is None and y.shape == x.shape
        want, tol = layer_ref.norm_rope(np64(x)[:, None], np64(w), np64(f), pos.numpy(), 1e-6, offset=32, amplitude=a)
        close(y[:, None], want, tol)
        dx, dw, _, _ = gsk.csa_norm_rope_bwd(x, w, f, y, **kw)
        a, ta, b, tb = layer_ref.norm_rope_grad(np64(x)[:, None], np64(w), np64(y)[:, None], np64(f), pos.numpy(), 1e-6,
                                                offset=32, amplitude=a)
        close(dx[:, None], a, ta)
        close(dw, b, tb)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_views_strides_and_in_place(gsk, layout):
    T, H, K, D, n = 13, 4, 2, 64, 32
    f, _ = gsk.csa_rope_freqs(n)
    pos = torch.arange(T, device="cuda") * 3
    wq, wk = weight(D, "bf16", 1), weight(D, "bf16", 2)
    base = make((T, H + 2 * K, D + 16), "bf16", 5)
    for c in (0, 8, 3):                                     # aligned, aligned, odd
        q, k = base[:, :H, c: c + D], base[:, H: H + K, c: c + D]
        check(gsk, q, wq, k, wk, f, pos, make((H, T, D), "bf16", 6).transpose(0, 1), make((1, K, D), "bf16", 7).expand(T, K, D),
              offset=16, layout=layout)
        y, z = gsk.csa_norm_rope(q, wq, f, pos, k=k, k_weight=wk, offset=16, layout=layout)
        hold = base.clone()
        qo, ko = hold[:, :H, c: c + D], hold[:, H: H + K, c: c + D]
        a, b = gsk.csa_norm_rope(qo, wq, f, pos, k=ko, k_weight=wk, offset=16, layout=layout, out=qo, k_out=ko)
        assert a is qo and b is ko and torch.equal(a, y) and torch.equal(b, z)
        rest = hold.clone()
        rest[:, : H + K, c: c + D] = base[:, : H + K, c: c + D]
        assert torch.equal(rest, base)                      # nothing else is touched
    x = make((T, 1, D), "bf16", 8).expand(T, H, D)          # one head for all
    check(gsk, x, wq, None, None, f, pos, make((T, H, D), "bf16", 9), None, offset=16, layout=layout)


def test_zero_rows_infinities_and_nan_stay_in_their_head(gsk):
    f, _ = gsk.csa_rope_freqs(32)
    pos = torch.tensor([1, 2, 3], device="cuda")
    w = weight(64, "fp32", 1)
    x = make((3, 2, 64), "fp32")
    x[0, 0] = 0.0
    x[1, 1, 5], x[2, 0, 40] = math.nan, math.inf
    y, _ = gsk.csa_norm_rope(x, w, f, pos)
    assert (y[0, 0] == 0).all()
    fine = torch.isfinite(y).all(-1)
    assert fine.tolist() == [[True, True], [True, False], [False, True]]
    dx, dw, _, _ = gsk.csa_norm_rope_bwd(x, w, f, torch.ones_like(x), pos)
    assert torch.isfinite(dx).all(-1).tolist() == [[True, True], [True, False], [False, True]] and not torch.isfinite(dw).any()
    z = torch.zeros(2, 1, 64, device="cuda")                # eps 0: 0 / 0, as the formula says
    assert torch.isnan(gsk.csa_norm_rope(z, w, f, pos[:2], eps=0.0)[0]).all()


def test_gradients_through_autograd_and_against_differences(gsk):
    from gated_softmax_kv_gb300 import autograd
    T, H, K, D = 6, 3, 2, 64
    f, _ = gsk.csa_rope_freqs(32)
    pos = torch.arange(T, device="cuda") * 11
    for layout in ("interleaved", "half"):
        kw = dict(offset=32, layout=layout, amplitude=1.5)
        leaves = [make((T, H, D), "fp32", 1), weight(D, "fp32", 2), make((T, K, D), "fp32", 3), weight(D, "fp32", 4)]
        leaves = [t.requires_grad_() for t in leaves]
        g = [make((T, H, D), "fp32", 5), make((T, K, D), "fp32", 6)]
        y, z = autograd.norm_rope(leaves[0], leaves[1], f, pos, k=leaves[2], k_weight=leaves[3], **kw)
        got = torch.autograd.grad([y, z], leaves, g)
        fn, p = np64(f), pos.cpu().numpy()
        for i in (0, 2):
            x, w, gg = np64(leaves[i]), np64(leaves[i + 1]), np64(g[i // 2])
            a, ta, b, tb = layer_ref.norm_rope_grad(x, w, gg, fn, p, 1e-6, **kw)
            close(got[i], a, ta)
            close(got[i + 1], b, tb)

            def loss(dx, dw):
                return (layer_ref.norm_rope(x + dx, w + dw, fn, p, 1e-6, **kw)[0] * gg).sum()

            d, e = np64(make((T, x.shape[1], D), "fp32", 7 + i)), np64(make((D,), "fp32", 8 + i))

            def slope(h):
                return (loss(h * d, h * e) - loss(-h * d, -h * e)) / (2 * h)

            # a central difference is off by h^2 / 6 of a third derivative: from h to h / 2 three quarters of it
            # go, so what is left is below the change; its rounding is 2^-53 of the loss's terms over h
            want, before = slope(5e-5), slope(1e-4)
            mag = np.abs(layer_ref.norm_rope(x, w, fn, p, 1e-6, **kw)[0] * gg).sum()
            tol = abs(want - before) + 2.0 ** -50 * mag / 5e-5
            tol += (layer_ref.rounded(a, ta, 2.0 ** -23) * np.abs(d)).sum() + (layer_ref.rounded(b, tb, 2.0 ** -23) * np.abs(e)).sum()
            # got's own distance from the formula is within ta and tb (checked above)
            have = (np64(got[i]) * d).sum() + (np64(got[i + 1]) * e).sum()
            assert abs(have - want) <= tol
    x = make((T, H, D), "bf16", 9).requires_grad_()         # a sum's broadcast gradient, no keys
    w = weight(D, "bf16", 1).requires_grad_()
    y, none = autograd.norm_rope(x, w, f, pos)
    assert none is None
    y.sum().backward()
    a, ta, b, tb = layer_ref.norm_rope_grad(np64(x), np64(w), np.ones(x.shape), fn, p, 1e-6)
    close(x.grad, a, ta)
    close(w.grad, b, tb)


def test_many_tokens_sum_the_same_way_each_time(gsk):
    T, D = 5001, 128
    f, _ = gsk.csa_rope_freqs(128)
    x, k, w = make((T, 3, D), "bf16", 1), make((T, 1, D), "bf16", 2), weight(D, "fp32", 3)
    pos = torch.arange(T, device="cuda")
    runs = [gsk.csa_norm_rope_bwd(x, w, f, x, pos, k=k, k_weight=w, k_grad=k, layout="half") for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_empty(gsk):
    f, _ = gsk.csa_rope_freqs(32)
    w = weight(64, "fp32", 1)
    x = make((4, 2, 64), "bf16")[:0]
    pos = torch.arange(4, device="cuda")[:0]
    y, z = gsk.csa_norm_rope(x, w, f, pos, k=x, k_weight=w)
    assert y.shape == z.shape == (0, 2, 64)
    dx, dw, dk, dkw = gsk.csa_norm_rope_bwd(x, w, f, x, pos, k=x, k_weight=w, k_grad=x)
    assert dx.shape == dk.shape == (0, 2, 64) and (dw == 0).all() and (dkw == 0).all()


def test_refusals(gsk):
    f, _ = gsk.csa_rope_freqs(32)
    pos = torch.arange(4, device="cuda")
    x, w = make((4, 2, 64), "bf16"), weight(64, "bf16", 1)
    for bad in (dict(layout="other"), dict(positions=pos[:3]), dict(positions=None), dict(out=x[:3]), dict(k_weight=w),
                dict(cu_seqlens_comp=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(k=x[:3], k_weight=w),
                dict(k=x[..., :32], k_weight=w), dict(k=make((4, 1, 64), "bf16"), k_weight=w[:32])):
        with pytest.raises(ValueError):
            gsk.csa_norm_rope(x, w, f, **{**dict(positions=pos), **bad})
    for bad in (dict(q=x.double()), dict(q_weight=w.half()), dict(k=x.float(), k_weight=w), dict(k=x, k_weight=w.float()),
                dict(freqs=f.float()), dict(positions=pos.float()), dict(out=x.float()), dict(k=x)):
        with pytest.raises(TypeError):
            gsk.csa_norm_rope(**{**dict(q=x, q_weight=w, freqs=f, positions=pos), **bad})
    for bad in (dict(offset=33), dict(eps=-1.0), dict(eps=math.nan), dict(cu_seqlens_comp=pos[:2].int(), positions=None, ratio=0)):
        with pytest.raises(gsk.CsaError):
            gsk.csa_norm_rope(x, w, f, **{**dict(positions=pos), **bad})
    with pytest.raises(gsk.CsaError):                       # wider than the kernels' heads
        gsk.csa_norm_rope(make((1, 1, 1040), "bf16"), weight(1040, "bf16", 1), f, pos[:1])
    big = make((5, 2, 64), "bf16")
    with pytest.raises(ValueError, match="overlaps"):
        gsk.csa_norm_rope(big[:4], w, f, pos, out=big[1:])
    with pytest.raises(ValueError, match="overlaps"):       # one output twice
        gsk.csa_norm_rope(x, w, f, pos, k=x.clone(), k_weight=w, out=big[:4], k_out=big[:4])
    with pytest.raises(ValueError, match="overlaps"):       # the keys' input is the queries' output
        gsk.csa_norm_rope(x, w, f, pos, k=big[:4], k_weight=w, out=big[:4])
    e = make((1, 2, 64), "bf16").expand(4, 2, 64)
    with pytest.raises(gsk.CsaError):
        gsk.csa_norm_rope(e, w, f, pos, out=e)              # output elements not distinct
    with pytest.raises(TypeError):
        gsk.csa_norm_rope_bwd(x, w, f, x[:3], pos)


def test_capture_other_stream_and_in_place_for_autograd(gsk):
    from gated_softmax_kv_gb300 import autograd
    f, _ = gsk.csa_rope_freqs(64)
    T = 100
    x, k, w = make((T, 2, 64), "bf16", 1).requires_grad_(), make((T, 1, 64), "bf16", 2), weight(64, "fp32", 3)
    g = [make((T, 2, 64), "bf16", 4), make((T, 1, 64), "bf16", 5)]
    pos = torch.arange(T, device="cuda")

    def step():
        y, z = autograd.norm_rope(x, w, f, pos, k=k, k_weight=w)
        return y, z, torch.autograd.grad([y], x, [g[0]])[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]     # two graphs share the pool's workspace
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(step())
    with torch.no_grad():
        x.copy_(make((T, 2, 64), "bf16", 6))
        pos.mul_(7)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want, tol = layer_ref.norm_rope(np64(x), np64(w), np64(f), pos.cpu().numpy(), 1e-6)
    a, ta, _, _ = layer_ref.norm_rope_grad(np64(x), np64(w), np64(g[0]), np64(f), pos.cpu().numpy(), 1e-6)
    for y, z, dx in outs:
        close(y, want, tol)
        close(dx, a, ta)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, _ = gsk.csa_norm_rope(x.detach(), w, f, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y2, outs[0][0])
    h = torch.randn(4, 2, 64, device="cuda")
    one = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
    total = (one * h).sum()
    gsk.csa_norm_rope(h, w, f, pos[:4], out=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        total.backward()


def test_long_and_wide(gsk):
    """Strides past 2^31 bytes."""
    T, D = 3, 64
    hold = torch.empty(2 * (2 ** 30 + 512) + 64, dtype=torch.bfloat16, device="cuda")
    x = hold.as_strided((T, 1, D), (2 ** 30 + 512, D, 1))
    x.copy_(make((T, 1, D), "bf16"))
    f, _ = gsk.csa_rope_freqs(64)
    pos, w = torch.tensor([1, 2, 3], device="cuda"), weight(D, "fp32", 1)
    want, tol = layer_ref.norm_rope(np64(x), np64(w), np64(f), pos.cpu().numpy(), 1e-6)
    gsk.csa_norm_rope(x, w, f, pos, out=x)
    close(x, want, tol)
