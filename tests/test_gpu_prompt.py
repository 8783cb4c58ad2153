"""Causal attention over packed sequences (csa_prompt_attend, its gradient,
autograd.prompt_attend) against the 64-bit formulas (layer_ref.py).

Tolerances, with e = eps / 2 of the type (half a step, relative) and U = 2^-24:
- z: a product's sum of up to 128 terms in fp32, which the tensor core may truncate: 128 * 2 U of
  scale * sum |q k|, bounded by scale * 128 * max|q| max|k| here as `zerr`; its exponential has that
  error, 2 ulp of its own and the rounding of z log2 e - m (|z| 2 U): `perr` relative.
- the weights are rounded to the type (e), their sum is not; sums of m terms: m * 2 U (truncation).
So |out - want| <= (e + 2 perr + 2 (m + 8) U) sum_j p_j |v_j| + e |want|; the rounding's part of a row whose
weights are fp16: below 2^-14 of the largest they lose up to 2^-25 * 2^-6 each.
- lse: perr + 2 (m + 8) U, and U |lse| roundings.
- gradients: P and dS are rounded (e each); dS = P (dP - delta) has the sums' errors in dP and delta:
  128 * 2 U of sum |g v| and the rest of out, 2^-16 of |g out| (bf16) or 2^-22 (fp16).
"""
import math

import numpy as np
import pytest

import layer_ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def sums(v):
    return np.concatenate([[0], np.cumsum(v)]).astype(int).tolist()


def make(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DTYPES[dtype]).cuda()


def inputs(nq, nk, H, KV, D, dtype, seed=0, spare=0, scale=1.5):
    """q, k, v with `spare` rows behind the last sequence."""
    T, N = sum(nq) + spare, sum(nk) + spare
    return make((T, H, D), dtype, seed, scale), make((N, KV, D), dtype, seed + 1), make((N, KV, D), dtype, seed + 2)


def errors_of(q, k, scale, dtype):
    """(e, perr): half a step, and a weight's relative error before its rounding."""
    D = q.shape[2]
    big = lambda t: np.abs(np64(t)[np.isfinite(np64(t))]).max(initial=0.0)  # noqa: E731
    # Cauchy-Schwarz on the largest rows: sum |q k| <= |q| |k|
    norm = lambda t: np.sqrt((np.nan_to_num(np64(t), nan=0, posinf=0, neginf=0) ** 2).sum(-1)).max(initial=0.0)  # noqa: E731
    z = scale * norm(q) * norm(k)
    return torch.finfo(DTYPES[dtype]).eps / 2, (2 * D + 8) * U * z + 4 * U


def check(gsk, q, k, v, cu_q, cu_k, scale, window=None, dtype="bf16", grad=True, glse=False):
    T, H, D = q.shape
    e, perr = errors_of(q, k, scale, dtype)
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    same = cu_k is None
    ck = cu_q if same else cu_k
    x, y, w = np64(q), np64(k), np64(v)
    want, wlse, parts = layer_ref.prompt(x, y, w, cu_q, ck, scale, window)
    kw = dict(cu_k=None if same else i32(cu_k), window=window)
    rest = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    out, lse = gsk.csa_prompt_attend(q, k, v, i32(cu_q), scale, rest=rest, **kw)
    m = max([b - a for a, b in zip(ck, ck[1:])] + [1])
    mag = layer_ref.prompt(x, y, np.abs(w), cu_q, ck, scale, window)[0]
    terms = 2 * (m + 8) * U
    tol = (e + 2 * perr + terms) * mag + tiny * (2.0 ** -6 * m * np.abs(w).max(initial=0) + 1)
    got, glsev = np64(out), np64(lse)
    bad = ~(np.abs(got - want) <= tol + e * (np.abs(want) + tol))
    assert not bad.any(), ("out", bad.sum(), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
    fine = np.isfinite(wlse)
    assert (np.isfinite(glsev) == fine).all() and (glsev[~fine] == -math.inf).all()
    with np.errstate(all="ignore"):
        bad = fine & ~(np.abs(glsev - wlse) <= perr + terms + 4 * U * np.abs(wlse))
    assert not bad.any(), ("lse", np.argwhere(bad)[:4], glsev[bad][:4], wlse[bad][:4])
    # out + rest: all but the weights' rounding
    exact = np64(out) + np64(rest)
    bad = ~(np.abs(exact - want) <= tol + e * e * np.abs(want) + tiny)
    assert not bad.any(), ("rest", np.argwhere(bad)[:4])
    if not grad:
        return out, lse
    g = make((T, H, D), dtype, 77)
    gl = torch.randn((T, H), generator=torch.Generator().manual_seed(78)).cuda() if glse else None
    got = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, i32(cu_q), scale, rest=rest, grad_lse=gl, **kw)
    gg, ggl = np64(g), None if gl is None else np64(gl)
    want3, mags = layer_ref.prompt_grad(x, y, w, cu_q, ck, scale, parts, want, gg, ggl)
    # the error of dS beside its own size: that of dP, delta and P, in units of P |g| |v|
    size = np.sqrt((gg ** 2).sum(-1)).max(initial=0) * np.sqrt((w ** 2).sum(-1)).max(initial=0)
    ds = (2 * D * U * 2 + e * e * 4 + 2 * (2 * perr + terms)) * size + (e + 2 * perr + terms) * size
    pk, pq = np.zeros(k.shape), np.zeros(q.shape)
    group = H // k.shape[1]
    for s in range(len(cu_q) - 1):
        a, b, c, d = cu_q[s], cu_q[s + 1], ck[s], ck[s + 1]
        for h in range(H):
            if b > a and d > c:
                p = parts[s * H + h] * layer_ref.seen(b - a, d - c, window)
                pq[a:b, h] += p @ np.abs(y[c:d, h // group])
                pk[c:d, h // group] += p.T @ np.abs(x[a:b, h])
    for name, a, b, t in (("dq", got[0], want3[0], e * 1.1 * mags[0] + ds * scale * pq),
                          ("dk", got[1], want3[1], e * 1.1 * mags[1] + ds * scale * pk),
                          ("dv", got[2], want3[2], (e * 1.1 + 2 * perr + 2 * (T * group + 8) * U) * mags[2])):
        # weights below fp32's 2^-126 are 0: each term of a sum loses at most that, times |g| |v| |k| < 2^20
        t = t + tiny * (1 + np.abs(b).max(initial=0)) + 2.0 ** -100
        r = np64(a)
        bad = ~(np.abs(r - b) <= t + e * (np.abs(b) + t))
        assert not bad.any(), (name, bad.sum(), np.argwhere(bad)[:4], r[bad][:4], b[bad][:4], t[bad][:4])
        # and as a whole: roundings are independent, so the norm of the error is well below the bound's
        n = np.linalg.norm(b)
        assert np.linalg.norm(r - b) <= 2.5 * e * n + tiny * math.sqrt(b.size) or n == 0, (name, np.linalg.norm(r - b) / n)
        if n == 0:
            assert (r == 0).all(), name
    return out, lse


# queries and keys of each sequence (None: the queries' own), heads, key heads, columns
CASES = [
    ([1], None, 1, 1, 64), ([1, 1, 1], None, 8, 2, 128), ([2, 0, 5], None, 4, 1, 64), ([127], None, 2, 2, 128),
    ([128], None, 2, 1, 128), ([129, 1, 300], None, 4, 2, 64), ([255, 257], None, 6, 2, 128), ([640], None, 3, 1, 64),
    ([513, 70], None, 16, 1, 128), ([40, 33], None, 64, 1, 64), ([300], None, 5, 1, 96), ([77, 200], None, 10, 2, 80),
    ([130], None, 7, 7, 8), ([50], None, 100, 1, 40), ([20], None, 128, 1, 128), ([200], None, 1, 1, 128),
    ([1], [1], 1, 1, 64), ([1, 1, 1], [1000, 1, 129], 8, 1, 128), ([5, 0, 64], [300, 50, 64], 4, 2, 64),
    ([3, 10], [1, 4], 4, 2, 64), ([2, 7], [0, 300], 2, 1, 128), ([100, 200], [700, 333], 12, 4, 64), ([130], [900], 8, 1, 128),
]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("nq,nk,H,KV,D", CASES)
def test_formulas(gsk, nq, nk, H, KV, D, dtype):
    q, k, v = inputs(nq, nk or nq, H, KV, D, dtype, sum(nq) + D, spare=9 if len(nq) == 2 else 0)
    check(gsk, q, k, v, sums(nq), None if nk is None else sums(nk), D ** -0.5, dtype=dtype, glse=H % 2 == 0)


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 300, 5000])
@pytest.mark.parametrize("nq,nk,H,KV,D", [([400, 3, 150], None, 4, 2, 64), ([200, 1, 5], [500, 300, 2], 8, 1, 128)])
def test_windows(gsk, nq, nk, H, KV, D, window):
    q, k, v = inputs(nq, nk or nq, H, KV, D, "bf16", window)
    check(gsk, q, k, v, sums(nq), None if nk is None else sums(nk), D ** -0.5, window=window, glse=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_large_and_small_logits(gsk, dtype):
    """References that rise by far, and logits that leave one key all the weight."""
    q, k, v = inputs([600], [600], 2, 1, 64, dtype, 5, scale=1.0)
    k = (k.float() * torch.linspace(0.1, 12, 600, device="cuda")[:, None, None]).to(k.dtype)
    check(gsk, q, k, v, [0, 600], None, 1.0, dtype=dtype)
    check(gsk, q, k.flip(0), v, [0, 600], None, 1.0, dtype=dtype)
    check(gsk, q * 0, k, v, [0, 600], None, 1.0, dtype=dtype)


def test_views_and_strides(gsk):
    nq, H, KV, D = [150, 61], 4, 2, 64
    x = make((211, H + 2 * KV, D), "bf16", 1)
    q, k, v = x[:, :H], x[:, H: H + KV], x[:, H + KV:]
    a = check(gsk, q, k, v, sums(nq), None, 0.125)
    b = gsk.csa_prompt_attend(q.contiguous(), k.contiguous(), v.contiguous(), i32(sums(nq)), 0.125)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = make((H + 1, 300, D + 8), "bf16", 2)             # heads before tokens
    q = wide[1:, :211, 8:].transpose(0, 1)
    check(gsk, q, k, v, sums(nq), None, 0.125)


@pytest.mark.parametrize("D", [64, 80, 128])
def test_results_at_16_bytes(gsk, D):
    """out, rest and every other tensor 16-byte aligned and no better."""
    def at16(shape, dtype=torch.bfloat16):
        n = math.prod(shape)
        t = torch.zeros(n + 16, dtype=dtype, device="cuda")
        t = t[8: 8 + n] if dtype is torch.bfloat16 else t[4: 4 + n]
        assert t.data_ptr() % 32 == 16
        return t.view(shape)

    q0, k0, v0 = inputs([150], [150], 4, 2, D, "bf16", 1)
    q, k, v, out, rest = at16(q0.shape), at16(k0.shape), at16(v0.shape), at16(q0.shape), at16(q0.shape)
    for a, b in ((q, q0), (k, k0), (v, v0)):
        a.copy_(b)
    lse = at16((150, 4), torch.float32)
    gsk.csa_prompt_attend(q, k, v, i32([0, 150]), 0.1, out=out, lse=lse, rest=rest)
    want = gsk.csa_prompt_attend(q0, k0, v0, i32([0, 150]), 0.1)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # the C call with gradients of that kind
    import gated_softmax_kv_gb300.prompt as p
    from gated_softmax_kv_gb300.binding import load
    cu = i32([0, 150])
    how, _ = p._describe(q, k, v, cu, None, 0.1, None)
    dq, dk, dv, g = at16(q.shape), at16(k.shape), at16(k.shape), at16(q.shape)
    g.copy_(make(q.shape, "bf16", 5))
    assert load().csa_prompt_attend_bwd(how, out.data_ptr(), rest.data_ptr(), lse.data_ptr(), g.data_ptr(), 4 * D, D, None,
                                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    back = gsk.csa_prompt_attend_bwd(q0, k0, v0, want[0], want[1], g.clone(), cu, 0.1, rest=rest.clone())
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), back))


def test_rows_of_no_sequence(gsk):
    nq, H, KV, D = [100, 30], 4, 2, 64
    q, k, v = inputs(nq, nq, H, KV, D, "bf16", 3, spare=20)
    cu = [5, 105, 135]                                      # five rows before the first, fifteen behind the last
    for t in (q, k, v):
        t[:5] = math.nan
        t[135:] = math.inf
    out, lse = gsk.csa_prompt_attend(q, k, v, i32(cu), 0.125)
    want, _ = gsk.csa_prompt_attend(q[5:135], k[5:135], v[5:135], i32([0, 100, 130]), 0.125)
    assert torch.equal(out[5:135], want)
    for r in (slice(0, 5), slice(135, 150)):
        assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
    hold, hl = torch.full_like(out, 7.0), torch.full_like(lse, 9.0)
    gsk.csa_prompt_attend(q, k, v, i32(cu), 0.125, out=hold, lse=hl)
    assert torch.equal(hold[5:135], want) and (hold[:5] == 7).all() and (hold[135:] == 7).all()
    assert (hl[:5] == 9).all() and (hl[135:] == 9).all() and torch.equal(hl[5:135], lse[5:135])
    g = make(q.shape, "bf16", 4)
    g[135:] = math.nan
    dq, dk, dv = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, i32(cu), 0.125)
    wq, wk, wv = gsk.csa_prompt_attend_bwd(q[5:135], k[5:135], v[5:135], want, lse[5:135].contiguous(), g[5:135], i32([0, 100, 130]), 0.125)
    for a, b in ((dq, wq), (dk, wk), (dv, wv)):
        assert torch.equal(a[5:135], b) and (a[:5] == 0).all() and (a[135:] == 0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_keys_that_a_query_does_not_see_take_no_part(gsk, bad):
    """A value that is not finite, in k or v, reaches the queries that see it and no other;
    so does one in a sequence's neighbour."""
    nq, H, KV, D = [200, 90], 2, 1, 64
    for name in ("k", "v"):
        for at in (0, 70, 150, 199, 230):
            q, k, v = inputs(nq, nq, H, KV, D, "bf16", at)
            want, wlse = gsk.csa_prompt_attend(q, k, v, i32(sums(nq)), 0.125, window=100)
            (k if name == "k" else v)[at, 0, 3] = bad
            out, lse = gsk.csa_prompt_attend(q, k, v, i32(sums(nq)), 0.125, window=100)
            t = torch.arange(290, device="cuda")
            sees = (t >= at) & (t < at + 100) & ((t < 200) == (at < 200))
            assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wlse[~sees])
            if name == "v":
                assert not torch.isfinite(out[sees][:, :, 3]).any() and torch.equal(lse, wlse)
                keep = [c for c in range(D) if c != 3]
                assert torch.equal(out[..., keep], want[..., keep])
            elif bad != bad:
                assert torch.isnan(out[sees]).all()


@pytest.mark.parametrize("name", ["q", "grad", "k", "v"])
def test_gradients_of_unseen_rows_take_no_part(gsk, name):
    nq, H, KV, D = [200, 90], 2, 1, 64
    for at in (1, 70, 199, 230):                            # (query 0 sees one key: no gradient, whatever grad holds)
        q, k, v = inputs(nq, nq, H, KV, D, "bf16", at)
        g = make(q.shape, "bf16", at + 5)
        args = dict(window=100)
        cu = i32(sums(nq))

        def grads():
            out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.125, **args)
            return gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.125, **args)

        want = grads()
        {"q": q, "grad": g, "k": k, "v": v}[name][at, 0, 3] = math.nan
        got = grads()
        t = torch.arange(290, device="cuda")
        same = (t < 200) == (at < 200)
        if name in ("q", "grad"):                           # keys that the query sees, and the query's own row
            qs, ks = t == at, (t <= at) & (t > at - 100) & same
        else:                                               # queries that see the key, and all that those see
            qs = (t >= at) & (t < at + 100) & same
            ks = (t > at - 100) & (t < at + 100) & same
        heads = slice(0, 1) if name in ("q", "grad") else slice(0, 2)
        assert torch.equal(got[0][~qs], want[0][~qs])
        assert torch.equal(got[1][~ks], want[1][~ks]) and torch.equal(got[2][~ks], want[2][~ks])
        assert not torch.isfinite(got[0][qs][:, heads]).all()
        assert torch.isfinite(got[0][:, 1:]).all() or name in ("k", "v")


def test_gradients_through_autograd_and_against_differences(gsk):
    from gated_softmax_kv_gb300 import autograd
    nq, H, KV, D, scale = [37, 150], 4, 2, 64, 0.125
    q, k, v = (t.requires_grad_() for t in inputs(nq, nq, H, KV, D, "bf16", 11))
    g, gl = make(q.shape, "bf16", 12), torch.randn(q.shape[:2], generator=torch.Generator().manual_seed(13)).cuda()
    cu = sums(nq)
    out, lse = autograd.prompt_attend(q, k, v, i32(cu), scale)
    got = torch.autograd.grad([out, lse], [q, k, v], [g, gl])
    x, gg, ggl = [np64(t) for t in (q, k, v)], np64(g), np64(gl)

    def loss(h, d):
        o, l, _ = layer_ref.prompt(*(a + h * b for a, b in zip(x, d)), cu, cu, scale)
        return (o * gg).sum() + (l * ggl).sum()

    e = 2.0 ** -8
    for i in range(3):
        d = [np64(make(t.shape, "bf16", 20 + j)) if i == j else np.zeros(t.shape) for j, t in enumerate((q, k, v))]

        def slope(h):
            return (loss(h, d) - loss(-h, d)) / (2 * h)

        want, before = slope(5e-5), slope(1e-4)
        # a gradient's elements are off by independent roundings of at most e (P or dS) and e (its own) of
        # terms whose norms are its own: 2.5 e of the norm, as `check` holds them to, times the direction's
        tol = abs(want - before) + 2.5 * e * np.linalg.norm(np64(got[i])) * np.linalg.norm(d[i])
        assert abs((np64(got[i]) * d[i]).sum() - want) <= tol
    # each output alone; a sum's broadcast gradient; one transposed
    (a,) = torch.autograd.grad(autograd.prompt_attend(q, k, v, i32(cu), scale)[1].sum(), q, retain_graph=False)
    b = gsk.csa_prompt_attend_bwd(q.detach(), k.detach(), v.detach(), out.detach(), lse.detach(), torch.zeros_like(q), i32(cu), scale,
                                  grad_lse=torch.ones_like(lse))
    # out's own rounding plays no part: its gradient is 0
    assert torch.equal(a, b[0])
    o = autograd.prompt_attend(q, k, v, i32(cu), scale)[0]
    a = torch.autograd.grad(o.sum(), [q, k, v], retain_graph=True)
    b = torch.autograd.grad(o, [q, k, v], torch.ones_like(o), retain_graph=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    w = make((H, D, sum(nq)), "bf16", 9).permute(2, 0, 1)
    a = torch.autograd.grad(o, [q, k, v], w, retain_graph=True)
    b = torch.autograd.grad(o, [q, k, v], w.contiguous())
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_small_gradients_in_fp16(gsk):
    """Gradients as small as a mean over many tokens makes them: dS is far below fp16's range."""
    q, k, v = inputs([500], [500], 2, 1, 64, "fp16", 1)
    g = make(q.shape, "fp16", 2)
    out, lse = gsk.csa_prompt_attend(q, k, v, i32([0, 500]), 0.125)
    one = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, i32([0, 500]), 0.125)
    # scaled by a power of two the same bits come out, until the result itself is subnormal
    small = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, (g.float() * 2.0 ** -9).half(), i32([0, 500]), 0.125)
    for a, b in zip(one, small):
        n = a.double().norm()
        # 2^-11 each from g's subnormals (below 2^-5 before the scale), the result's rounding and dS's
        assert ((b.double() * 512 - a.double()).norm() / n) <= 2.0 ** -10
    # rows of no sequence have no say in how dS is scaled
    more = [torch.cat([t, torch.full_like(t[:7], 60000.0)]) for t in (q, k, v, out, g)]
    tail = torch.cat([lse, torch.full_like(lse[:7], -math.inf)])
    got = gsk.csa_prompt_attend_bwd(*more[:4], tail, more[4], i32([0, 500]), 0.125)
    assert all(torch.equal(a[:500], b) and (a[500:] == 0).all() for a, b in zip(got, one))
    big = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, (g.float() * 64).half(), i32([0, 500]), 0.125)
    for a, b in zip(one, big):
        assert torch.isfinite(b).all() and ((b.double() / 64 - a.double()).norm() / a.double().norm()) <= 2.0 ** -10


def test_same_bits_each_time(gsk):
    q, k, v = inputs([700, 1, 333], [700, 1, 333], 8, 2, 128, "bf16", 2)
    g, cu = make(q.shape, "bf16", 3), i32([0, 700, 701, 1034])
    runs = []
    for _ in range(3):
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.1)
        runs.append((out, lse, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.1)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("nq,nk,H,KV,D,window", [
    ([1500, 9, 700], None, 8, 2, 128, None), ([900, 333], None, 6, 2, 64, None), ([1000], None, 8, 1, 64, 100),
    ([3, 1], [5000, 700], 16, 2, 128, None), ([130, 64], [2000, 64], 4, 2, 128, None)])
def test_many_launches_one_behind_the_other(gsk, nq, nk, H, KV, D, window):
    """Forward and gradient without a pause between the launches, whose CTAs take over one
    another's work: every launch gives the first one's bits."""
    q, k, v = inputs(nq, nk or nq, H, KV, D, "bf16", 5)
    g, cu, ck = make(q.shape, "bf16", 6), i32(sums(nq)), None if nk is None else i32(sums(nk))
    runs = []
    for _ in range(60):
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.1, cu_k=ck, window=window)
        runs.append((out, lse, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.1, cu_k=ck, window=window)))
    torch.cuda.synchronize()
    for i, r in enumerate(runs):
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0])), i
    assert all(torch.isfinite(t).all() for t in runs[0])


def test_two_streams_at_once(gsk):
    """Calls of different sizes on two streams, forward and gradient, with nothing between
    them: each has its own workspace, and its own results."""
    sets = []
    for i, (nq, nk, H, KV, D) in enumerate([([700, 300], None, 8, 2, 128), ([5, 3, 1], [900, 200, 2000], 16, 2, 64)]):
        q, k, v = inputs(nq, nk or nq, H, KV, D, "bf16", i)
        sets.append((q, k, v, make(q.shape, "bf16", 9), i32(sums(nq)), None if nk is None else i32(sums(nk))))

    def step(q, k, v, g, cu, ck):
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.1, cu_k=ck)
        return (out, lse, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.1, cu_k=ck))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(40):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(r, w))


def test_many_sequences(gsk):
    """More sequences than a warp searches at a time, some empty, in both lists."""
    r = np.random.RandomState(3)
    nq = [int(x) for x in r.randint(0, 9, 1500)]
    nk = [a + int(x) * (i % 3 == 0) for i, (a, x) in enumerate(zip(nq, r.randint(0, 40, 1500)))]
    q, k, v = inputs(nq, nk, 2, 1, 64, "bf16", 1)
    check(gsk, q, k, v, sums(nq), sums(nk), 0.125)


def test_long_and_wide(gsk):
    """Strides past 2^31 bytes."""
    n, D = 3, 64
    hold = torch.empty(2 * (2 ** 30 + 512) + 256, dtype=torch.bfloat16, device="cuda")
    x = hold.as_strided((n, 3, D), (2 ** 30 + 512, D, 1))
    x.copy_(make((n, 3, D), "bf16", 1))
    q, k, v = x[:, :1], x[:, 1:2], x[:, 2:]
    check(gsk, q, k, v, [0, n], None, 0.125)


def test_empty(gsk):
    q, k, v = inputs([4], [4], 2, 1, 64, "bf16")
    out, lse = gsk.csa_prompt_attend(q[:0], k[:0], v[:0], i32([0, 0]), 1.0)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out, lse = gsk.csa_prompt_attend(q, k[:0], v[:0], i32([0, 4]), 1.0, cu_k=i32([0, 0]))
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = gsk.csa_prompt_attend_bwd(q, k[:0], v[:0], out, lse, q, i32([0, 4]), 1.0, cu_k=i32([0, 0]))
    assert (dq == 0).all() and dk.shape == (0, 1, 64)
    e, l = gsk.csa_prompt_attend(q[:0], k, v, i32([0, 0]), 1.0, cu_k=i32([0, 4]))
    dq, dk, dv = gsk.csa_prompt_attend_bwd(q[:0], k, v, e, l, q[:0], i32([0, 0]), 1.0, cu_k=i32([0, 4]))
    assert dq.shape == (0, 2, 64) and (dk == 0).all() and (dv == 0).all()


def test_lists_that_make_no_sense_stay_inside(gsk):
    q, k, v = inputs([300], [300], 2, 1, 64, "bf16")
    g = make(q.shape, "bf16", 3)
    hold = torch.full((400, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for cu_q, cu_k in (([0, 900], [0, 900]), ([-5, 300], [0, 300]), ([0, 200, 100], [0, 100, 300]), ([0, 300], [0, 301]),
                       ([0, 300], [-4, 300]), ([300, 0], [0, 300]), ([2 ** 31 - 1, -2 ** 31], [0, 10]), ([0, 100, 400], [0, 300, 310])):
        gsk.csa_prompt_attend(q, k, v, i32(cu_q), 0.125, cu_k=i32(cu_k), out=hold[50:350])
        out, lse = gsk.csa_prompt_attend(q, k, v, i32(cu_q), 0.125, cu_k=i32(cu_k))
        gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, i32(cu_q), 0.125, cu_k=i32(cu_k))
        torch.cuda.synchronize()
        assert (hold[:50] == 7).all() and (hold[350:] == 7).all()


def test_refusals(gsk):
    q, k, v = inputs([8], [8], 4, 2, 64, "bf16")
    cu = i32([0, 8])
    call = lambda **kw: gsk.csa_prompt_attend(**{**dict(q=q, k=k, v=v, cu_q=cu, sm_scale=0.125), **kw})  # noqa: E731
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(cu_q=cu.long()), dict(out=q.float())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(k=k[:4]), dict(k=k[:4], v=v[:4]), dict(q=q[:, :3]), dict(window=0), dict(cu_k=i32([0, 4, 8])), dict(cu_q=cu[:1]),
                dict(out=q), dict(out=q[:4]), dict(lse=torch.zeros(8, 3, device="cuda")), dict(k=k[..., :32], v=v[..., :32]),
                dict(q=q.transpose(1, 2)), dict(rest=q[:4]), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    big = make((8, 4, 136), "bf16", 1)
    for bad in (dict(sm_scale=0.0), dict(sm_scale=-1.0), dict(sm_scale=math.inf), dict(sm_scale=math.nan),
                dict(q=big, k=big, v=big), dict(q=big[..., :12], k=big[..., :12], v=big[..., :12]),   # columns
                dict(q=big[..., 4:68], k=big[..., 4:68], v=big[..., 4:68]),                           # alignment
                dict(k=k[:, :1].expand(8, 2, 64)),                                                    # a broadcast head
                dict(q=make((8, 258, 64), "bf16", 2), k=k, v=v)):                                     # 129 heads a key head
        with pytest.raises(gsk.CsaError):
            call(**bad)
    out, lse = call()
    back = lambda **kw: gsk.csa_prompt_attend_bwd(**{**dict(q=q, k=k, v=v, out=out, lse=lse, grad=q, cu_q=cu, sm_scale=0.125), **kw})  # noqa: E731
    for bad in (dict(grad=q[:4]), dict(out=out[:4]), dict(lse=lse[:, :2]), dict(grad_lse=lse[:4]), dict(rest=out[:4])):
        with pytest.raises(ValueError):
            back(**bad)
    with pytest.raises(gsk.CsaError):
        back(grad=q[:1].expand(8, 4, 64))


def test_capture_streams_and_outputs_of_the_callers(gsk):
    from gated_softmax_kv_gb300 import autograd
    nq, H, KV, D = [150, 40], 4, 2, 64
    q, k, v = (t.requires_grad_() for t in inputs(nq, nq, H, KV, D, "bf16", 4))
    g, cu = make(q.shape, "bf16", 5), i32(sums(nq))

    def step():
        out, lse = autograd.prompt_attend(q, k, v, cu, 0.125)
        return (out, lse, *torch.autograd.grad(out, [q, k, v], g))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:                                    # two graphs share the pool's workspace
        with torch.cuda.graph(graph):
            outs.append(step())
    with torch.no_grad():
        for t, s in ((q, 6), (k, 7), (v, 8), (g, 9)):
            t.copy_(make(t.shape, "bf16", s))
        cu.copy_(i32([0, 33, 190]))
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    want = [t.detach().clone() for t in step()]
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = gsk.csa_prompt_attend(q.detach(), k.detach(), v.detach(), cu, 0.125, stream=s)
    back = gsk.csa_prompt_attend_bwd(q.detach(), k.detach(), v.detach(), out, lse, g, cu, 0.125, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(back[2], want[4])
    hold = torch.zeros_like(out)
    w = torch.ones_like(out, requires_grad=True)
    total = (w * hold).sum()
    gsk.csa_prompt_attend(q.detach(), k.detach(), v.detach(), cu, 0.125, out=hold)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        total.backward()
