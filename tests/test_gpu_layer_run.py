"""The operators of a layer as they are used together: projections, norms with the
rotation, attention over the prompt, its gradient; a local window joined with the
compressed rows of the cache; a prompt in chunks; a single token replayed from a graph."""
import numpy as np
import pytest

import cache_ref
import layer_ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

E = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().double().cpu().numpy()


def make(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16().cuda()


@pytest.mark.parametrize("window", [None, 50])
def test_a_training_step(gsk, window):
    """Norms with the rotation, then attention, both with gradients; autograd's chain is
    the calls one after the other, to the bit, and near the chain in 64 bits."""
    from gated_softmax_kv_gb300 import autograd
    H, KV, D, lens, spare = 4, 2, 64, [70, 131, 1], 6
    cu = np.concatenate([[0], np.cumsum(lens)])
    T, scale = cu[-1] + spare, D ** -0.5
    x = make((T, H + 2 * KV, D), 1).requires_grad_()        # a projection's output
    wq, wk = ((1 + 0.2 * make((D,), s).float()).requires_grad_() for s in (2, 3))
    f, _ = gsk.csa_rope_freqs(D)
    c, g = i32(cu.tolist()), make((T, H, D), 5)
    q, k = autograd.norm_rope(x[:, :H], wq, f, k=x[:, H: H + KV], k_weight=wk, cu_seqlens_comp=c, layout="half")
    out, lse = autograd.prompt_attend(q, k, x[:, H + KV:], c, scale, window=window)
    dx, dwq, dwk = torch.autograd.grad(out, [x, wq, wk], g)
    # the same by hand
    with torch.no_grad():
        kw = dict(cu_seqlens_comp=c, layout="half")
        q2, k2 = gsk.csa_norm_rope(x[:, :H], wq, f, k=x[:, H: H + KV], k_weight=wk, **kw)
        rest = torch.empty_like(q2)
        o2, l2 = gsk.csa_prompt_attend(q2, k2, x[:, H + KV:], c, scale, window=window, rest=rest)
        dq, dk, dv = gsk.csa_prompt_attend_bwd(q2, k2, x[:, H + KV:], o2, l2, g, c, scale, window=window, rest=rest)
        a = gsk.csa_norm_rope_bwd(x[:, :H], wq, f, dq, k=x[:, H: H + KV], k_weight=wk, k_grad=dk, **kw)
    assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(dwq, a[1]) and torch.equal(dwk, a[3])
    assert torch.equal(dx, torch.cat([a[0], a[2], dv], 1))
    # in 64 bits throughout
    pos = np.concatenate([np.arange(n) for n in lens] + [np.zeros(spare, int)])
    X, fn = np64(x), np64(f)
    Q, _ = layer_ref.norm_rope(X[:, :H], np64(wq), fn, pos, 1e-6, layout="half")
    K, _ = layer_ref.norm_rope(X[:, H: H + KV], np64(wk), fn, pos, 1e-6, layout="half")
    V, G = X[:, H + KV:], np64(g).copy()
    G[cu[-1]:] = 0
    want, _, parts = layer_ref.prompt(Q, K, V, cu.tolist(), cu.tolist(), scale, window)
    (rq, rk, rv), _ = layer_ref.prompt_grad(Q, K, V, cu.tolist(), cu.tolist(), scale, parts, want, G)
    ax, _, bq, _ = layer_ref.norm_rope_grad(X[:, :H], np64(wq), rq, fn, pos, 1e-6, layout="half")
    kx, _, bk, _ = layer_ref.norm_rope_grad(X[:, H: H + KV], np64(wk), rk, fn, pos, 1e-6, layout="half")
    # q and k are rounded, which moves a logit by at most 2 E of the largest, z, and a weight by 2 z of
    # that on either side of its sum; then come the weights' rounding, dS's, the gradients' and the
    # result's: each moves a norm by at most E of it
    z = scale * np.sqrt((Q ** 2).sum(-1)).max() * np.sqrt((K ** 2).sum(-1)).max()
    bound = (6 + 4 * z) * E
    for got, ref in ((out, want), (dx, np.concatenate([ax, kx, rv], 1)), (dwq, bq), (dwk, bk)):
        assert np.linalg.norm(np64(got) - ref) <= bound * np.linalg.norm(ref)


def test_a_prompt_in_chunks(gsk):
    """Chunks of a prompt behind what is held are the whole prompt's rows."""
    H, KV, D, n = 8, 2, 128, 333
    q, k, v = make((n, H, D), 1, 1.5), make((n, KV, D), 2), make((n, KV, D), 3)
    whole, lse = gsk.csa_prompt_attend(q, k, v, i32([0, n]), D ** -0.5)
    want, wlse, _ = layer_ref.prompt(np64(q), np64(k), np64(v), [0, n], [0, n], D ** -0.5)
    mass, _, _ = layer_ref.prompt(np64(q), np64(k), np.abs(np64(v)), [0, n], [0, n], D ** -0.5)
    for a, b in ((0, 1), (1, 100), (100, 300), (300, 333)):
        o, l = gsk.csa_prompt_attend(q[a:b], k[:b], v[:b], i32([0, b - a]), D ** -0.5, cu_k=i32([0, b]))
        # weights and result rounded: E each of what they are a part of, twice for the two sides of a
        # difference; sums and exponentials are 2^-12 of it at the most
        tol = 2 * (E * mass[a:b] + E * np.abs(want[a:b])) + 2.0 ** -12 * mass[a:b]
        assert (np.abs(np64(o) - np64(whole[a:b])) <= tol).all()
        assert np.abs(np64(l) - wlse[a:b]).max() <= 1e-4 and np.abs(np64(l) - np64(lse[a:b])).max() <= 1e-4


def test_a_window_joined_with_compressed_rows(gsk):
    """The last tokens as they are and the rows before them compressed: two calls joined by
    their lse are one softmax over both. Then a decoding step of it, replayed from a graph."""
    H, D, ratio, window, n = 16, 128, 4, 24, 150
    page, block = 16, 16
    rows = n // ratio
    kv, score = make((n, 2 * D), 1), make((n, 2 * D), 2)
    ape = torch.randn((ratio, 2 * D), generator=torch.Generator().manual_seed(3)).cuda()
    cu, cuc = i32([0, n]), i32([0, rows])
    f, _ = gsk.csa_rope_freqs(64)
    w = (1 + 0.2 * make((D,), 4).float())
    comp = gsk.csa_compress_fwd(kv, score, ape, cu, cuc, rows, ratio, 2, D)
    turned, _ = gsk.csa_norm_rope(comp, w, f, cu_seqlens_comp=cuc, ratio=ratio, offset=D - 64)
    cache = torch.zeros((4, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales, table = torch.zeros((4, 1, 1), device="cuda"), i32([[2, 0, 3]])
    held = i32([0])
    gsk.csa_cache_append(turned[:, None], cache, scales, table, held, cuc)
    held += rows
    qk = make((n, H + 1, D), 5)
    q, k = gsk.csa_norm_rope(qk[:, :H], w, f, k=qk[:, H:], k_weight=w, cu_seqlens_comp=cu, offset=D - 64)
    scale = D ** -0.5
    # a token sees the rows that end before its window begins
    visible = ((torch.arange(n, device="cuda") + 1 - window).clamp(min=0) // ratio).int()

    def joined(q, k, v, cu_q, cu_k, visible):
        o1, l1 = gsk.csa_prompt_attend(q, k, v, cu_q, scale, cu_k=cu_k, window=window)
        o2, l2 = gsk.csa_cache_attend(q, cache, scales, table, held, cu_q, 1, scale, shared=True, visible=visible)
        both = torch.logaddexp(l1, l2)
        return (l1 - both).exp()[..., None] * o1.float() + (l2 - both).exp()[..., None] * o2.float(), both

    got, lse = joined(q, k, k, cu, None, visible)
    x = cache_ref.TABLE[cache.view(torch.uint8).cpu().numpy()] * np64(scales).repeat(block, -1)[..., None]
    x = x[[2, 0, 3], 0].reshape(-1, D)[:rows]
    Q, K, vis = np64(q), np64(k)[:, 0], visible.tolist()
    for t in (0, 1, window, 60, 111, n - 1):
        keys = np.concatenate([x[: vis[t]], K[max(0, t + 1 - window): t + 1]])
        z = Q[t] @ keys.T * scale
        top = z.max(-1, keepdims=True)
        p = np.exp(z - top)
        want = p @ keys / p.sum(-1, keepdims=True)
        mass = p @ np.abs(keys) / p.sum(-1, keepdims=True)
        # each part's weights and result rounded to bf16, E each; sums and exponentials far below
        assert (np.abs(np64(got[t]) - want) <= (2 * E + 2.0 ** -12) * mass).all()
        assert np.abs(np64(lse[t]) - (np.log(p.sum(-1)) + top[:, 0])).max() <= 1e-4
    # the last token alone, over the window's keys: the same rows
    one, last = i32([0, 1]), slice(n - window, n)
    new, place = qk[n - 1:].clone(), torch.tensor([n - 1], device="cuda")
    ring = k[last].clone()

    def step():
        q1, k1 = gsk.csa_norm_rope(new[:, :H], w, f, place, k=new[:, H:], k_weight=w, offset=D - 64)
        ring[-1:].copy_(k1)
        return joined(q1, ring, ring, one, ends, visible[n - 1:])

    ends = i32([0, window])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    ring.zero_()
    ring[:-1].copy_(k[last][:-1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ring, k[last])
    assert (np.abs(np64(out[0][0]) - np64(got[n - 1])) <= 2 * (2 * E + 2.0 ** -12) * mass).all()
    assert np.abs(np64(out[1][0]) - np64(lse[n - 1])).max() <= 2e-4
