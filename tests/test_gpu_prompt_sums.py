"""Sums over very many rows, in the gradient of attention over packed sequences."""
import pytest

from test_gpu_prompt import check, gsk, i32, inputs, make, sums  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_a_long_sequence_of_many_heads_over_one(gsk):  # noqa: F811
    """Sampled rows against the formulas in 64 bits, from the kernel's own lse (itself compared).
    Roundings of P, dS and of the results are independent: 2.5 half steps of a row's norm, as test_gpu_prompt.py
    holds whole results to; lse by its tolerance there (100003 sums of fp32, truncated)."""
    T, H, D, scale, U = 100003, 64, 64, 0.125, 2.0 ** -24
    q, k, v = inputs([T], [T], H, 1, D, "bf16", 3, scale=1.0)
    g, cu = make(q.shape, "bf16", 4), i32([0, T])
    rest = torch.empty_like(q)
    out, lse = gsk.csa_prompt_attend(q, k, v, cu, scale, rest=rest)
    dq, dk, dv = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, scale, rest=rest)
    x, y, e = k[:, 0].double(), v[:, 0].double(), 2.0 ** -8

    def near(a, b):
        assert (a.double() - b).norm() <= 2.5 * e * b.norm()

    for t in (0, 1, 777, 50000, T - 1):
        z = q[t].double() @ x[: t + 1].T * scale
        want = torch.logsumexp(z, -1)
        assert ((lse[t].double() - want).abs() <= 2 * (T + 8) * U + 4 * U * want.abs() + 1e-4).all()
        p = torch.softmax(z, -1)
        o = p @ y[: t + 1]
        near(out[t], o)
        ds = p * (g[t].double() @ y[: t + 1].T - (g[t].double() * o).sum(-1, keepdim=True))
        if t:
            near(dq[t], ds @ x[: t + 1] * scale)
        else:
            assert (dq[t] == 0).all()
    for j in (0, 3, 50001, 99000):
        wk, wv = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
        for h in range(0, H, 8):
            a, b, o = (s[j:, h: h + 8].double() for s in (q, g, out))
            o += rest[j:, h: h + 8].double()
            p = (a @ x[j] * scale - lse[j:, h: h + 8].double()).exp()
            ds = p * (b @ y[j] - (b * o).sum(-1))
            if j == 0:
                ds[0] = 0                                  # query 0 sees this key alone
            wk += torch.einsum("th,thd->d", ds, a) * scale
            wv += torch.einsum("th,thd->d", p, b)
        near(dk[j, 0], wk)
        near(dv[j, 0], wv)


@pytest.mark.parametrize("dtype,D,window", [("bf16", 64, None), ("fp16", 128, None), ("bf16", 128, 600)])
def test_items_of_several_stretches(gsk, dtype, D, window):  # noqa: F811
    """128 heads over one: a tile a token, so that a block of keys meets up to 1500 tiles, and CTAs do
    several such items; the same bits each time, and beside another call on a second stream."""
    nq = [1500, 3, 700]
    q, k, v = inputs(nq, nq, 128, 1, D, dtype, 3)
    cu, scale = i32(sums(nq)), D ** -0.5
    out, lse = check(gsk, q, k, v, sums(nq), None, scale, window=window, dtype=dtype)
    g = make(q.shape, dtype, 9)
    want = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, scale, window=window)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(8):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, scale, window=window))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_stretches_in_graphs(gsk):  # noqa: F811
    """Two captured calls, replayed one behind the other and again, on inputs that change between."""
    q, k, v = inputs([900, 700], [900, 700], 128, 1, 64, "bf16", 1)
    g, cu = make(q.shape, "bf16", 2), i32([0, 900, 1600])

    def step():
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.125)
        return (out, lse, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.125))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(step())
    for seed in (5, 9):
        for i, t in enumerate((q, k, v, g)):
            t.copy_(make(t.shape, "bf16", seed + i))
        for graph in graphs * 2:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_sums_of_like_terms_are_not_biased(gsk):  # noqa: F811
    """dV of a key that every query weighs the same, of gradients that are all 1: 128 heads by 4000 tokens over
    one key each, 512000 terms of 1. What is truncated on the way would be missing from the sum."""
    T, H, D = 4000, 128, 64
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    k, v = make((T, 1, D), "bf16", 1), make((T, 1, D), "bf16", 2)
    cu = i32([0, T])
    out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.125)
    dv = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, torch.ones_like(q), cu, 0.125)[2].double()
    # query t weighs each of its t + 1 keys 1 / (t + 1), rounded to bf16 (half a step, 2^-8, alike for all heads)
    w = (1.0 / torch.arange(1, T + 1, device="cuda", dtype=torch.float64)).bfloat16().double() * H
    want = w.flip(0).cumsum(0).flip(0)[:, None, None].expand_as(dv)
    # the result's own half step, 512 tiles of 8 truncations of 2^-24, and lse's and the exponential's roundings of
    # weights that lie beside a tie of bf16: a step, 2^-7, of fewer than one in 64
    assert ((dv - want).abs() <= (2.0 ** -8 + 4096 * 2.0 ** -24 + 2.0 ** -13) * want).all()
