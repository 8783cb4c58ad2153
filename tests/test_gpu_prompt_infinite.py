"""Rows of queries, keys and gradients that hold infinities, in attention over packed sequences:
the same bits each time, and keys whose logits are -inf.

A key whose logit is -inf for every query that sees it has weight 0: out, lse, dq, dk and dv are those of the same
sequences with that key left out of every sum. Only the key's infinite column of dq (0 times infinity) is
not compared. Tolerance: roundings of P, dS and of the results are independent, so that the norm of a
result's error is within 2.5 half steps of its norm (test_gpu_prompt.py)."""
import math

import numpy as np
import pytest

import layer_ref
from test_gpu_prompt import DTYPES, gsk, i32, inputs, make, np64, sums  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int32 if t.dtype is torch.float32 else torch.int16)


@pytest.mark.parametrize("bad", [math.inf, -math.inf])
@pytest.mark.parametrize("name", ["q", "grad", "k", "v"])
@pytest.mark.parametrize("H,KV,D,window", [(4, 2, 64, 100), (3, 1, 128, None)])
def test_the_same_bits_each_time(gsk, name, bad, H, KV, D, window):  # noqa: F811
    nq = [300, 1, 190]
    q, k, v = inputs(nq, nq, H, KV, D, "bf16", 7)
    g, cu = make(q.shape, "bf16", 8), i32(sums(nq))
    t = {"q": q, "grad": g, "k": k, "v": v}[name]
    for at in range(5, 490, 40):
        t[at, 0, at % D] = bad
    runs = []
    for _ in range(40):
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.1, window=window)
        runs.append((out, lse, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.1, window=window)))
    torch.cuda.synchronize()
    for i, r in enumerate(runs):
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(r, runs[0])), i


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,KV,D,window", [(2, 1, 64, None), (3, 1, 64, None), (5, 1, 128, None), (6, 2, 128, 90)])
def test_keys_of_infinite_logits_have_no_weight(gsk, dtype, H, KV, D, window):  # noqa: F811
    nq, scale = [400, 150], 0.125
    q, k, v = inputs(nq, nq, H, KV, D, dtype, 3)
    g, cu, c = make(q.shape, dtype, 4), sums(nq), 3
    q[..., c] = q[..., c].abs() + 0.5
    at = [2, 77, 127, 128, 260, 399, 400, 530]
    k[at, :, c] = -math.inf
    x, y, w, gg = (np64(t) for t in (q, k, v, g))
    want, wlse, parts = layer_ref.prompt(x, y, w, cu, cu, scale, window)
    finite = np.where(np.isfinite(y), y, 0.0)               # their weights are 0
    grads, _ = layer_ref.prompt_grad(x, finite, w, cu, cu, scale, parts, want, gg)
    rest = torch.empty_like(q)
    out, lse = gsk.csa_prompt_attend(q, k, v, i32(cu), scale, window=window, rest=rest)
    got = [out, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, i32(cu), scale, window=window, rest=rest)]
    for t in ("dk", "dv"):
        assert (got[2 if t == "dk" else 3][at] == 0).all(), t
    keep = [i for i in range(D) if i != c]
    e = torch.finfo(DTYPES[dtype]).eps / 2
    assert (np.isfinite(np64(lse)) == np.isfinite(wlse)).all()
    for n, a, b in zip(("out", "dq", "dk", "dv"), got, (want, *grads)):
        a = np64(a)
        if n == "dq":
            a, b = a[..., keep], b[..., keep]
        assert np.isfinite(a).all(), (n, np.argwhere(~np.isfinite(a))[:4])
        assert np.linalg.norm(a - b) <= 2.5 * e * np.linalg.norm(b), (n, np.linalg.norm(a - b) / np.linalg.norm(b))
