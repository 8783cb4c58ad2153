"""Gradients of attention over packed sequences in fp16 beside rows that are not finite: dS is
scaled by one power of two for the whole call, in which only finite rows that see keys have a say.

Tolerance: another power of two rounds dS the same way but for what falls below fp16's normal range (2^-14, at most
2^-25 lost of weights whose largest is near 2^13), so a gradient moves by its own rounding at most, a step
of 2^-10 relative to each element, and its norm by no more than that of its norm."""
import math

import pytest

from test_gpu_prompt import gsk, i32, inputs, make, sums  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def near(got, want):
    assert torch.isfinite(got).all()
    a, b = got.double(), want.double()
    assert (a - b).norm() <= 2.0 ** -10 * b.norm()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name", ["q", "grad", "k", "v", "grad_lse"])
def test_a_row_that_is_not_finite_leaves_other_sequences_alone(gsk, name, bad):  # noqa: F811
    """Unit normals of 64 columns: P |dP - delta| is above 2 in many rows of either sequence."""
    nq, H, KV, D = [200, 90], 2, 1, 64
    for at in (3, 199, 230):
        q, k, v = inputs(nq, nq, H, KV, D, "fp16", at)
        g, gl = make(q.shape, "fp16", at + 5), torch.randn((290, H), generator=torch.Generator().manual_seed(at)).cuda()
        cu = i32(sums(nq))

        def grads():
            out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.125)
            return gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.125, grad_lse=gl)

        want = grads()
        if name == "grad_lse":
            gl[at, 0] = bad
        else:
            {"q": q, "grad": g, "k": k, "v": v}[name][at, 0, 3] = bad
        got = grads()
        rows = slice(200, 290) if at < 200 else slice(0, 200)
        for a, b in zip(got, want):
            near(a[rows], b[rows])
        if bad != bad:                                     # an infinity may leave a key no weight, and no trace
            assert not all(torch.isfinite(t[:200] if at < 200 else t[200:]).all() for t in got)


def test_queries_without_keys_have_no_say(gsk):  # noqa: F811
    """lse is -inf there; its gradient in a join with another such row is NaN."""
    q, k, v = inputs([5, 120], [2, 120], 4, 2, 64, "fp16", 1)
    g, gl = make(q.shape, "fp16", 2), torch.randn((125, 4), generator=torch.Generator().manual_seed(3)).cuda()
    cu, ck = i32([0, 5, 125]), i32([0, 2, 122])
    out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.125, cu_k=ck)
    assert (lse[:3] == -math.inf).all() and torch.isfinite(lse[3:]).all()
    want = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.125, cu_k=ck, grad_lse=gl)
    for fill in (math.nan, math.inf, 60000.0):
        g[:3] = fill
        gl[:3] = fill
        got = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.125, cu_k=ck, grad_lse=gl)
        assert (got[0][:3] == 0).all()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_the_largest_gradient_of_lse(gsk):  # noqa: F811
    """A gradient of lse near fp32's largest is still a size: its row overflows fp16, and no row becomes NaN."""
    q, k, v = inputs([60], [60], 2, 1, 64, "fp16", 4)
    cu, gl = i32([0, 60]), torch.zeros((60, 2), device="cuda")
    out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.125)
    gl[50, 0] = 3.4e38
    dq, dk, dv = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, torch.zeros_like(q), cu, 0.125, grad_lse=gl)
    assert not torch.isnan(dq).any() and not torch.isnan(dk).any() and (dv == 0).all()
    assert torch.isinf(dq[50, 0]).any() and (dq[:50] == 0).all() and (dq[51:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_join_of_two_calls_where_a_query_sees_nothing_in_either(gsk, dtype):  # noqa: F811
    """A window joined with other rows through lse, with gradients: such a row is 0 and has no gradient,
    and leaves the others' alone."""
    from gated_softmax_kv_gb300 import autograd
    nq, D = [6, 50], 64
    q, k, v = (t.requires_grad_() for t in inputs(nq, [4, 50], 2, 1, D, dtype, 1))
    k2, v2 = (t.requires_grad_() for t in inputs(nq, [3, 70], 2, 1, D, dtype, 5)[1:])
    cu = i32(sums(nq))

    def join(q, k, v, k2, v2, cu, ck, ck2):
        o, lse = autograd.prompt_attend(q, k, v, cu, 0.125, cu_k=i32(ck), window=8)
        o2, lse2 = autograd.prompt_attend(q, k2, v2, cu, 0.125, cu_k=i32(ck2))
        both = torch.logaddexp(lse, lse2).clamp_min(-1e30)
        return (lse - both).exp()[..., None] * o + (lse2 - both).exp()[..., None] * o2

    out = join(q, k, v, k2, v2, cu, [0, 4, 54], [0, 3, 73])
    assert (out[:2] == 0).all() and (out[2:].abs().sum(-1) > 0).all()
    g = torch.randn(out.shape, generator=torch.Generator().manual_seed(2)).cuda()
    got = torch.autograd.grad(out, [q, k, v, k2, v2], g)
    assert all(torch.isfinite(t).all() for t in got) and (got[0][:2] == 0).all()
    # the second sequence alone
    alone = [t.detach()[n:].requires_grad_() for t, n in ((q, 6), (k, 4), (v, 4), (k2, 3), (v2, 3))]
    one = join(*alone, i32([0, 50]), [0, 50], [0, 70])
    assert torch.equal(one, out[6:])
    for a, b, n in zip(got, torch.autograd.grad(one, alone, g[6:]), (6, 4, 4, 3, 3)):
        near(a[n:], b)
