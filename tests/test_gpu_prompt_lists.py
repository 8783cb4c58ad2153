"""Lists of attention over packed sequences that pass the tensors: every row of a result is
written, and what the other sequences get is what they get alone."""
import math

import pytest

from test_gpu_prompt import gsk, i32, inputs, make  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def dirty(like):
    """Leaves memory of these sizes full of sevens to the allocator."""
    held = [torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in like]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("H,KV,D", [(2, 1, 64), (6, 2, 128), (128, 1, 64)])
@pytest.mark.parametrize("cu_q,cu_k,good", [
    ([0, 100, 300], [0, 100, 400], 1),            # the last sequence's keys end behind the tensor
    ([0, 100, 400], [0, 100, 300], 1),            # its queries do
    ([0, 100, 200, 300], [0, 100, 500, 600], 1),  # and the next begins there
    ([0, 300], [0, 301], 0), ([0, 301], [0, 300], 0), ([0, 300], [-4, 300], 0), ([-5, 300], [0, 300], 0)])
def test_sequences_that_pass_the_tensors_see_nothing(gsk, cu_q, cu_k, good, H, KV, D):  # noqa: F811
    q, k, v = inputs([300], [300], H, KV, D, "bf16", 1)
    g = make(q.shape, "bf16", 2)
    n = 100 if good else 0
    rest = torch.empty_like(q)
    dirty([q, q[..., 0].float()])
    out, lse = gsk.csa_prompt_attend(q, k, v, i32(cu_q), 0.125, cu_k=i32(cu_k))
    gsk.csa_prompt_attend(q, k, v, i32(cu_q), 0.125, cu_k=i32(cu_k), rest=rest)
    dirty([q, k, v])
    dq, dk, dv = gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, i32(cu_q), 0.125, cu_k=i32(cu_k), rest=rest)
    if good:
        wo, wl = gsk.csa_prompt_attend(q[:n], k[:n], v[:n], i32([0, n]), 0.125)
        back = gsk.csa_prompt_attend_bwd(q[:n], k[:n], v[:n], wo, wl, g[:n], i32([0, n]), 0.125, rest=rest[:n].contiguous())
        assert torch.equal(out[:n], wo) and torch.equal(lse[:n], wl)
        for a, b in zip((dq, dk, dv), back):
            assert torch.equal(a[:n], b)
    assert (out[n:] == 0).all() and (rest[n:] == 0).all() and (lse[n:] == -math.inf).all()
    for t in (dq, dk, dv):
        assert (t[n:] == 0).all()
